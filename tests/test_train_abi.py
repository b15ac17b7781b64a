"""The gated feed-forward block and the optimizer step: exports of the header,
and the refusal of invalid arguments on the host before anything is enqueued.

CPU only: every call fails validation or has nothing to do, so no HIP runtime
call is made.
"""
import ctypes
import math
import os
import re

import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from fp8_fine_grained_quantize_amd import train

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "libfp8blk_train.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p
FAKE = P(0x100000)  # never dereferenced
MIS = P(0x100002)   # aligned for 2-byte elements only
ODD = P(0x100001)
NULL = P(0)


def test_exports_every_declared_symbol():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"\b(fp8blk_[a-z0-9_]+)\s*\(", text)))
    assert sorted(fb.TRAIN_SYMBOLS) == declared
    for name in declared:
        assert hasattr(fb.lib(), name), name
    assert fb.train_abi_version() == 1
    for name in fb.__all__:
        assert hasattr(fb, name), name


F32, BF16, E4M3 = 0, 1, 2


def _entry(**kw):
    d = dict(param=0x100000, grad=0x200000, m=0x300000, v=0x400000, m_scale=None, v_scale=None, copy=None, rows=3,
             cols=20, ldp=20, ldg=20, ldc=0, decay=0.1, flags=3, index=0, reserved=0)
    d.update(kw)
    return train._Tensor(*d.values())


def _build(state=F32, n=1, chunks=True, room=None, **kw):
    L = fb.lib()
    table = torch.zeros(64, dtype=torch.int64)
    nb = L.fp8blk_adamw_table_bytes(1) if room is None else room
    c = ctypes.c_int64(-7)
    e = _entry(**kw)
    got = L.fp8blk_adamw_table_build(ctypes.byref(e), n, state, table.data_ptr(), nb,
                                     ctypes.cast(ctypes.pointer(c), P) if chunks else None)
    return got, c.value


def test_table_refuses():
    assert _build() == (OK, 1) and _build(rows=1, cols=1025, ldp=1025, ldg=1025) == (OK, 2)
    assert _build(n=0) == (OK, 0)
    scaled = dict(m_scale=0x500000, v_scale=0x600000)
    assert _build(E4M3, **scaled) == (OK, 1) and _build(BF16, m=0x300002, v=0x400002) == (OK, 1)
    assert _build(flags=0, param=0x100002, grad=0x200002) == (OK, 1)
    for bad in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=0x100002), dict(grad=0x200002),
                dict(m=0x300002), dict(v=0x400002), dict(rows=0), dict(cols=0), dict(rows=-1), dict(ldp=19), dict(ldg=19),
                dict(copy=0x700000, ldc=19), dict(copy=0x700001, ldc=20), dict(flags=4), dict(reserved=1),
                dict(n=-1), dict(chunks=False), dict(room=8), dict(state=3), dict(state=-1), scaled,
                dict(m_scale=0x500000), dict(ldp=2 ** 62), dict(rows=2 ** 60)):
        assert _build(**bad)[0] == INVALID, bad
    for bad in (dict(), dict(m_scale=0x500000), dict(scaled, v_scale=0x600002), dict(scaled, m=0x300002)):
        assert _build(E4M3, **bad)[0] == INVALID, bad


class _Step(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("lr_at", P),
                ("step_at", P), ("seed_at", P), ("norm", P), ("max_norm", ctypes.c_float), ("clip_eps", ctypes.c_float)]


def _step(table=FAKE, n=1, chunks=1, state=F32, args=True, **kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, seed=0, flags=0, lr_at=None, step_at=None, seed_at=None,
             norm=None, max_norm=0.0, clip_eps=0.0)
    d.update(kw)
    s = _Step(*d.values())
    return fb.lib().fp8blk_adamw_step(table, n, chunks, state, ctypes.byref(s) if args else None, NULL)


def test_step_refuses():
    for bad in (dict(table=NULL), dict(table=P(0x100004)), dict(n=-1), dict(chunks=0), dict(n=0), dict(state=3),
                dict(args=False), dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=1.0), dict(beta2=math.nan), dict(eps=-1e-8), dict(eps=math.nan), dict(step=0), dict(flags=2),
                dict(lr_at=0x100002), dict(step_at=0x100004), dict(seed_at=0x100004), dict(norm=0x100002),
                dict(norm=0x100000, max_norm=-1.0), dict(norm=0x100000, max_norm=math.nan),
                dict(norm=0x100000, clip_eps=-1.0)):
        assert _step(**bad) == INVALID, bad
    assert _step(n=0, chunks=0, table=NULL) == OK


# --- the binding's lists, on the CPU ----------------------------------------

def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _rows_of(p, g, c=None):
    e = train._entries(fb.AdamWState([p], copies=None if c is None else [c]), [g])
    return [(x.rows, x.cols, x.ldp, x.ldg, x.ldc) for x in e]


def test_layouts():
    assert _rows_of(_t(3, 4, 5), _t(3, 4, 5)) == [(1, 60, 60, 60, 60)]
    assert _rows_of(_t(()), _t(())) == [(1, 1, 1, 1, 1)] and _rows_of(_t(0, 4), _t(0, 4)) == []
    wide = _t(6, 24)
    assert _rows_of(wide[:, :20], _t(6, 20)) == [(6, 20, 24, 20, 20)]
    assert _rows_of(_t(6, 20), wide[:, :20], _t(6, 32, dtype=torch.bfloat16)[:, :20]) == [(6, 20, 20, 24, 32)]
    assert _rows_of(_t(2, 3, 24)[:, :, :20], _t(2, 3, 20)) == [(6, 20, 24, 20, 20)]
    assert _rows_of(_t(4, 7).t(), _t(4, 7).t()) == [(1, 28, 28, 28, 28)]    # the same order in both
    assert _rows_of(_t(9)[::2], _t(9)[::2]) == [(5, 1, 2, 2, 1)]
    assert _rows_of(_t(6, 24)[:, ::2], _t(6, 12)) == [(72, 1, 2, 1, 1)]      # evenly spaced throughout
    for p, g in ((_t(4, 7).t(), _t(7, 4)), (_t(6, 26)[:, :24:2], _t(6, 12)), (_t(2, 3, 24)[:, :, :20], _t(2, 4, 30)[:, :3, :20])):
        with pytest.raises(ValueError, match="same order"):
            _rows_of(p, g)
    with pytest.raises(ValueError, match="shape"):
        _rows_of(_t(4, 7), _t(7, 4))


def test_state_refuses():
    p = _t(10)
    s = fb.AdamWState([p, _t(300)], dtype=torch.float8_e4m3fn)
    assert [t.numel() for t in s.m_scales] == [1, 3] and s.ms[1].dtype == torch.uint8 and s.state == 2
    assert fb.AdamWState([p], dtype=torch.bfloat16).vs[0].dtype == torch.bfloat16
    assert fb.AdamWState([], decay=[]).params == []
    one, u8 = [_t(10)], [_t(10, dtype=torch.uint8)]
    for kw in (dict(ms=one), dict(ms=one, vs=[_t(9)]), dict(ms=one, vs=one, m_scales=[_t(1)], v_scales=[_t(1)]),
               dict(ms=u8, vs=u8), dict(ms=u8, vs=u8, m_scales=[_t(2)], v_scales=[_t(1)]), dict(decay=[0.1, 0.1]),
               dict(ms=one, vs=[_t(20)[::2]]), dict(copies=[_t(9, dtype=torch.bfloat16)]), dict(ms=[], vs=[]),
               dict(copies=[_t(1, dtype=torch.bfloat16).expand(10)])):
        with pytest.raises(ValueError):
            fb.AdamWState([p], **kw)
    for kw in (dict(ms=one, vs=[_t(10, dtype=torch.bfloat16)]), dict(dtype=torch.float16), dict(copies=one),
               dict(copies=[3]), dict(ms=[None], vs=one), dict(ms=u8, vs=u8, m_scales=[_t(1).double()], v_scales=[_t(1)])):
        with pytest.raises(TypeError):
            fb.AdamWState([p], **kw)
    with pytest.raises(TypeError, match="parameter 1 must be a tensor"):
        fb.AdamWState([p, None])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        fb.AdamWState([_t(3).double()])
    with pytest.raises(ValueError, match="share memory"):
        fb.AdamWState([_t(1).expand(4)])
    with pytest.raises(TypeError, match="AdamWState"):
        fb.adamw_table([p], one)
    with pytest.raises(TypeError, match="AdamWTable"):
        fb.adamw_step(fb.AdamWState([p]), 1e-3, 1)
    with pytest.raises(ValueError, match="1 parameters, 2 gradients"):
        fb.adamw_table(fb.AdamWState([p]), [p, p])
    with pytest.raises(ValueError, match="current GPU"):
        fb.adamw_table(fb.AdamWState([p]), one)


def _shared(params, grads, **kw):
    s = fb.AdamWState(params, **kw)
    e = train._entries(s, grads)
    return train._shared((train._Tensor * max(1, len(e)))(*e), len(e), s.state)


def test_lists_that_share_memory():
    a, b, g = _t(20), _t(20), _t(20)
    assert _shared([a, b], [g, g]) is None                       # gradients are only read
    assert _shared([a[:10], a[10:]], [g[:10], g[10:]]) is None
    t = _t(6, 24)
    assert _shared([t[:, :10], t[:, 10:]], [_t(6, 10), _t(6, 14)]) is None
    assert _shared([t[:, :11], t[:, 10:]], [_t(6, 11), _t(6, 14)]) is not None
    assert "parameter 0" in _shared([a, a], [g, b])              # a tied weight listed twice
    assert "gradient" in _shared([a], [a])
    assert "moment" in _shared([a], [g], ms=[b], vs=[b])
    assert "copy" in _shared([a], [g], copies=[g.view(torch.bfloat16)[:20]])
    q, sc = _t(256, dtype=torch.uint8), _t(4)
    p = [_t(128), _t(128)]
    kw = dict(ms=[q[:128], q[128:]], vs=[_t(128, dtype=torch.uint8), _t(128, dtype=torch.uint8)])
    assert _shared(p, p[::-1], **kw, m_scales=[sc[:1], sc[1:2]], v_scales=[sc[2:3], sc[3:]]) is not None  # each other's parameter
    g2 = [_t(128), _t(128)]
    assert _shared(p, g2, **kw, m_scales=[sc[:1], sc[1:2]], v_scales=[sc[2:3], sc[3:]]) is None
    assert "scales" in _shared(p, g2, **kw, m_scales=[sc[:1], sc[1:2]], v_scales=[sc[1:2], sc[3:]])


# --- the gated feed-forward block --------------------------------------------

def _gated(M=4, H=256, K=384, A=FAKE, lda=384, sA=FAKE, B=FAKE, ldb=512, opB=0, sB=FAKE, act=0, u=FAKE, ldu=512, h=FAKE,
           ldh=256, q=NULL, ldq=0, s=NULL, qflags=0):
    return fb.lib().fp8blk_gated_gemm_fp8_blockscaled(M, H, K, A, lda, sA, B, ldb, opB, sB, act, u, ldu, h, ldh, q, ldq, s,
                                                      qflags, NULL, 0, NULL)


def _gated_grad(M=4, H=256, K=384, A=FAKE, lda=384, sA=FAKE, B=FAKE, ldb=384, opB=1, sB=FAKE, act=0, u=FAKE, ldu=512,
                du=P(0x200000), lddu=512, h=FAKE, ldh=256, q=NULL, ldq=0, s=NULL, qflags=0):
    return fb.lib().fp8blk_gated_gemm_backward_fp8_blockscaled(M, H, K, A, lda, sA, B, ldb, opB, sB, act, u, ldu, du, lddu, h,
                                                               ldh, q, ldq, s, qflags, NULL, 0, NULL)


COMMON = [dict(M=-1), dict(H=-128), dict(K=-128), dict(H=100), dict(K=100), dict(K=0), dict(A=NULL), dict(A=MIS), dict(lda=368),
          dict(lda=392), dict(sA=NULL), dict(sA=MIS), dict(B=NULL), dict(B=MIS), dict(ldb=368), dict(opB=2), dict(opB=0x200),
          dict(sB=NULL), dict(sB=MIS), dict(act=2), dict(act=-1), dict(u=MIS), dict(ldu=504), dict(h=MIS), dict(ldh=248),
          dict(ldh=260), dict(q=FAKE, ldq=512), dict(s=FAKE), dict(q=MIS, ldq=512, s=FAKE), dict(q=FAKE, ldq=504, s=FAKE),
          dict(q=FAKE, ldq=512, s=MIS), dict(qflags=2)]


def test_gated_refuses():
    for bad in COMMON + [dict(h=NULL), dict(q=FAKE, ldq=240, s=FAKE)]:
        assert _gated(**bad) == INVALID, bad
    assert _gated(lda=2 ** 23) == UNSUPPORTED and _gated(ldb=2 ** 23) == UNSUPPORTED and _gated(M=2 ** 32) == UNSUPPORTED
    assert _gated(H=2 ** 20, opB=1, ldb=2 ** 12, ldu=2 ** 21, ldh=2 ** 20) == UNSUPPORTED  # up rows past 2^31 bytes
    assert _gated(M=0, A=NULL, sA=NULL) == OK and _gated(H=0, B=NULL, sB=NULL) == OK
    w = fb.lib().fp8blk_gated_gemm_workspace_bytes
    assert w(0, 256, 384) == 0 and w(16, 100, 384) == 0 and w(16, 256, 100) == 0 and w(-1, 256, 384) == 0
    assert w(8192, 2048, 7168) == 0 and w(2 ** 62, 2 ** 62 - 2 ** 62 % 128, 128) == 0
    most = 2 ** 31  # sizes whose products pass 64 bits
    assert w(most, most, most) == 0 and w(16, 256, 2 ** 62) == 0 and w(most + 1, 256, 128) == 0
    assert w(16, 256, 7168) >= 2 * 16 * 512 * 4 and w(16, 256, 7168) % (16 * 512 * 4) == 0  # two parts or more


def test_gated_gradient_refuses():
    for bad in COMMON + [dict(u=NULL), dict(du=NULL), dict(du=MIS), dict(lddu=504), dict(du=FAKE, lddu=520),
                         dict(q=FAKE, ldq=496, s=FAKE)]:
        assert _gated_grad(**bad) == INVALID, bad
    assert _gated_grad(lda=2 ** 23) == UNSUPPORTED and _gated_grad(ldb=2 ** 23) == UNSUPPORTED
    assert _gated_grad(M=0, A=NULL, sA=NULL, u=NULL) == OK and _gated_grad(H=0, B=NULL, sB=NULL) == OK
    w = fb.lib().fp8blk_gated_gemm_backward_workspace_bytes
    assert w(0, 256, 384) == 0 and w(8192, 4096, 7168) == 0 and w(16, 256, 384) % (16 * 256 * 4) == 0


def test_grouped_gated_refuses():
    def call(G=3, off=FAKE, M=4, most=0, strideB=384 * 512, opB=0, stride_sB=12, K=384, h=FAKE):
        return fb.lib().fp8blk_grouped_gated_gemm_fp8_blockscaled(G, off, M, most, 256, K, FAKE, 384, FAKE, FAKE, 512, strideB,
                                                                  opB, FAKE, stride_sB, 0, FAKE, 512, h, 256, NULL, 0, NULL,
                                                                  0, NULL)

    def grad(G=3, off=FAKE, M=4, most=0, strideB=384 * 256, opB=1, stride_sB=6, du=P(0x200000)):
        return fb.lib().fp8blk_grouped_gated_gemm_backward_fp8_blockscaled(
            G, off, M, most, 256, 384, FAKE, 384, FAKE, FAKE, 384, strideB, opB, FAKE, stride_sB, 0, FAKE, 512, du, 512, NULL,
            0, NULL, 0, NULL, 0, NULL)

    for f in (call, grad):
        for bad in (dict(G=-1), dict(off=NULL), dict(off=MIS), dict(M=-1), dict(most=-1), dict(strideB=100), dict(stride_sB=5),
                    dict(opB=7)):
            assert f(**bad) == INVALID, (f, bad)
        assert f(G=0) == OK and f(M=0) == OK
        assert f(G=2 ** 40) == UNSUPPORTED
    assert call(strideB=384 * 512 + 8) == INVALID and call(h=NULL) == INVALID and call(K=128 * 4) == INVALID
    assert grad(du=NULL) == INVALID


X = torch.zeros(4, 128, dtype=torch.uint8)
S = torch.zeros(1, 4)


@pytest.mark.parametrize("name,call", [
    ("A", lambda v: fb.gated_gemm_fp8_blockscaled(v, S, X, S)), ("sA", lambda v: fb.gated_gemm_fp8_blockscaled(X, v, X, S)),
    ("B", lambda v: fb.gated_gemm_fp8_blockscaled(X, S, v, S)), ("sB", lambda v: fb.gated_gemm_fp8_blockscaled(X, S, X, v)),
    ("offsets", lambda v: fb.grouped_gated_gemm_fp8_blockscaled(v, X, S, X, S)),
    ("offsets", lambda v: fb.grouped_gated_gemm_backward_fp8_blockscaled(v, X, S, X, S, X)),
    ("u", lambda v: fb.gated_gemm_backward_fp8_blockscaled(X, S, torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(1, 1), v))])
@pytest.mark.parametrize("value", [None, 3, [[1.0]], X.numpy()])
def test_no_tensor(name, call, value):
    with pytest.raises(TypeError, match=f"^{name} must be a tensor"):
        call(value)
