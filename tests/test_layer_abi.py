"""The operators around the GEMMs: exports of the header, and the refusal of
invalid arguments on the host before anything is enqueued.

CPU only: every call fails validation or has nothing to do, so no HIP runtime
call is made.
"""
import ctypes
import os
import re

import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from fp8_fine_grained_quantize_amd import layer

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "libfp8blk_layer.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p
FAKE = P(0x100000)  # never dereferenced
MIS = P(0x100002)   # aligned for 2-byte elements only
NULL = P(0)


def test_exports_every_declared_symbol():
    text = open(HEADER).read()
    declared = sorted(set(re.findall(r"\b(fp8blk_[a-z0-9_]+)\s*\(", text)))
    assert sorted(fb.LAYER_SYMBOLS) == declared
    for name in declared:
        assert hasattr(fb.lib(), name), name
    assert fb.layer_abi_version() == 1
    for name in fb.__all__:
        assert hasattr(fb, name), name


def test_sort_refuses():
    f = fb.lib().fp8blk_moe_sort

    def call(ids=FAKE, T=4, K=2, ld=2, E=8, off=FAKE, row=FAKE, slot=FAKE, ws=NULL, nb=0, flags=0):
        return f(ids, T, K, ld, E, off, row, slot, ws, nb, flags, NULL)

    for bad in (dict(ids=NULL), dict(off=NULL), dict(row=NULL), dict(slot=NULL), dict(ld=1), dict(T=-1), dict(K=-1),
                dict(E=-1), dict(flags=2), dict(ids=MIS), dict(off=MIS), dict(row=MIS), dict(slot=MIS),
                dict(ids=P(0x100004), flags=1)):
        assert call(**bad) == INVALID, bad
    assert call(E=961) == UNSUPPORTED
    assert call(T=2 ** 30, K=2) == UNSUPPORTED and call(T=2 ** 62, K=2 ** 62) == UNSUPPORTED
    need = fb.lib().fp8blk_moe_sort_workspace_bytes
    assert need(16, 8, 256) == 0 and need(-1, 8, 256) == 0 and need(8192, 8, 256) > 0
    nb = need(8192, 8, 256)
    assert call(T=8192, K=8, ld=8, E=256, ws=FAKE, nb=nb - 1) == INVALID
    assert call(T=8192, K=8, ld=8, E=256, ws=NULL, nb=nb) == INVALID
    assert call(T=8192, K=8, ld=8, E=256, ws=MIS, nb=nb) == INVALID


def test_dispatch_refuses():
    f = fb.lib().fp8blk_moe_dispatch

    def call(x=FAKE, T=4, C=64, ldx=64, K=2, row=FAKE, out=FAKE, ldo=64):
        return f(x, T, C, ldx, K, row, out, ldo, NULL)

    for bad in (dict(x=NULL), dict(out=NULL), dict(row=NULL), dict(ldx=56), dict(ldo=63), dict(ldx=68), dict(x=MIS),
                dict(out=MIS), dict(row=MIS), dict(T=-1), dict(C=-1), dict(K=-1)):
        assert call(**bad) == INVALID, bad
    assert call(T=2 ** 31, K=1) == UNSUPPORTED
    assert call(T=2 ** 24, C=4096, ldx=4096, ldo=4096) == UNSUPPORTED  # more lanes than a launch has
    for none in (dict(T=0), dict(K=0), dict(C=0)):
        assert call(x=NULL, row=NULL, out=NULL, **none) == OK
    g = fb.lib().fp8blk_moe_dispatch_fp8

    def call8(q=FAKE, T=4, C=64, ldq=64, s=FAKE, K=2, row=FAKE, slot=FAKE, qr=FAKE, ldqr=64, sr=FAKE):
        return g(q, T, C, ldq, s, K, row, slot, qr, ldqr, sr, NULL)

    for bad in (dict(q=NULL), dict(s=NULL), dict(row=NULL), dict(slot=NULL), dict(qr=NULL), dict(sr=NULL),
                dict(ldq=48), dict(ldqr=72), dict(q=MIS), dict(s=MIS), dict(sr=MIS), dict(slot=MIS)):
        assert call8(**bad) == INVALID, bad
    assert call8(T=0, q=NULL, s=NULL, row=NULL, slot=NULL, qr=NULL, sr=NULL) == OK


def test_combine_refuses():
    f = fb.lib().fp8blk_moe_combine

    def call(rows=FAKE, T=4, K=2, C=64, ldr=64, row=FAKE, w=FAKE, y=FAKE, ldy=64, flags=0):
        return f(rows, T, K, C, ldr, row, w, y, ldy, flags, NULL)

    for bad in (dict(rows=NULL), dict(row=NULL), dict(y=NULL), dict(ldr=56), dict(ldy=68), dict(rows=MIS), dict(y=MIS),
                dict(w=MIS), dict(flags=4), dict(T=-1), dict(K=-2), dict(C=-1), dict(flags=1, ldr=66)):
        assert call(**bad) == INVALID, bad
    assert call(T=0, rows=NULL, row=NULL, y=NULL) == OK and call(C=0, rows=NULL, y=NULL) == OK
    assert call(T=2 ** 22, K=1, C=2 ** 14, ldr=2 ** 14, ldy=2 ** 14) == UNSUPPORTED
    g = fb.lib().fp8blk_moe_combine_backward

    def callb(dy=FAKE, lddy=64, rows=FAKE, ldr=64, T=4, K=2, C=64, row=FAKE, w=FAKE, dr=FAKE, lddr=64, dw=FAKE, flags=0):
        return g(dy, lddy, rows, ldr, T, K, C, row, w, dr, lddr, dw, flags, NULL)

    for bad in (dict(dy=NULL), dict(rows=NULL), dict(row=NULL), dict(w=NULL), dict(dr=NULL), dict(dw=NULL),
                dict(lddy=60), dict(ldr=63), dict(lddr=56), dict(flags=8), dict(dw=MIS), dict(w=MIS), dict(T=-1)):
        assert callb(**bad) == INVALID, bad
    assert callb(T=0) == OK and callb(K=0) == OK


def test_norm_refuses():
    f = fb.lib().fp8blk_residual_norm

    def call(M=4, C=64, x=FAKE, ldx=64, f_=FAKE, ldf=64, wp=FAKE, gate=FAKE, ldg=0, wn=FAKE, eps=1e-6, xo=FAKE, ldxo=64,
             n=FAKE, ldn=64, q=FAKE, ldq=64, s=FAKE, r1=FAKE, r2=FAKE, flags=0):
        return f(M, C, x, ldx, f_, ldf, wp, gate, ldg, 1.0, wn, eps, xo, ldxo, n, ldn, q, ldq, s, r1, r2, flags, NULL)

    odd = P(0x100001)
    for bad in (dict(M=-1), dict(C=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(flags=2), dict(x=NULL),
                dict(x=MIS), dict(ldx=56), dict(ldx=68), dict(f_=NULL), dict(xo=NULL), dict(ldf=60), dict(ldxo=63),
                dict(wp=odd), dict(wn=odd), dict(gate=odd), dict(wp=MIS, flags=0x20), dict(gate=NULL, flags=0x40),
                dict(flags=0x40, ldg=60), dict(q=NULL), dict(s=NULL), dict(n=MIS), dict(q=MIS), dict(s=MIS), dict(ldn=63),
                dict(ldq=72), dict(wn=NULL), dict(n=NULL, q=NULL, s=NULL), dict(xo=P(0x100000), ldxo=72),
                dict(r1=MIS), dict(r2=MIS), dict(wp=NULL), dict(q=NULL, s=NULL, flags=1),
                dict(f_=NULL, wp=NULL, gate=NULL, r1=NULL),              # x_out without f
                dict(f_=NULL, wp=NULL, gate=NULL, r1=NULL, xo=NULL, wn=NULL, n=NULL, q=NULL, s=NULL, r2=NULL)):
        assert call(**bad) == INVALID, bad
    wide = 16385 + 7
    assert call(C=wide, ldx=16392, ldf=16392, ldxo=16392, ldn=16392, ldq=16400) == UNSUPPORTED
    assert call(M=0, x=NULL) == OK and call(C=0, x=NULL) == OK


def test_norm_backward_refuses():
    f = fb.lib().fp8blk_residual_norm_backward
    nb = 1 << 40

    def call(M=4, C=64, x=FAKE, ldx=64, dxo=FAKE, lddxo=64, dn=FAKE, lddn=64, r2=FAKE, wn=FAKE, f_=FAKE, ldf=64, r1=FAKE,
             wp=FAKE, gate=FAKE, ldg=64, dx=FAKE, lddx=64, df=FAKE, lddf=64, dwn=FAKE, dwp=FAKE, dg=FAKE, lddg=64,
             ws=FAKE, nb=nb, flags=0):
        return f(M, C, x, ldx, dxo, lddxo, dn, lddn, r2, wn, f_, ldf, r1, wp, gate, ldg, 1.0, dx, lddx, df, lddf, dwn,
                 dwp, dg, lddg, ws, nb, flags, NULL)

    for bad in (dict(M=-1), dict(C=-1), dict(flags=1), dict(x=NULL), dict(dn=NULL), dict(r2=NULL), dict(wn=NULL),
                dict(dwn=NULL), dict(f_=NULL), dict(df=NULL), dict(r1=NULL), dict(wp=NULL), dict(dwp=NULL),
                dict(gate=NULL), dict(dg=NULL), dict(ws=NULL), dict(nb=4), dict(ldx=56), dict(lddxo=60), dict(lddn=63),
                dict(ldf=56), dict(lddx=63), dict(lddf=60), dict(dg=MIS), dict(dwn=MIS), dict(dwp=MIS),
                dict(flags=0x40, lddg=60), dict(flags=0x40, ldg=60), dict(flags=0x20, wp=MIS), dict(ws=P(0x100008)),
                dict(dxo=NULL, dn=NULL, r2=NULL, wn=NULL, dwn=NULL)):
        assert call(**bad) == INVALID, bad
    assert call(C=16392) == UNSUPPORTED
    assert call(C=0) == OK
    need = fb.lib().fp8blk_residual_norm_backward_workspace_bytes
    assert need(0, 64) == 0 and need(4, 0) == 0 and need(4, 16392) == 0 and need(4, 64) > 0


def _grad(**k):
    g = layer._Grad(0x100000, 0x100000, 1, 100, 100, 100, 0x3, 0)
    for n, v in k.items():
        setattr(g, n, v)
    return g


def _build(*gs, nbytes=None):
    L = fb.lib()
    need = L.fp8blk_grad_table_bytes(len(gs)) if nbytes is None else nbytes
    buf = (ctypes.c_int64 * 64)()
    arr = (layer._Grad * max(1, len(gs)))(*gs)
    chunks = ctypes.c_int64(-1)
    st = L.fp8blk_grad_table_build(ctypes.cast(arr, P), len(gs), ctypes.cast(buf, P), need,
                                   ctypes.cast(ctypes.pointer(chunks), P))
    return st, chunks.value


def test_grad_table():
    assert _build(_grad()) == (OK, 1)
    one = _build(_grad(cols=8192, ld=8192, ldo=8192))[1]
    assert _build(_grad(cols=8192, ld=8192, ldo=8192), _grad(out=0x200000, rows=3, cols=8192, ld=9000, ldo=8192)) == \
        (OK, 4 * one)
    assert _build() == (OK, 0)
    for bad in (dict(grad=0), dict(out=0), dict(grad=0x100002), dict(out=0x100001, flags=0), dict(rows=0), dict(cols=0),
                dict(rows=-1), dict(ld=99), dict(ldo=99), dict(flags=4), dict(reserved=1), dict(flags=1),
                dict(ldo=200), dict(rows=2 ** 60, ld=2 ** 20, out=0x200000)):
        assert _build(_grad(**bad))[0] == INVALID, bad
    assert _build(_grad(), nbytes=8)[0] == INVALID
    L = fb.lib()
    assert L.fp8blk_grad_table_build(NULL, 1, FAKE, 1 << 20, FAKE) == INVALID
    assert L.fp8blk_grad_table_build(NULL, 0, NULL, 0, NULL) == INVALID
    assert L.fp8blk_grad_table_bytes(-1) == 0


def test_grad_calls_refuse():
    L = fb.lib()
    W = 16384
    for t, n, c, norm, ws, wb in ((NULL, 1, 1, FAKE, FAKE, W), (FAKE, -1, 1, FAKE, FAKE, W), (FAKE, 2, 1, FAKE, FAKE, W),
                                  (FAKE, 0, 1, FAKE, FAKE, W), (P(0x100004), 1, 1, FAKE, FAKE, W),
                                  (FAKE, 1, 1, NULL, FAKE, W), (FAKE, 1, 1, MIS, FAKE, W), (FAKE, 1, 1, FAKE, NULL, W),
                                  (FAKE, 1, 1, FAKE, P(0x100004), W), (FAKE, 1, 1, FAKE, FAKE, W - 1)):
        assert L.fp8blk_grad_norm(t, n, c, norm, ws, wb, NULL) == INVALID
        assert L.fp8blk_grad_clip_norm(t, n, c, 1.0, 0.0, norm, ws, wb, NULL) == INVALID
    for max_norm, eps in ((-1.0, 0.0), (float("nan"), 0.0), (1.0, -1.0), (1.0, float("nan"))):
        assert L.fp8blk_grad_clip_norm(FAKE, 1, 1, max_norm, eps, FAKE, FAKE, W, NULL) == INVALID
        assert L.fp8blk_grad_clip(FAKE, 1, 1, FAKE, max_norm, eps, NULL) == INVALID
    assert L.fp8blk_grad_clip(FAKE, 1, 1, NULL, 1.0, 0.0, NULL) == INVALID
    assert L.fp8blk_grad_clip(NULL, 0, 0, FAKE, 1.0, 0.0, NULL) == OK


def test_rows_of_gradients():
    """Every layout as evenly spaced rows, or not at all."""
    r = lambda t: layer._as_rows(t.shape, t.stride())  # noqa: E731
    t = torch.empty(6, 10, 8)
    assert r(t) == (1, 480, 480) and r(t.permute(2, 0, 1)) == (1, 480, 480)
    assert r(t[:, :, :5]) == (60, 5, 8) and r(t[:, 2:, :]) == (6, 64, 80) and r(t[:, 1:9, :5]) is None
    assert r(torch.empty(9)[::2]) == (5, 1, 2) and r(torch.empty(())) == (1, 1, 1)
    assert r(torch.empty(4, 1, 3)) == (1, 12, 12)
    entries = []
    layer._grad_entries(t[:, 1:9, :5], t[:, 1:9, :5], 3, entries)
    assert [(e.rows, e.cols, e.ld) for e in entries] == [(8, 5, 8)] * 6
    entries = []
    layer._grad_entries(torch.empty(4, 6).t(), torch.empty(6, 4), 3, entries)   # element order differs
    assert [(e.rows, e.cols, e.ld, e.ldo) for e in entries] == [(4, 1, 6, 1)] * 6


def test_shared_memory_is_found():
    t = torch.empty(6, 10, 8)
    for ok in (t, t.permute(1, 2, 0), t[:, 2:7, ::3], t[0, 0, 0], torch.empty(1, 5).expand(1, 5), torch.empty(0, 3)):
        assert not layer._overlaps(ok)
    for bad in (torch.empty(5, 1).expand(5, 4), torch.empty(20).as_strided((5, 4), (2, 1)),
                torch.empty(40).as_strided((3, 3, 3), (9, 2, 1))):
        assert layer._overlaps(bad)


def test_binding_refuses():
    """Shapes, types and devices are checked before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        fb.moe_sort(ids.float(), 8)
    with pytest.raises(ValueError):
        fb.moe_sort(ids, 8)  # not on a GPU
    with pytest.raises(TypeError):
        fb.moe_dispatch(x.float(), ids)
    with pytest.raises(ValueError):
        fb.moe_dispatch(x, ids)
    with pytest.raises(ValueError):
        fb.residual_norm(x, w_pre=torch.ones(64))
    with pytest.raises(ValueError):
        fb.grad_norm([x])
    for bad in (x[:1].expand(4, 64), x.t(), x[:, ::2]):  # rows on top of each other, columns apart
        with pytest.raises(ValueError, match="row-major|shape|T ="):
            fb.moe_dispatch(bad, ids)
    with pytest.raises(TypeError):
        fb.moe_combine(torch.zeros(8, 64, dtype=torch.bfloat16), ids, weights=3)
    with pytest.raises(TypeError):
        fb.moe_combine(torch.zeros(8, 64, dtype=torch.float16), ids)
    with pytest.raises(ValueError):
        fb.residual_norm(x, w_pre=torch.ones(63))
    with pytest.raises(TypeError):
        fb.residual_norm(x, w_pre=torch.ones(64), f=x, w_post=torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        fb.residual_norm(x)
    with pytest.raises(ValueError):
        fb.residual_norm_backward(x, dx_out=x, dn=x)
    with pytest.raises(ValueError):
        fb.residual_norm_backward(x)
    lent = torch.zeros(1, dtype=torch.int32).expand(1 << 20)  # four bytes, however long
    with pytest.raises(ValueError, match="contiguous"):
        fb.moe_sort(ids, 8, workspace=lent)
    with pytest.raises(ValueError, match="contiguous"):
        fb.residual_norm_backward(x, dx_out=x, workspace=lent)


def test_binding_fails_loudly_without_its_extension(monkeypatch):
    import sys
    monkeypatch.setattr(layer, "_EXT", None)
    monkeypatch.delattr(fb, "_layer_ext", raising=False)
    monkeypatch.setitem(sys.modules, "fp8_fine_grained_quantize_amd._layer_ext", None)  # as if it were missing
    with pytest.raises(fb.Fp8BlkError, match="build"):
        layer._ext()
