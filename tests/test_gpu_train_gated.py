"""GPU tests of the gated feed-forward block and its gradient.

The fused forms accumulate as gemm_fp8_blockscaled does, so that u equals that
GEMM's BF16 output bit for bit, and h, du are compared with 64-bit forms of its
FP32 output (bounds in train_ref.py); codes and scales equal quantize_1x128 of
the BF16 result bit for bit.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import train_ref as ref
from tests.layer_ref import U, UB

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _bf16(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def _np(t):
    return t.detach().cpu().double().numpy()


def _weights(rows, cols, seed, pow2, G=None):
    """Codes and block scales; G: of every expert."""
    if G is None:
        return fb.quantize_block128(_bf16((rows, cols), seed, 0.05), pow2=pow2)
    q, s = fb.quantize_block128(_bf16((G * rows, cols), seed, 0.05), pow2=pow2)
    return q.view(G, rows, cols), s.view(G, rows // 128, cols // 128)


def _half(x, e):
    return np.abs(x) * UB + e * (1 + UB) + 2.0 ** -134


def _check_h(h, C, H, act, eu=None):
    g, v = C[:, :H], C[:, H:]
    want, e = ref.gated(g, v, act)
    if eu is not None:
        e = e + ref.gated_slope(g, v, act, eu[:, :H], eu[:, H:])
    assert np.all(np.abs(_np(h) - want) <= _half(want, e))


def _check_grad(r, dh, u, act, ed=0.0):
    H = u.shape[1] // 2
    g, v = _np(u[:, :H]), _np(u[:, H:])
    want = ref.gated_grad(dh, g, v, act)
    unit = ref.gated_grad(np.ones_like(dh), g, v, act)  # what an error of dh becomes
    for name, got in (("dg", r.du[:, :H]), ("dv", r.du[:, H:]), ("h", r.h)):
        x, e = want[name]
        if name != "h":
            e = e + ed * np.abs(unit[name][0]) * (1 + 2.0 ** -20)
        assert np.all(np.abs(_np(got) - x) <= _half(x, e)), name


def _split_error(x, sx, w, sw, opB, M, N):
    """How far two orders of adding the same group products can lie apart: the sums over the groups differ by
    fewer than 2 (groups + splits) roundings of at most the sum of magnitudes."""
    K = x.shape[1]
    A = (x.view(torch.float8_e4m3fn).float().abs().view(M, K // 128, 128) * sx.t()[:, :, None]).view(M, K).double()
    B = w.view(torch.float8_e4m3fn).double().abs() * sw.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return _np(A @ (B.t().contiguous() if opB else B)) * U * 2 * (K // 128 + 16)


MS = [1, 5, 127, 129, 256, 257, 777]


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("K,H", [(128, 128), (384, 256), (1152, 384)])
@pytest.mark.parametrize("act,opB,pow2", [("silu", 0, False), ("gelu", 1, True), ("silu", 1, False), ("gelu", 0, True)])
def test_forward(M, K, H, act, opB, pow2):
    print(f"[train] gated {M} {K} {H} {act} {opB} {pow2}", flush=True)
    x, sx = fb.quantize_1x128(_bf16((M, K), 1), pow2=pow2)
    w, sw = _weights(*((2 * H, K) if opB else (K, 2 * H)), 2, pow2)
    C = fb.gemm_fp8_blockscaled(x, sx, w, sw, opB=opB, split_k=False, pow2_scales=pow2)
    r = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, act=act, opB=opB, pow2_scales=pow2, quantize=True, pow2=pow2,
                                      split_k=False)
    assert torch.equal(r.u, C.to(BF))
    _check_h(r.h, _np(C), H, act)
    q, s = fb.quantize_1x128(r.h, pow2=pow2)
    assert torch.equal(r.q, q) and torch.equal(r.s, s)
    # fewer outputs, the other kind of scale: the same values
    only = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, act=act, opB=opB, pow2_scales=pow2, quantize=True, pow2=not pow2,
                                         want_h=False, want_u=False, split_k=False)
    q, s = fb.quantize_1x128(r.h, pow2=not pow2)
    assert only.u is None and only.h is None and torch.equal(only.q, q) and torch.equal(only.s, s)
    # split over K and joined
    e = _split_error(x, sx, w, sw, opB, M, 2 * H)
    j = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, act=act, opB=opB, pow2_scales=pow2, quantize=True, pow2=pow2)
    assert np.all(np.abs(_np(j.u) - _np(C)) <= _half(_np(C), e))
    _check_h(j.h, _np(C), H, act, e)
    q, s = fb.quantize_1x128(j.h, pow2=pow2)
    assert torch.equal(j.q, q) and torch.equal(j.s, s)


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("K,H", [(128, 128), (384, 256), (1152, 384)])
@pytest.mark.parametrize("act,opB,pow2", [("silu", 1, False), ("gelu", 0, True), ("silu", 0, False), ("gelu", 1, True)])
def test_gradient(M, K, H, act, opB, pow2):
    print(f"[train] gated gradient {M} {K} {H} {act} {opB} {pow2}", flush=True)
    x, sx = fb.quantize_1x128(_bf16((M, K), 1), pow2=pow2)
    w, sw = _weights(*((H, K) if opB else (K, H)), 2, pow2)
    u = _bf16((M, 2 * H), 3, 2.0)
    dh = fb.gemm_fp8_blockscaled(x, sx, w, sw, opB=opB, split_k=False, pow2_scales=pow2)
    kw = dict(act=act, opB=opB, pow2_scales=pow2, quantize=True, pow2=pow2)
    r = fb.gated_gemm_backward_fp8_blockscaled(x, sx, w, sw, u, split_k=False, **kw)
    _check_grad(r, _np(dh), u, act)
    q, s = fb.quantize_1x128(r.du, pow2=pow2)
    assert torch.equal(r.q, q) and torch.equal(r.s, s)
    only = fb.gated_gemm_backward_fp8_blockscaled(x, sx, w, sw, u, split_k=False, want_h=False, want_du=False,
                                                  **dict(kw, pow2=not pow2))
    q, s = fb.quantize_1x128(r.du, pow2=not pow2)
    assert only.du is None and only.h is None and torch.equal(only.q, q) and torch.equal(only.s, s)
    j = fb.gated_gemm_backward_fp8_blockscaled(x, sx, w, sw, u, **kw)
    _check_grad(j, _np(dh), u, act, _split_error(x, sx, w, sw, opB, M, H))
    q, s = fb.quantize_1x128(j.du, pow2=pow2)
    assert torch.equal(j.q, q) and torch.equal(j.s, s)
    for split, want in ((False, r), (True, j)):  # in place
        v = u.clone()
        got = fb.gated_gemm_backward_fp8_blockscaled(x, sx, w, sw, v, split_k=split, du=v, **kw)
        assert got.du.data_ptr() == v.data_ptr() and torch.equal(v, want.du) and torch.equal(got.h, want.h)
        assert torch.equal(got.q, want.q)


@pytest.mark.parametrize("M", [70, 300, 800, 2100, 4101])
@pytest.mark.parametrize("opB,pow2", [(0, False), (1, True)])
def test_tile_sizes(M, opB, pow2):
    """Rows for every tile height, fused and in parts that are joined."""
    K, H = 384, 1024
    x, sx = fb.quantize_1x128(_bf16((M, K), 1), pow2=pow2)
    w, sw = _weights(*((2 * H, K) if opB else (K, 2 * H)), 2, pow2)
    C = fb.gemm_fp8_blockscaled(x, sx, w, sw, opB=opB, split_k=False, pow2_scales=pow2)
    kw = dict(opB=opB, pow2_scales=pow2, quantize=True, pow2=pow2)
    fused = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, split_k=False, **kw)
    r = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, **kw)
    assert torch.equal(fused.u, C.to(BF))
    e = _split_error(x, sx, w, sw, opB, M, 2 * H)
    assert np.all(np.abs(_np(r.u) - _np(C)) <= _half(_np(C), e))
    for o in (fused, r):
        _check_h(o.h, _np(C), H, "silu", e)
        q, s = fb.quantize_1x128(o.h, pow2=pow2)
        assert torch.equal(o.q, q) and torch.equal(o.s, s)
    d, sd = _weights(*((2 * H, K) if opB else (K, 2 * H)), 3, pow2)
    dh = fb.gemm_fp8_blockscaled(x, sx, d, sd, opB=opB, split_k=False, pow2_scales=pow2)
    u = _bf16((M, 4 * H), 4)
    e = _split_error(x, sx, d, sd, opB, M, 2 * H)
    for split in (False, True):
        g = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, u, split_k=split, **kw)
        _check_grad(g, _np(dh), u, "silu", e if split else 0.0)
        q, s = fb.quantize_1x128(g.du, pow2=pow2)
        assert torch.equal(g.q, q) and torch.equal(g.s, s)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _counts(G, seed, most):
    rng = np.random.RandomState(seed)
    c = rng.randint(0, most, G) * (rng.rand(G) < 0.7)
    c[G // 2] = 300 if most > 20 else 70
    c[0] += most > 200  # odd row counts throughout
    return c


@pytest.mark.parametrize("G,most", [(1, 60), (7, 60), (70, 60), (300, 60), (12, 14), (70, 14), (300, 6), (6, 400), (5, 1200)])
@pytest.mark.parametrize("act,t,pow2", [("silu", False, False), ("gelu", True, True), ("silu", True, False)])
def test_experts(G, most, act, t, pow2):
    """Every expert's rows as the grouped GEMM makes them, many rows each and few; rows no expert owns stay as they were."""
    print(f"[train] experts {G} {most} {act} {t} {pow2}", flush=True)
    K, H, past = 256 if most > 20 else 768, 128 if G == 300 else 256, 19
    counts = _counts(G, G, most)
    P, off = int(counts.sum()), _offsets(counts)
    M = P + past
    x, sx = fb.quantize_1x128(_bf16((M, K), 1), pow2=pow2)
    w, sw = _weights(*((2 * H, K) if t else (K, 2 * H)), 2, pow2, G)
    opB = int(t)
    C = fb.grouped_gemm_fp8_blockscaled(off, x, sx, w, sw, opB=opB, pow2_scales=pow2)[:P]
    lent = dict(u=torch.full((M, 2 * H), 7.0, dtype=BF, device="cuda"), h=torch.full((M, H), 7.0, dtype=BF, device="cuda"),
                q=torch.full((M, H), 77, dtype=torch.uint8, device="cuda"), s=torch.full((H // 128, M), 7.0, device="cuda"))
    for bound in (None, 0, int(counts.max())):
        r = fb.grouped_gated_gemm_fp8_blockscaled(off, x, sx, w, sw, act=act, opB=opB, pow2_scales=pow2, quantize=True,
                                                  pow2=pow2, max_group_rows=bound, **lent)
        assert torch.equal(r.u[:P], C.to(BF))
        _check_h(r.h[:P], _np(C), H, act)
        q, s = fb.quantize_1x128(r.h[:P], pow2=pow2)
        assert torch.equal(r.q[:P], q) and torch.equal(r.s[:, :P], s)
        assert (r.u[P:] == 7).all() and (r.h[P:] == 7).all() and (r.q[P:] == 77).all() and (r.s[:, P:] == 7).all()
    # gradient of the same block: K is the down projection's width now
    d, sd = _weights(*((H, K) if t else (K, H)), 5, pow2, G)
    dh = fb.grouped_gemm_fp8_blockscaled(off, x, sx, d, sd, opB=opB, pow2_scales=pow2)[:P]
    g = fb.grouped_gated_gemm_backward_fp8_blockscaled(off, x, sx, d, sd, lent["u"], act=act, opB=opB, pow2_scales=pow2,
                                                       quantize=True, pow2=pow2,
                                                       du=torch.full((M, 2 * H), 7.0, dtype=BF, device="cuda"))
    _check_grad(fb.GatedGemmGrad(g.du[:P], g.h[:P], None, None), _np(dh), lent["u"][:P], act)
    q, s = fb.quantize_1x128(g.du[:P], pow2=pow2)
    assert torch.equal(g.q[:P], q) and torch.equal(g.s[:, :P], s) and (g.du[P:] == 7).all()
    assert torch.equal(g.h[:P], fb.gated_gemm_backward_fp8_blockscaled(x, sx, d[0], sd[0], lent["u"], act=act, opB=opB,
                                                                       pow2_scales=pow2).h[:P])


@pytest.mark.parametrize("t,pow2", [(False, False), (True, True), (True, False)])
def test_experts_past_the_caches(t, pow2):
    """Few rows for each of many experts, whose weights are more than the caches hold: the grouped GEMM's bits."""
    print(f"[train] experts past the caches {t} {pow2}", flush=True)
    G, K, H, past = 280, 1024, 1024, 3
    counts = np.random.RandomState(7).randint(0, 4, G)
    counts[3] = 70  # two tiles
    P, off, opB = int(counts.sum()), _offsets(counts), int(t)
    assert 257 < P <= 20 * G  # one MB of codes an expert in the gradient, two forward
    x, sx = fb.quantize_1x128(_bf16((P + past, K), 1), pow2=pow2)
    w, sw = _weights(*((2 * H, K) if t else (K, 2 * H)), 2, pow2, G)
    r = fb.grouped_gated_gemm_fp8_blockscaled(off, x, sx, w, sw, opB=opB, pow2_scales=pow2, quantize=True, pow2=pow2,
                                              u=torch.full((P + past, 2 * H), 7.0, dtype=BF, device="cuda"))
    C = fb.grouped_gemm_fp8_blockscaled(off, x, sx, w, sw, opB=opB, pow2_scales=pow2)[:P]
    assert torch.equal(r.u[:P], C.to(BF)) and (r.u[P:] == 7).all()
    _check_h(r.h[:P], _np(C), H, "silu")
    q, s = fb.quantize_1x128(r.h[:P].contiguous(), pow2=pow2)
    assert torch.equal(r.q[:P], q) and torch.equal(r.s[:, :P], s)
    d, sd = _weights(*((H, K) if t else (K, H)), 5, pow2, G)
    dh = fb.grouped_gemm_fp8_blockscaled(off, x, sx, d, sd, opB=opB, pow2_scales=pow2)[:P]
    g = fb.grouped_gated_gemm_backward_fp8_blockscaled(off, x, sx, d, sd, r.u, opB=opB, pow2_scales=pow2, quantize=True,
                                                       pow2=pow2)
    _check_grad(fb.GatedGemmGrad(g.du[:P], g.h[:P], None, None), _np(dh), r.u[:P], "silu")
    q, s = fb.quantize_1x128(g.du[:P].contiguous(), pow2=pow2)
    assert torch.equal(g.q[:P], q) and torch.equal(g.s[:, :P], s)


def test_no_rows():
    w, sw = _weights(256, 512, 1, False)
    x, sx = fb.quantize_1x128(_bf16((0, 256), 1))
    r = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, quantize=True)
    assert r.u.shape == (0, 512) and r.h.shape == (0, 256) and r.q.shape == (0, 256) and r.s.shape == (2, 0)
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    w3, s3 = _weights(256, 512, 1, False, 3)
    assert fb.grouped_gated_gemm_fp8_blockscaled(off, x, sx, w3, s3).h.shape == (0, 256)
    y, sy = fb.quantize_1x128(_bf16((5, 256), 1))
    h = torch.full((5, 256), 3.0, dtype=BF, device="cuda")
    fb.grouped_gated_gemm_fp8_blockscaled(off, y, sy, w3, s3, h=h, want_u=False)
    assert (h == 3).all()
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    fb.grouped_gated_gemm_fp8_blockscaled(none, y, sy, w3[:0], s3[:0], h=h, want_u=False)
    assert (h == 3).all()


@pytest.mark.parametrize("split", [False, True])
def test_pitches(split):
    """Operands and outputs whose rows lie apart; what lies between is left alone."""
    M, K, H = 300, 256, 384
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    w, sw = _weights(K, 2 * H, 2, False)
    ref_ = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, quantize=True, split_k=split)
    xp = torch.zeros(M, K + 48, dtype=torch.uint8, device="cuda")[:, :K]
    xp.copy_(x)
    wp = torch.zeros(K, 2 * H + 16, dtype=torch.uint8, device="cuda")[:, :2 * H]
    wp.copy_(w)
    u, h = (torch.full((M, n + 8), 7.0, dtype=BF, device="cuda") for n in (2 * H, H))
    q = torch.full((M, H + 16), 77, dtype=torch.uint8, device="cuda")
    r = fb.gated_gemm_fp8_blockscaled(xp, sx, wp, sw, quantize=True, split_k=split, u=u[:, :2 * H], h=h[:, :H], q=q[:, :H])
    for name, t in (("u", u), ("h", h), ("q", q)):
        want = getattr(ref_, name)
        assert torch.equal(t[:, :want.shape[1]], want) and (t[:, want.shape[1]:] == (77 if name == "q" else 7)).all()
    assert torch.equal(r.s, ref_.s)
    d, sd = _weights(H, K, 3, False)
    want = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, ref_.u, split_k=split, quantize=True)
    du = torch.full((M, 2 * H + 24), 7.0, dtype=BF, device="cuda")
    got = fb.gated_gemm_backward_fp8_blockscaled(xp, sx, d, sd, u[:, :2 * H], split_k=split, quantize=True,
                                                 du=du[:, :2 * H], h=h[:, :H], q=torch.empty(M, 2 * H + 32, dtype=torch.uint8,
                                                                                            device="cuda")[:, :2 * H])
    assert torch.equal(du[:, :2 * H], want.du) and (du[:, 2 * H:] == 7).all() and torch.equal(got.q, want.q)
    assert torch.equal(got.h, want.h) and torch.equal(got.s, want.s)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_values(act):
    """Gate values over FP32's exponents: no NaN where the formula has none."""
    M, K, H = 64, 128, 128
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    d, sd = _weights(H, K, 2, False)
    u = _bf16((M, 2 * H), 3)
    u[:, :H] *= torch.logspace(-30, 30, H, device="cuda").to(BF)
    for split in (False, True):
        r = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, u, act=act, split_k=split)
        assert torch.isfinite(r.du).all() and torch.isfinite(r.h).all()
    dh = fb.gemm_fp8_blockscaled(x, sx, d, sd, opB=1, split_k=False)
    near = _np(u[:, :H]).__abs__().max(0) < 1e4  # z^3 stays where the bounds are stated
    r = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, u, act=act, split_k=False)
    both = np.concatenate([near, near])
    keep = torch.from_numpy(both).cuda()
    _check_grad(fb.GatedGemmGrad(r.du[:, keep], r.h[:, keep[:H]], None, None), _np(dh)[:, near], u[:, keep], act)


def test_large():
    """More than 2^32 bytes of u, and the last rows as a product of their own."""
    M, K, H = 1_100_009, 128, 1024
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    w, sw = _weights(K, 2 * H, 2, False)
    r = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, quantize=True)
    n = 777
    tail = fb.gated_gemm_fp8_blockscaled(x[-n:].contiguous(), sx[:, -n:].contiguous(), w, sw, quantize=True, split_k=False)
    assert all(torch.equal(a[-n:], b) for a, b in zip(r[:3], tail[:3])) and torch.equal(r.s[:, -n:], tail.s)
    d, sd = _weights(H, K, 3, False)
    kw = dict(quantize=True, want_h=False)
    g = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, r.u, du=r.u, **kw)
    t = fb.gated_gemm_backward_fp8_blockscaled(x[-n:].contiguous(), sx[:, -n:].contiguous(), d, sd, tail.u, split_k=False, **kw)
    assert torch.equal(g.du[-n:], t.du) and torch.equal(g.q[-n:], t.q) and torch.equal(g.s[:, -n:], t.s)


def test_streams_and_graphs():
    """Two calls on two streams at once, and captured ones: the same bits as one after the other."""
    M, K, H = 40, 2048, 512
    ops = []
    for seed in (1, 50):
        x, sx = fb.quantize_1x128(_bf16((M, K), seed))
        w, sw = _weights(K, 2 * H, seed + 1, False)
        d, sd = _weights(H, K, seed + 2, False)
        ops.append((x, sx, w, sw, d, sd))

    def run(o):
        x, sx, w, sw, d, sd = o
        r = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, quantize=True)
        g = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, r.u, quantize=True)
        return [*r, *g]

    want = [[t.clone() for t in run(o)] for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(3):
        got = []
        for s, o in zip(streams, ops):
            with torch.cuda.stream(s):
                got.append(run(o))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    graphs, outs = [], []
    for o in ops:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(o))
    torch.cuda.synchronize()
    for rep in range(4):
        if rep == 2:  # new inputs in place
            for o in ops:
                o[0].copy_(o[0].roll(1, 0))
                o[1].copy_(o[1].roll(1, 1))
            want = [[t.clone() for t in run(o)] for o in ops]
            torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(outs, want) for a, b in zip(g, w)), rep
        run(ops[0])
        torch.cuda.synchronize()


def test_refuses():
    x, sx = fb.quantize_1x128(_bf16((8, 256), 1))
    w, sw = _weights(256, 512, 2, False)
    u = _bf16((8, 1024), 3)
    f, b = fb.gated_gemm_fp8_blockscaled, fb.gated_gemm_backward_fp8_blockscaled
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: f(x, sx, w, sw, act="relu"), lambda: f(x, sx, w, sw, opB=2), lambda: f(x, sx, w[:128], sw[:1]),
                 lambda: f(x, sx, w[:, :384], sw[:, :3]), lambda: f(x, sx[:1], w, sw), lambda: f(x, sx, w, sw[:1]),
                 lambda: f(x, sx, w, sw, q=torch.empty(8, 256, dtype=torch.uint8, device="cuda")),
                 lambda: f(x, sx, w, sw, h=_bf16((8, 128), 1)), lambda: f(x, sx, w, sw, u=u.t()), lambda: f(x.cpu(), sx, w, sw),
                 lambda: f(x, sx.cpu(), w, sw), lambda: f(x, sx, w.view(1, 256, 512), sw.view(1, 2, 4)),
                 lambda: b(x, sx, w, sw, u), lambda: b(x, sx, w, sw, u[:, :512], opB=0),
                 lambda: b(x, sx, w, sw, u[:7], opB=0),
                 lambda: fb.grouped_gated_gemm_fp8_blockscaled(off, x, sx, w, sw),
                 lambda: fb.grouped_gated_gemm_fp8_blockscaled(off[:1], x, sx, w.view(1, 256, 512), sw.view(1, 2, 4))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(None, sx, w, sw), lambda: f(x, sx, w.view(torch.int8), sw), lambda: f(x, sx.half(), w, sw),
                 lambda: f(x, sx, w, sw, h=torch.empty(8, 256, device="cuda")), lambda: b(x, sx, w, sw, None, opB=0),
                 lambda: b(x, sx, w, sw, u.float(), opB=0), lambda: fb.grouped_gated_gemm_fp8_blockscaled(None, x, sx, w, sw),
                 lambda: fb.grouped_gated_gemm_fp8_blockscaled(off.long(), x, sx, w.view(1, 256, 512), sw.view(1, 2, 4))):
        with pytest.raises(TypeError):
            call()
    shifted = torch.empty(8 * 512 + 8, dtype=BF, device="cuda")[1:8 * 512 + 1].view(8, 512)
    for call in (lambda: f(x, sx, w, sw, u=shifted), lambda: b(x, sx, w[:, :256].contiguous(), sw[:, :2].contiguous(), shifted)):
        with pytest.raises(fb.Fp8BlkError):
            call()


def test_refuses_outputs_in_u():
    """du is u element for element or shares nothing with it; h and q share nothing with it."""
    x, sx = fb.quantize_1x128(_bf16((8, 256), 1))
    d, sd = _weights(256, 256, 2, False)
    room = _bf16((17, 512), 3)
    u = room[:8]
    b = fb.gated_gemm_backward_fp8_blockscaled
    want = b(x, sx, d, sd, u, opB=0)
    for what, call in (("du", lambda: b(x, sx, d, sd, u, opB=0, du=room[1:9])),
                       ("du", lambda: b(x, sx, d, sd, u, opB=0, du=room[:16:2])),
                       ("h", lambda: b(x, sx, d, sd, u, opB=0, h=u[:, 256:])),
                       ("q", lambda: b(x, sx, d, sd, u, opB=0, quantize=True, q=u.view(torch.uint8)[:, :512]))):
        with pytest.raises(ValueError, match=f"^{what} shares memory with u"):
            call()
    w, sw = _weights(256, 512, 4, False)
    with pytest.raises(ValueError, match="^h shares memory with u"):
        fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, u=u, h=u[:, :256])
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="^du shares memory with u"):
        fb.grouped_gated_gemm_backward_fp8_blockscaled(off, x, sx, d[None], sd[None], u, opB=0, du=room[1:9])
    spaced = room[1:17].view(8, 1024)[:, 512:]  # rows between u's, from a u whose rows lie apart
    between = room[1:17].view(8, 1024)[:, :512]
    between.copy_(u.clone())
    kept = between.clone()
    got = b(x, sx, d, sd, between, opB=0, du=spaced)
    ref_ = b(x, sx, d, sd, kept, opB=0)
    assert torch.equal(got.du, ref_.du) and torch.equal(got.h, ref_.h) and torch.equal(between, kept)
    same = kept.clone()
    assert torch.equal(b(x, sx, d, sd, same, opB=0, du=same).du, ref_.du) and torch.equal(same, ref_.du)
    assert want.du.shape == (8, 512)
