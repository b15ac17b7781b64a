"""GPU tests of the gated products and the optimizer step at values and places
that the tests of their forms do not reach: infinities and NaN through the
forward product, the gradient's h beside the forward's, tiles without a split's
allowance, elements past 2^32, steps from values in device memory.
"""
import math

import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import train_ref as ref
from tests.layer_ref import UB
from tests.test_gpu_train_gated import _bf16, _check_h, _half, _np, _weights

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _same(a, b):
    """Equal, NaN where the other has one."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,split", [(300, False), (600, False), (40, True), (40, False)])
@pytest.mark.parametrize("opB", [0, 1])
def test_forward_of_what_is_not_finite(act, M, split, opB):
    """NaN codes and infinite scales stay in their rows, and become what the formula makes of them."""
    K, H = 1024, 256
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    w, sw = _weights(*((2 * H, K) if opB else (K, 2 * H)), 2, False)
    clean = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, act=act, opB=opB, quantize=True, split_k=split)
    x[3, 200], x[17, 900] = 0x7F, 0xFF
    sx[2, 5], sx[7, 20], sx[0, 33] = math.inf, math.nan, 2.0 ** 126
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[3, 17, 5, 20, 33]] = True
    r = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, act=act, opB=opB, quantize=True, split_k=split)
    for a, b in ((r.u, clean.u), (r.h, clean.h), (r.q, clean.q), (r.s.t(), clean.s.t())):
        assert torch.equal(a[~bad], b[~bad])
    C = fb.gemm_fp8_blockscaled(x, sx, w, sw, opB=opB, split_k=False)
    assert _same(r.u[bad], C[bad].to(BF))
    assert r.u[[3, 17, 20]].isnan().all() and r.u[5].isinf().any()
    g, v = C[bad][:, :H].double(), C[bad][:, H:].double()
    z = g if act == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    # p is 0 in FP32 where e^-z passes its range: g p, -0 then, is -inf 0 for g = -inf only
    p = torch.where(z < -89, torch.zeros_like(z), torch.sigmoid(z))
    want = (g * p * v).float().to(BF)
    far = torch.isfinite(want) & (want.abs() > 1e-30)
    got = r.h[bad]
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    assert torch.allclose(got[far].double(), (g * p * v)[far], rtol=2.0 ** -7, atol=0.0)
    q, s = fb.quantize_1x128(r.h)
    assert torch.equal(r.q, q) and torch.equal(r.s.view(torch.int32), s.view(torch.int32))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [16, 300, 2100])
def test_h_of_both_directions(act, M):
    """The forward forms h from FP32 products, the gradient from u as kept in BF16: apart by u's rounding."""
    K, H = 512, 512
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    w, sw = _weights(K, 2 * H, 2, False)
    d, sd = _weights(H, K, 3, False)
    f = fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, act=act, split_k=False)
    C = _np(fb.gemm_fp8_blockscaled(x, sx, w, sw, split_k=False))
    g = fb.gated_gemm_backward_fp8_blockscaled(x, sx, d, sd, f.u, act=act)
    _check_h(f.h, C, H, act)
    _check_h(g.h, C, H, act, np.abs(C) * UB + 2.0 ** -134)
    want, e = ref.gated(_np(f.u[:, :H]), _np(f.u[:, H:]), act)
    assert np.all(np.abs(_np(g.h) - want) <= _half(want, e))


@pytest.mark.parametrize("M", [70, 300, 800, 2100, 4101])
@pytest.mark.parametrize("opB,pow2", [(0, False), (1, True)])
def test_tiles_without_a_split(M, opB, pow2):
    """h of every tile height from the GEMM's own FP32 products, which the fused form accumulates in the same order."""
    K, H = 384, 1024
    x, sx = fb.quantize_1x128(_bf16((M, K), 1), pow2=pow2)
    w, sw = _weights(*((2 * H, K) if opB else (K, 2 * H)), 2, pow2)
    C = _np(fb.gemm_fp8_blockscaled(x, sx, w, sw, opB=opB, split_k=False, pow2_scales=pow2))
    _check_h(fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, opB=opB, pow2_scales=pow2, split_k=False).h, C, H, "silu")


def test_elements_past_32_bits():
    """Rounding at random, codes and parameters on either side of element 2^32, bit by bit (their places' high half counts)."""
    n, tail = 2 ** 32 + 128 * 20 + 57, 128 * 40 + 57
    lo = n - tail
    rng = np.random.RandomState(1)
    g = np.clip(rng.randn(tail) * np.exp2(rng.randint(-14, 4, tail)), -400, 400).astype(np.float32)
    g = torch.from_numpy(g).to(BF)
    g[g == 0] = 1.0
    g[::128] = 448.0  # scales of one: the quotients are exact
    grad = torch.full((n,), 448.0, dtype=BF, device="cuda")
    grad[lo:] = g.cuda()
    s = fb.AdamWState([torch.zeros(n, dtype=BF, device="cuda")], dtype=E4)
    fb.adamw_step(fb.adamw_table(s, [grad]), 0.3, 1, beta1=0.0, beta2=0.0, eps=0.0, seed=99)
    gn, at, key = g.float().numpy(), np.arange(lo, n), ref.key_of(99)
    r, rp = ref.random_bits(key, at), ref.random_bits(key ^ 0x5BD1E995, at)
    assert (r != ref.random_bits(key, at & 0xFFFFFFFF)).any()

    def codes(x, r16, floor):
        a = np.abs(x)
        up = np.where(a < 2.0 ** -6, np.float32(2.0 ** -6), np.float32(0))
        a = ref.drop(a + up, 20, r16 << 4) - up
        if floor:
            a = np.where((x > 0) & (a == 0), np.float32(2.0 ** -9), a)
        return np.copysign(a, x).astype(np.float64)

    def tail_of(t):
        return t[-tail:].cpu().numpy()

    assert (s.m_scales[0] == 1.0).all() and (s.v_scales[0] == 1.0).all()
    assert np.array_equal(ref.decode(tail_of(s.ms[0])), codes(gn, r & 0xFFFF, False))
    assert np.array_equal(ref.decode(tail_of(s.vs[0])), codes(np.abs(gn), r >> 16, True))  # the root of an exact square
    want = ref.drop(-np.sign(gn) * np.float32(0.3), 16, rp & 0xFFFF)
    assert np.array_equal(s.params[0][-tail:].float().cpu().numpy(), want)
    first = ref.drop(np.full(4096, -0.3, np.float32), 16, ref.random_bits(key ^ 0x5BD1E995, np.arange(4096)) & 0xFFFF)
    assert np.array_equal(s.params[0][:4096].float().cpu().numpy(), first)


@pytest.mark.parametrize("kind", [F32, BF, E4])
def test_captured_step_equals_device_values(kind):
    """A replayed step and an eager one that take the same values from device memory: the same bits at every replay."""
    sizes = [5000, 77, 40000]

    def fresh():
        s = fb.AdamWState([_bf16(n, i) for i, n in enumerate(sizes)], dtype=kind, decay=0.1)
        grads = [_bf16(n, 40 + i, 1e-2) for i, n in enumerate(sizes)]
        return s, fb.adamw_table(s, grads), grads

    def all_of(s):
        return [t for ts in (s.params, s.ms, s.vs, s.m_scales, s.v_scales) for t in ts if t is not None]

    a, ta, ga = fresh()
    b, tb, gb = fresh()
    lr = torch.zeros((), device="cuda")
    step, seed = (torch.zeros((), dtype=torch.int64, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.adamw_step(ta, lr, step, seed=seed)
    for k in range(1, 6):
        lr.fill_(1e-2 / k)
        step.fill_(k)
        seed.fill_(17 * k)
        for x, y in zip(ga, gb):
            x.mul_(0.9)
            y.mul_(0.9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        fb.adamw_step(tb, lr, step, seed=seed)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(all_of(a), all_of(b))), k
