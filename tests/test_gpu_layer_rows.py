"""GPU tests of the norms around a block where every workgroup takes several
rows: the next row asked for while one is worked on, sums over a workgroup's
rows, rows that end inside a chunk.  Workgroups of rows above 512 channels are
at most (lanes a compute unit holds / lanes of a row) times the compute units,
256 on an MI355X; each case has more than two rows for each of them.

Bounds and plain forms are those of test_gpu_layer_norm.py.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import test_gpu_layer_norm as norm
from tests.layer_ref import U

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# Forward: 16, 10, 4, 3, 2 and 3 workgroups a compute unit.
@pytest.mark.parametrize("M,C,post,gate,res", [
    (8500, 519, "norm", "channel", BF), (8500, 519, "none", "none", F32), (5300, 1025, "norm", "row", BF),
    (5300, 1025, "add", "channel", F32), (1700, 3584, "norm", "channel", F32), (1700, 5001, "norm", "channel", BF),
    (1700, 5001, "norm", "row", F32), (1100, 7168, "norm", "row", BF), (1700, 9001, "norm", "channel", F32),
    (1700, 9001, "norm", "row", BF)])
def test_forward(M, C, post, gate, res):
    norm.test_forward(M, C, post, True, gate, res, F32 if res == BF else BF)


@pytest.mark.parametrize("M,C", [(5300, 1025), (1700, 5001), (1700, 9001)])
def test_forward_in_place(M, C):
    print(f"[layer] norm in place M={M} C={C}", flush=True)
    d = norm._inputs(M, C, "norm", True, "channel", BF, F32, pad=1)
    want = fb.residual_norm(alpha=norm.ALPHA, quantize=True, **d)
    got = fb.residual_norm(alpha=norm.ALPHA, quantize=True, x_out=d["x"], **d)
    assert got.x is d["x"] and all(torch.equal(a, b) for a, b in zip(got, want))


# Gradient with the block's output: 4, 2, 1 workgroups a compute unit; without
# one: 8, 8, 5, 1.  The last two sizes with a gate per token and FP32 rows, and
# above 8192 channels, read their rows twice.
@pytest.mark.parametrize("M,C,post,gate,res", [
    (2600, 519, "norm", "channel", BF), (2600, 519, "norm", "row", F32), (2600, 520, "add", "channel", BF),
    (1200, 1025, "norm", "channel", F32), (1200, 1025, "add", "row", BF), (600, 5001, "norm", "channel", BF),
    (600, 7168, "norm", "channel", F32), (600, 5001, "norm", "row", F32), (600, 9001, "norm", "channel", BF),
    (600, 9001, "norm", "row", F32),
    (4300, 519, "none", "none", BF), (4300, 1024, "none", "none", F32), (2700, 1025, "none", "none", BF),
    (600, 5001, "none", "none", F32), (600, 7168, "none", "none", BF), (600, 9001, "none", "none", BF)])
def test_backward(M, C, post, gate, res):
    for pre in ((True,) if post == "none" else (True, False)):
        norm.test_backward(M, C, post, pre, gate, res, F32 if res == BF else BF)


@pytest.mark.parametrize("M,C", [(2600, 519), (1200, 1025), (600, 5001), (600, 9001)])
def test_backward_in_place(M, C):
    print(f"[layer] norm grad in place M={M} C={C}", flush=True)
    norm.test_backward_in_place(M, C)


@pytest.mark.parametrize("M,C", [(6000, 7168), (8192, 2051), (3200, 16384), (1 << 17, 136)])
@pytest.mark.parametrize("post", ["norm", "none"])
def test_sums_over_many_rows(M, C, post):
    """All three sums over tokens, gate per channel, against 64-bit sums."""
    print(f"[layer] norm grad sums M={M} C={C} {post}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M)

    def rnd(*s, dtype=BF):
        t = torch.randn(*s, generator=g, device="cuda").to(dtype)
        return fb.as_pitched(t) if len(s) == 2 else t

    x, dx, dn = rnd(M, C), rnd(M, C), rnd(M, C)
    w1 = 1 + 0.1 * rnd(C, dtype=F32)
    f, w2, gate = (rnd(M, C), 1 + 0.1 * rnd(C, dtype=F32), rnd(C, dtype=F32)) if post == "norm" else (None,) * 3
    r1 = torch.rsqrt(x.float().square().mean(1) + 1e-6)
    r2 = torch.rsqrt(f.float().square().mean(1) + 1e-6) if post == "norm" else None
    got = fb.residual_norm_backward(x, dx_out=dx, dn=dn, rstd_pre=r1, w_pre=w1, f=f, rstd_post=r2, w_post=w2, gate=gate,
                                    alpha=0.5)
    # a part of the rows at a time: sums of the terms and of the bounds on their errors
    want, bound = {}, {}

    def add(name, terms, err):
        want[name] = want.get(name, 0) + terms.sum(0)
        # (M + 4) U for the sum, as in test_gpu_layer_norm.py, and each term's own error
        bound[name] = bound.get(name, 0) + (2 * (M + 4) * U * err[0] + err[1]).sum(0)

    rel = 2 * (C + 12) * U  # of a row's terms (test_gpu_layer_norm.py)
    for i in range(0, M, 2048):
        cut = slice(i, i + 2048)
        h = x[cut].double() * r1[cut].double()[:, None]
        v = dn[cut].double() * w1.double()
        t = dn[cut].double() * h
        add("dw_pre", t, (t.abs(), 0 * t))
        if post == "none":
            continue
        r = r1[cut].double()[:, None]
        gx = dx[cut].double() + r * (v - h * (v * h).mean(1, keepdim=True))
        mag = dx[cut].double().abs() + r * (v.abs() + h.abs() * (v * h).abs().mean(1, keepdim=True))
        hf = f[cut].double() * r2[cut].double()[:, None]
        for name, factor in (("dw_post", gate), ("dgate", w2)):
            k = 0.5 * factor.double() * hf
            add(name, gx * k, (mag * k.abs(), 2 * rel * mag * k.abs()))
    for name in want:
        assert bool(((getattr(got, name).double() - want[name]).abs() <= bound[name]).all()), name
    assert np.isfinite(float(got.dw_pre.sum()))
