"""GPU tests of what the operators around the GEMMs do with inputs and outputs
out of the ordinary: infinities where a formula does not read them.
"""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import test_gpu_layer_norm as norm

pytestmark = pytest.mark.gpu


# Without a norm after the block df = alpha gate g, whatever f holds.  Sizes of
# every form of the kernel: rows that share workgroups, rows held in registers
# (whole chunks, ragged, two chunks), rows that are read twice.
@pytest.mark.parametrize("M,C", [(5, 100), (6, 1032), (6, 2051), (4, 5001), (4, 7168), (3, 9001), (3, 16384)])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_infinities_of_an_unnormed_block_stay_out_of_its_gradient(M, C, gate, pre, res):
    print(f"[layer] unnormed block M={M} C={C} {gate} {pre} {res}", flush=True)
    xo, a = norm._grads(M, C, "add", pre, gate, res, torch.float32)
    clean = fb.residual_norm_backward(xo, alpha=0.5, **a)
    at = [(0, 0), (1, C // 2), (2, C - 1)]
    for (i, j), v in zip(at, ("inf", "-inf", "nan")):
        a["f"][i, j] = float(v)
    g = fb.residual_norm_backward(xo, alpha=0.5, **a)
    assert torch.isfinite(clean.df).all() and torch.equal(g.df, clean.df) and torch.equal(g.dx, clean.dx)
    assert not pre or torch.equal(g.dw_pre, clean.dw_pre)
    if gate == "none":
        return
    bad = torch.zeros_like(clean.dgate, dtype=torch.bool)  # dgate = alpha g f: there, and only there
    for i, j in at:
        bad[(i, j) if gate == "row" else j] = True
    assert torch.equal(~torch.isfinite(g.dgate), bad) and torch.equal(g.dgate[~bad], clean.dgate[~bad])
