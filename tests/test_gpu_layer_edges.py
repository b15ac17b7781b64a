"""GPU tests of what the operators around the GEMMs do with inputs and outputs
out of the ordinary: infinities where a formula does not read them, lent
outputs and lists of gradients that share memory.
"""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests import test_gpu_layer_norm as norm
from tests.layer_ref import U

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


def _lent(shape, dtype):
    """A matrix to lend to a call, and a second tensor of the same values that
    shares its memory until one of the two is written."""
    t = torch.full(shape, 3, dtype=dtype, device="cuda")
    return torch._lazy_clone(t), t


def test_lent_outputs_that_share_memory_until_written():
    T, K, E, C = 24, 2, 4, 256
    ids = torch.randint(0, E, (T, K), generator=torch.Generator().manual_seed(1)).cuda()
    x, f, dx = (norm._matrix(T, C, torch.bfloat16, i) for i in (1, 2, 3))
    w, p = norm._vector(C, torch.float32, 4), torch.rand(T, K, device="cuda")
    bf, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    pairs = []

    def lend(shape, dtype):
        pairs.append(_lent(shape, dtype))
        return pairs[-1][0]

    maps = fb.moe_sort(ids, E, lend((E + 1,), i32), lend((T, K), i32), lend((T * K,), i32))
    want = [*fb.moe_sort(ids, E)]
    row_of, slot_of = want[1:]
    rows = fb.moe_dispatch(x, row_of)
    got = [*maps, fb.moe_dispatch(x, row_of, out=lend((T * K, C), bf))]
    want += [rows]
    q, s = fb.quantize_1x128(x)
    got += fb.moe_dispatch_fp8(q, s, row_of, slot_of, lend((T * K, C), u8), lend((C // 128, T * K), f32))
    want += fb.moe_dispatch_fp8(q, s, row_of, slot_of)
    got += [fb.moe_combine(rows, row_of, p, out=lend((T, C), bf))]
    want += [fb.moe_combine(rows, row_of, p)]
    got += fb.moe_combine_backward(dx, rows, row_of, p, drows=lend((T * K, C), bf), dweights=lend((T, K), f32))
    want += fb.moe_combine_backward(dx, rows, row_of, p)
    a = dict(w_pre=w, f=f, w_post=w, alpha=0.5)
    r = fb.residual_norm(x, quantize=True, **a)
    got += fb.residual_norm(x, quantize=True, x_out=lend((T, C), bf), n=lend((T, C), bf), q=lend((T, C), u8),
                            s=lend((C // 128, T), f32), **a)
    want += r
    a.update(dx_out=dx, dn=f, rstd_pre=r.rstd_pre, rstd_post=r.rstd_post)
    ws = lend((fb.lib().fp8blk_residual_norm_backward_workspace_bytes(T, C) // 4,), f32)
    got += fb.residual_norm_backward(r.x, dx=lend((T, C), bf), df=lend((T, C), bf), workspace=ws, **a)
    want += fb.residual_norm_backward(r.x, **a)
    outs = [lend((T, C), bf), lend((T, K), f32)]
    fb.clip_grad_norm(fb.grad_table([x, p], outs), 1.0)
    grads = [x.clone(), p.clone()]
    fb.clip_grad_norm(grads, 1.0)
    for i, (g, t) in enumerate(zip(got + outs, want + grads)):
        assert (g is None and t is None) or torch.equal(g, t), i
    for i, (_, other) in enumerate(pairs):
        assert (other == 3).all(), i


def test_in_place_on_memory_shared_until_written():
    x = norm._matrix(9, 200, torch.bfloat16, 1)
    f = norm._matrix(9, 200, torch.bfloat16, 2)
    want = fb.residual_norm(x, f=f, alpha=0.5).x
    keep = x.clone()
    mine = torch._lazy_clone(x)
    assert fb.residual_norm(mine, f=f, alpha=0.5, x_out=mine).x is mine
    assert torch.equal(mine, want) and torch.equal(x, keep)


def test_clipping_refuses_gradients_that_share_memory():
    """Which lists do is tested in test_layer_grad_lists.py."""
    g, o = torch.randn(5000, device="cuda"), torch.zeros(5000, device="cuda")
    before, n = g.clone(), float(g.double().square().sum())
    for table in ([g, g], fb.grad_table([g, o, g[100:]]), fb.grad_table([g, g], [o, o]), fb.grad_table([g[1:]], [g[:-1]])):
        with pytest.raises(ValueError, match="share memory"):
            fb.clip_grad_norm(table, 1.0)
        with pytest.raises(ValueError, match="share memory"):
            fb.grad_clip(table, torch.ones((), device="cuda"), 1.0)
    assert torch.equal(g, before) and not o.any()
    assert abs(float(fb.grad_norm([g, g])) - (2 * n) ** 0.5) <= 2 * U * (2 * n) ** 0.5  # read only: counted twice
    p = torch.zeros(5000, dtype=torch.bfloat16, device="cuda")
    fb.clip_grad_norm(fb.grad_table([g, g], [o, p]), 1e9)
    assert torch.equal(o, g) and torch.equal(p, g.to(torch.bfloat16))


def test_gradient_of_the_combine_of_many_narrow_tokens():
    """As many tokens as a launch of 64 lanes each takes, not one of 512."""
    T, C = 2 ** 23 + 3, 8
    print(f"[layer] combine grad T={T} C={C}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(T, 1, generator=g, device="cuda")
    row_of = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, 1)
    drows, dw = fb.moe_combine_backward(dy, rows, row_of, w)
    assert torch.equal(drows, (w * dy.float()).to(torch.bfloat16).flip(0))
    terms = dy.double() * rows.double().flip(0)
    assert bool(((dw.double() - terms.sum(1, keepdim=True)).abs() <= 2 * C * U * terms.abs().sum(1, keepdim=True)).all())


@pytest.mark.parametrize("E", [-1, 961, 2 ** 31, 2 ** 40, 2 ** 63 - 1])
def test_a_number_of_experts_out_of_range_takes_no_memory(E):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    with pytest.raises(fb.Fp8BlkError, match="moe_sort"):
        fb.moe_sort(ids, E)
    assert torch.cuda.max_memory_allocated() - held < 1 << 20
