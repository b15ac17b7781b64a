"""GPU tests of how the gated products and the optimizer step treat their
callers' tensors: writes that autograd has to see, lent workspaces, tables whose
tensors have other memory by now.
"""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
M, K, H = 16, 2048, 512


def _bf16(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def _forward():
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    w, sw = fb.quantize_block128(_bf16((K, 2 * H), 2, 0.05))
    return lambda **kw: fb.gated_gemm_fp8_blockscaled(x, sx, w, sw, quantize=True, **kw)


def _backward():
    x, sx = fb.quantize_1x128(_bf16((M, K), 1))
    w, sw = fb.quantize_block128(_bf16((H, K), 2, 0.05))
    own = _bf16((M, 2 * H), 3)
    return lambda u=own, **kw: fb.gated_gemm_backward_fp8_blockscaled(x, sx, w, sw, u, quantize=True, **kw)


# --- what autograd has to know ---------------------------------------------------

def _square(t):
    """A graph that needs t as it is."""
    return (t * t).sum()


def _spoiled(out):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()


@pytest.mark.parametrize("dtype", [torch.float32, BF, E4])
def test_step_counts_as_a_write(dtype):
    p = [torch.nn.Parameter(_bf16(300, i).float()) for i in range(2)]
    g, c = [_bf16(300, 5).float(), _bf16(300, 6)], [torch.zeros(300, dtype=BF, device="cuda").requires_grad_() for _ in p]
    s = fb.AdamWState(p, dtype=dtype, copies=c)
    t = fb.adamw_table(s, g)
    needs = [_square(x) for x in (*p, *c)]
    written = [x for ts in (p, c, s.ms, s.vs, s.m_scales, s.v_scales) for x in ts if x is not None]
    before = [x._version for x in written], [x._version for x in g]
    fb.adamw_step(t, 1e-3, 1)
    assert all(x._version > v for x, v in zip(written, before[0]))
    assert [x._version for x in g] == before[1]
    for out in needs:
        _spoiled(out)
    fresh = _square(p[0])
    with pytest.raises(fb.Fp8BlkError):
        fb.adamw_step(t, float("nan"), 2)  # refused: nothing was written
    fresh.backward()
    assert torch.equal(p[0].grad, 2 * p[0].detach())


def test_lent_outputs_count_as_written():
    f, b = _forward(), _backward()
    u, h = (torch.zeros(M, n, dtype=BF, device="cuda", requires_grad=True) for n in (2 * H, H))
    needs = [_square(u), _square(h)]
    f(u=u, h=h)
    for out in needs:
        _spoiled(out)
    u = _bf16((M, 2 * H), 3).requires_grad_()
    out = _square(u)
    r = b(u)  # read only
    out.backward(retain_graph=True)
    assert b(u, du=u).du.data_ptr() == u.data_ptr() and torch.equal(u.detach(), r.du)
    _spoiled(out)


def test_inference_tensors():
    """They have no versions: written as before, inside inference mode and outside."""
    with torch.inference_mode():
        p, g = torch.zeros(300, device="cuda"), torch.ones(300, device="cuda")
        u = _bf16((M, 2 * H), 3)
        t = fb.adamw_table(fb.AdamWState([p]), [g])
        fb.adamw_step(t, 0.5, 1, eps=0.0)
    fb.adamw_step(t, 0.5, 1, eps=0.0)
    assert (p < -0.5).all()
    b = _backward()
    want = b(u.clone()).du
    assert torch.equal(b(u, du=u).du, want)


# --- lent workspaces --------------------------------------------------------------

@pytest.mark.parametrize("call,query", [(_forward, "fp8blk_gated_gemm_workspace_bytes"),
                                        (_backward, "fp8blk_gated_gemm_backward_workspace_bytes")])
def test_workspaces(call, query):
    """One that is large enough serves as the binding's own; one that is too small or not aligned leaves the call to one launch."""
    f, need = call(), getattr(fb.lib(), query)(M, H, K)
    assert need > 0
    whole, split = f(split_k=False), f()
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))
    room = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    for w, want in ((room[:need], split), (room, split), (room[16:], split), (room[:need].view(torch.int32), split),
                    (room[:need - 1], whole), (room[:0], whole), (room[8:need + 8], whole)):
        room.fill_(0xFF)  # NaN: what is not written is not read
        assert same(f(workspace=w), want), (w.numel(), w.data_ptr() % 16)
        end = w.data_ptr() - room.data_ptr() + need
        assert (room[end:] == 0xFF).all() and (want is split or (room == 0xFF).all())
    room.fill_(0xFF)
    assert same(f(workspace=room, split_k=False), whole) and (room == 0xFF).all()
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        f(workspace=room[::2])
    with pytest.raises(ValueError, match="different devices"):
        f(workspace=torch.empty(need, dtype=torch.uint8))


# --- tables and their tensors' memory -------------------------------------------

def test_table_of_moved_memory():
    p, g = torch.nn.Parameter(torch.zeros(300, device="cuda")), torch.ones(300, device="cuda")
    s = fb.AdamWState([p])
    t = fb.adamw_table(s, [g])
    fb.adamw_step(t, 0.5, 1, eps=0.0)
    old = p.data
    p.data = torch.zeros(300, device="cuda")
    with pytest.raises(ValueError, match="^parameter 0 has other memory"):
        fb.adamw_step(t, 0.5, 2, eps=0.0)
    assert not p.any() and (old == -0.5).all()
    t = fb.adamw_table(s, [g])
    fb.adamw_step(t, 0.5, 2, eps=0.0)
    assert (p < -0.4).all()
    p.data = torch.zeros(301, device="cuda")  # refused on the host, by its moments
    with pytest.raises(ValueError, match="moments of parameter 0"):
        fb.adamw_table(s, [torch.ones(301, device="cuda")])
    s = fb.AdamWState([torch.zeros(300)])  # moments on the CPU, the parameter moved since
    s.params[0] = torch.zeros(300, device="cuda")
    with pytest.raises(ValueError, match="moments of parameter 0"):
        fb.adamw_table(s, [g])
    s = fb.AdamWState([torch.zeros(300, device="cuda")], dtype=E4)
    t = fb.adamw_table(s, [g])
    kept = s.ms[0]
    s.ms[0] = torch.zeros_like(kept)  # the table goes on with the tensors that it was built of
    fb.adamw_step(t, 0.5, 1)
    assert kept.any() and not s.ms[0].any()


def test_table_of_a_state_that_holds_other_moments_now():
    """A step goes by the moments that its table was built of."""
    p, g = torch.zeros(300, device="cuda"), torch.ones(300, device="cuda")
    s = fb.AdamWState([p])
    t = fb.adamw_table(s, [g])
    old = s.ms[0]
    s.__init__([p], dtype=E4)
    fb.adamw_step(t, 0.5, 1, eps=0.0)
    assert (p == -0.5).all() and old.all() and not s.ms[0].any()
