"""GPU tests at sizes past the Infinity Cache (256 MB moved), where the
operators around the GEMMs stream past the caches: the outputs must be those
of the same call on a part of the tokens, bit for bit, which is small enough
to go through the caches.  Sums over tokens are formed in another order there
and are compared with 64-bit sums.
"""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests.layer_ref import U

pytestmark = pytest.mark.gpu

T, K, E, C = 2600, 8, 64, 7168   # 2600 * 9 * 7168 * 2 bytes = 335 MB
PART = slice(1300, 1364)


def _randn(shape, seed, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.fixture(scope="module")
def maps():
    g = torch.Generator(device="cuda").manual_seed(1)
    return fb.moe_sort(torch.randint(-1, E, (T, K), generator=g, device="cuda"), E)


def _part(row_of, rows):
    """The part's own maps: its rows gathered in pair order (dropped ones too)."""
    r = row_of[PART].long()
    at = torch.where(r < 0, -1 - r, r).reshape(-1)
    mine = torch.arange(at.numel(), dtype=torch.int32, device="cuda").view_as(row_of[PART])
    return at, torch.where(row_of[PART] < 0, -1 - mine, mine).contiguous(), None if rows is None else rows[at].contiguous()


def test_dispatch(maps):
    _, row_of, slot_of = maps
    x = _randn((T, C), 2)
    at, part_row, _ = _part(row_of, None)
    assert torch.equal(fb.moe_dispatch(x, row_of)[at], fb.moe_dispatch(x[PART], part_row))
    x2 = _randn((T, 2 * C), 3)  # 2600 * 9 * 14336 bytes of codes
    q, s = fb.quantize_1x128(x2)
    qr, sr = fb.moe_dispatch_fp8(q, s, row_of, slot_of)
    part_slot = torch.empty(at.numel(), dtype=torch.int32, device="cuda")
    n = torch.arange(at.numel(), dtype=torch.int32, device="cuda")
    part_slot[:] = torch.where(part_row.reshape(-1) < 0, -1 - n, n)
    pq, ps = fb.moe_dispatch_fp8(q[PART], s[:, PART].contiguous(), part_row, part_slot)
    assert torch.equal(qr[at], pq) and torch.equal(sr[:, at], ps)


@pytest.mark.parametrize("rows_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out_dt", [torch.bfloat16, torch.float32])
def test_combine(maps, rows_dt, out_dt):
    _, row_of, _ = maps
    rows, w = _randn((T * K, C), 4, rows_dt), _randn((T, K), 5, torch.float32)
    _, part_row, part_rows = _part(row_of, rows)
    for wt, pw in ((w, w[PART].contiguous()), (None, None)):
        big = fb.moe_combine(rows, row_of, wt, out_dtype=out_dt)
        assert torch.equal(big[PART], fb.moe_combine(part_rows, part_row, pw, out_dtype=out_dt))


@pytest.mark.parametrize("dy_dt,rows_dt,drows_dt", [(torch.bfloat16, torch.bfloat16, torch.bfloat16),
                                                    (torch.float32, torch.bfloat16, torch.float32),
                                                    (torch.bfloat16, torch.float32, torch.bfloat16)])
def test_combine_backward(maps, dy_dt, rows_dt, drows_dt):
    _, row_of, _ = maps
    rows, w, dy = _randn((T * K, C), 6, rows_dt), _randn((T, K), 7, torch.float32), _randn((T, C), 8, dy_dt)
    at, part_row, part_rows = _part(row_of, rows)
    dr, dw = fb.moe_combine_backward(dy, rows, row_of, w, drows_dtype=drows_dt)
    pr, pw = fb.moe_combine_backward(dy[PART], part_rows, part_row, w[PART].contiguous(), drows_dtype=drows_dt)
    assert torch.equal(dr[at], pr) and torch.equal(dw[PART], pw)


@pytest.mark.parametrize("res,gate_row", [(torch.bfloat16, False), (torch.float32, True)])
@pytest.mark.parametrize("M,C", [(6000, 7168), (12000, 4096), (3200, 16384)])
def test_norm_and_gradient(M, C, res, gate_row):
    print(f"[layer] large norm {M} x {C} {res}", flush=True)
    x, f = _randn((M, C), 9, res), _randn((M, C), 10)
    w1, w2 = 1 + 0.1 * _randn((C,), 11, torch.float32), 1 + 0.1 * _randn((C,), 12, torch.float32)
    gate = _randn((M, C), 13) if gate_row else _randn((C,), 13, torch.float32)
    cut = lambda t: t[PART] if t.dim() == 2 else t  # noqa: E731
    r = fb.residual_norm(x, w_pre=w1, f=f, w_post=w2, gate=gate, alpha=0.5, quantize=True)
    p = fb.residual_norm(x[PART], w_pre=w1, f=f[PART], w_post=w2, gate=cut(gate), alpha=0.5, quantize=True)
    for name in ("x", "n", "q", "rstd_post", "rstd_pre"):
        assert torch.equal(getattr(r, name)[PART], getattr(p, name)), name
    assert torch.equal(r.s[:, PART], p.s)
    dx, dn = _randn((M, C), 14, res), _randn((M, C), 15)
    g = fb.residual_norm_backward(r.x, dx_out=dx, dn=dn, rstd_pre=r.rstd_pre, w_pre=w1, f=f, rstd_post=r.rstd_post,
                                  w_post=w2, gate=gate, alpha=0.5)
    q = fb.residual_norm_backward(r.x[PART], dx_out=dx[PART], dn=dn[PART], rstd_pre=p.rstd_pre, w_pre=w1, f=f[PART],
                                  rstd_post=p.rstd_post, w_post=w2, gate=cut(gate), alpha=0.5)
    assert torch.equal(g.dx[PART], q.dx) and torch.equal(g.df[PART], q.df)
    if gate_row:
        assert torch.equal(g.dgate[PART], q.dgate)
    t = dn.double() * r.x.double() * r.rstd_pre.double()[:, None]
    assert bool(((g.dw_pre - t.sum(0)).abs() <= 2 * (M + 4) * U * t.abs().sum(0)).all())


@pytest.mark.parametrize("src,dst", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                     (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_clip(src, dst):
    """Past 2^24 elements, with pieces that start off the 16-byte grid."""
    sizes = [2 ** 24 + 3, 5, 1 << 20, 4097, 3 * 2 ** 20 + 1]
    flat = _randn((sum(sizes) + 1,), 16, src, 1e-3)[1:]
    ts = list(torch.split(flat, sizes))
    out = torch.empty(sum(sizes) + 1, dtype=dst, device="cuda")[1:]
    norm = fb.clip_grad_norm(fb.grad_table(ts, list(torch.split(out, sizes))), 0.25)
    want = float(flat.double().square().sum().sqrt())
    assert abs(float(norm) - want) <= 2 * U * want
    c = torch.tensor(0.25, device="cuda") / (norm + 1e-6)
    assert torch.equal(out, (flat.float() * c).to(dst))
    small = [t.clone() for t in ts[1:4]]
    fb.grad_clip(small, norm, 0.25)
    for t, s in zip(ts[1:4], small):
        assert torch.equal(s, (t.float() * c).to(src))
