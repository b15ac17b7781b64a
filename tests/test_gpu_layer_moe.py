"""GPU tests of the sort by expert, dispatch and combine and their gradients,
against the plain 64-bit forms of layer_ref.py.

The maps are whole numbers and the dispatched rows copies: both must be equal.
Sums are held to the bounds of layer_ref.py.  Rows of dropped pairs hold NaN
wherever an operator must not read them.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
import oracle
import synthetic
from tests import layer_ref as ref
from tests.layer_ref import U, UB

pytestmark = pytest.mark.gpu


def _routing(T, K, E, drop, seed):
    """ids [T][K] int64 (numpy): skewed over the experts, -1 or >= E where dropped."""
    rng = np.random.default_rng(seed)
    p = np.exp(rng.normal(size=max(E, 1)))
    ids = rng.choice(max(E, 1), size=(T, K), p=p / p.sum()).astype(np.int64)
    gone = rng.random((T, K)) < drop
    ids[gone] = rng.choice([-1, E, E + 7, -(2 ** 31), 2 ** 31 - 1], size=int(gone.sum()))
    return ids


def _maps(ids, E):
    off, row_of, slot_of = ref.sort_pairs(ids, E)
    return off, row_of, slot_of, torch.from_numpy(row_of.astype(np.int32)).cuda(), \
        torch.from_numpy(slot_of.astype(np.int32)).cuda()


def _matrix(rows, cols, dtype, seed, std=1.0, pad=0):
    """Device matrix with `pad` extra 16-byte units of pitch; the padding holds a marker."""
    g = torch.Generator().manual_seed(seed)
    es = torch.empty(0, dtype=dtype).element_size()
    per = 16 // es
    pitch = (-(-cols // per) + pad) * per
    full = torch.full((rows, pitch), 77, dtype=dtype)
    full[:, :cols] = (torch.randn(rows, cols, generator=g) * std).to(dtype)
    return full.cuda()[:, :cols]


def _np(t):
    return t.detach().cpu().double().numpy()


SORTS = [(1, 1, 1, 0.0), (1, 8, 256, 0.0), (16, 8, 256, 0.0), (63, 1, 7, 0.3), (64, 1, 1, 1.0), (65, 3, 960, 0.1),
         (512, 8, 256, 0.05), (513, 8, 300, 0.05), (3000, 8, 256, 0.0), (2731, 7, 63, 0.5), (5000, 3, 960, 0.02),
         (8192, 8, 256, 0.03), (40000, 8, 64, 0.0), (7, 5, 0, 0.0), (9001, 1, 128, 1.0)]


@pytest.mark.parametrize("T,K,E,drop", SORTS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, K, E, drop, dtype):
    print(f"[layer] sort T={T} K={K} E={E} drop={drop} {dtype}", flush=True)
    ids = _routing(T, K, E, drop, T + K)
    off, row_of, slot_of = ref.sort_pairs(ids, E)
    got = fb.moe_sort(torch.from_numpy(ids).to(dtype).cuda(), E)
    for name, a, b in zip(("offsets", "row_of", "slot_of"), got, (off, row_of, slot_of)):
        assert a.dtype == torch.int32 and np.array_equal(a.cpu().numpy(), b), name


def test_sort_strided_ids_and_given_outputs():
    ids = _routing(700, 6, 32, 0.1, 3)
    wide = torch.full((700, 9), -5, dtype=torch.int32)
    wide[:, 2:8] = torch.from_numpy(ids).to(torch.int32)
    view = wide.cuda()[:, 2:8]
    off, row_of, slot_of = ref.sort_pairs(ids, 32)
    out = [torch.full(s, 99, dtype=torch.int32, device="cuda") for s in ((33,), (700, 6), (4200,))]
    fb.moe_sort(view, 32, *out)
    for a, b in zip(out, (off, row_of, slot_of)):
        assert np.array_equal(a.cpu().numpy(), b)
    got = fb.moe_sort(view.t().contiguous().t(), 32)  # column-major ids
    assert np.array_equal(got[1].cpu().numpy(), row_of)


# Around the sizes where one workgroup, several that count all pairs, and two
# launches take over; all pairs of one expert, and none kept.
TURNS = [(2048, 1, 256, 0.0), (683, 3, 9, 0.2), (2049, 1, 512, 0.1), (1000, 8, 1, 0.0), (1024, 8, 256, 0.0),
         (1024, 8, 500, 1.0), (2731, 3, 64, 0.1), (1025, 8, 512, 0.1), (512, 8, 600, 0.1), (513, 8, 600, 0.1)]


@pytest.mark.parametrize("T,K,E,drop", TURNS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_where_its_form_changes(T, K, E, drop, dtype):
    test_sort(T, K, E, drop, dtype)


@pytest.mark.parametrize("T,K", [(0, 8), (5, 0), (0, 0)])
def test_sort_empty(T, K):
    off, row_of, slot_of = fb.moe_sort(torch.empty(T, K, dtype=torch.int32, device="cuda"), 17)
    assert off.tolist() == [0] * 18 and row_of.shape == (T, K) and slot_of.numel() == 0


def test_sort_many_pairs_many_workgroups():
    """More pairs per wave than one 64-lane step: against torch's stable sort."""
    T, K, E = 150001, 9, 200
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-2, E + 3, (T, K), generator=g, device="cuda")
    key = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E)).reshape(-1).cpu()
    order = torch.sort(key, stable=True).indices
    off, row_of, slot_of = fb.moe_sort(ids, E)
    s = slot_of.cpu().long()
    assert torch.equal(torch.where(s < 0, -1 - s, s), order)
    assert off.cpu().tolist() == [0] + torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0).tolist()
    r = row_of.reshape(-1).cpu().long()
    assert torch.equal(torch.where(r < 0, -1 - r, r)[order], torch.arange(T * K))
    assert torch.equal(r < 0, key == E)


SHAPES = [(1, 1, 8, 64, 0.0), (16, 8, 256, 7168, 0.0), (5, 3, 4, 1, 0.0), (33, 2, 7, 2051, 0.2), (70, 9, 30, 128, 0.1),
          (129, 8, 64, 200, 0.05), (20, 4, 5, 333, 1.0), (3, 17, 40, 4100, 0.3)]


@pytest.mark.parametrize("T,K,E,C,drop", SHAPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_dispatch(T, K, E, C, drop, pad):
    print(f"[layer] dispatch T={T} K={K} C={C} drop={drop}", flush=True)
    off, row_of, slot_of, dr, ds = _maps(_routing(T, K, E, drop, 11), E)
    tok = np.where(slot_of < 0, -1, slot_of // K)
    x = _matrix(T, C, torch.bfloat16, 5, pad=pad)
    out = _matrix(T * K, C, torch.bfloat16, 6, pad=pad)
    fb.moe_dispatch(x, dr, out=out)
    want = np.where((tok >= 0)[:, None], _np(x)[np.maximum(tok, 0)], 0.0)
    assert np.array_equal(_np(out), want)
    assert torch.equal(fb.moe_dispatch(x, dr), out)
    if pad:  # the padding between rows is not written
        assert (torch.as_strided(out, (T * K - 1, out.stride(0) - C), (out.stride(0), 1),
                                 out.storage_offset() + C) == 77).all()
    q = fb.empty_pitched(T, C, torch.uint8)
    q.copy_(synthetic.random_codes((T, C), 3))
    s = synthetic.random_scales((-(-C // 128), T), 4)
    qr, sr = fb.moe_dispatch_fp8(q, s, dr, ds)
    assert np.array_equal(qr.cpu().numpy(), np.where((tok >= 0)[:, None], q.cpu().numpy()[np.maximum(tok, 0)], 0))
    assert np.array_equal(sr.cpu().numpy(), np.where((tok >= 0)[None], s.cpu().numpy()[:, np.maximum(tok, 0)], 1.0))


@pytest.mark.parametrize("T,K,E,C,drop", SHAPES)
@pytest.mark.parametrize("rows_dt,out_dt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                            (torch.bfloat16, torch.float32), (torch.float32, torch.float32)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, K, E, C, drop, rows_dt, out_dt, weighted):
    print(f"[layer] combine T={T} K={K} C={C} drop={drop} {rows_dt} {out_dt} {weighted}", flush=True)
    off, row_of, _, dr, _ = _maps(_routing(T, K, E, drop, 12), E)
    rows = _matrix(T * K, C, rows_dt, 7, pad=1)
    rows[int(off[-1]):] = float("nan")
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(2)).cuda() if weighted else None
    y = fb.moe_combine(rows, dr, w, out_dtype=out_dt)
    want, mag = ref.combine(_np(rows), row_of, None if w is None else _np(w))
    bound = 2 * (K + 1) * U * mag + (UB * np.abs(want) if out_dt == torch.bfloat16 else 0)
    assert y.dtype == out_dt and np.all(np.abs(_np(y) - want) <= bound)


@pytest.mark.parametrize("T,K,E,C,drop", SHAPES)
@pytest.mark.parametrize("dy_dt,rows_dt,drows_dt", [
    (torch.bfloat16, torch.bfloat16, None), (torch.float32, torch.float32, None),
    (torch.bfloat16, torch.float32, torch.bfloat16), (torch.float32, torch.bfloat16, torch.float32)])
def test_combine_backward(T, K, E, C, drop, dy_dt, rows_dt, drows_dt):
    print(f"[layer] combine grad T={T} K={K} C={C} drop={drop} {dy_dt} {rows_dt}", flush=True)
    off, row_of, _, dr, _ = _maps(_routing(T, K, E, drop, 13), E)
    rows = _matrix(T * K, C, rows_dt, 8)
    rows[int(off[-1]):] = float("nan")
    dy = _matrix(T, C, dy_dt, 9, pad=2)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(3)).cuda()
    drows, dw = fb.moe_combine_backward(dy, rows, dr, w, drows_dtype=drows_dt)
    wr, wd, mag = ref.combine_backward(_np(dy), _np(rows), row_of, _np(w))
    bound = 2 * U * np.abs(wr) + (UB * np.abs(wr) if drows.dtype == torch.bfloat16 else 0)
    assert drows.dtype == (drows_dt or rows_dt) and np.all(np.abs(_np(drows) - wr) <= bound)
    assert np.all(np.abs(_np(dw) - wd) <= 2 * C * U * mag)


@pytest.mark.parametrize("C", [3, 4, 7, 8, 9, 15, 16, 17, 31, 33, 65, 513, 1027, 2049])
def test_row_ends(C):
    """Rows around the widths that one lane moves or sums; the last lane's share
    overlaps the one before."""
    test_dispatch(37, 3, 9, C, 0.1, 1)
    for a, b in ((torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)):
        test_combine(37, 3, 9, C, 0.1, a, b, True)
        test_combine_backward(37, 3, 9, C, 0.1, a, b, a)


def test_an_infinity_at_a_row_end_counts_once():
    T, C = 4, 1027
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    _, row_of, _ = fb.moe_sort(ids, 1)
    dy = fb.as_pitched(torch.ones(T, C, dtype=torch.bfloat16, device="cuda"))
    rows, w = dy.clone(), torch.ones(T, 1, device="cuda")
    rows = fb.as_pitched(rows)
    rows[1, C - 5], rows[2, C - 1], dy[3, C - 2] = float("inf"), float("-inf"), float("inf")
    drows, dw = fb.moe_combine_backward(dy, rows, row_of, w)
    assert dw[:, 0].tolist() == [float(C), float("inf"), float("-inf"), float("inf")]
    assert torch.equal(drows, dy)


def test_gradients_by_differences():
    """Central differences of the 64-bit combine: exact up to rounding, as it
    is linear in the rows and in the weights."""
    T, K, E, C = 6, 3, 5, 40
    off, row_of, _, dr, _ = _maps(_routing(T, K, E, 0.2, 14), E)
    rows = _matrix(T * K, C, torch.float32, 1)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(4)).cuda()
    dy = _matrix(T, C, torch.float32, 2)
    drows, dw = fb.moe_combine_backward(dy, rows, dr, w)
    R, W, D = _np(rows), _np(w), _np(dy)

    def loss(r_, w_):
        return float((ref.combine(r_, row_of, w_)[0] * D).sum())

    h = 2.0 ** -6
    rng = np.random.default_rng(0)
    size = float(np.abs(D).sum() * np.abs(R).max())
    for _ in range(20):
        i, j = int(rng.integers(T * K)), int(rng.integers(C))
        e = np.zeros_like(R)
        e[i, j] = h
        d = (loss(R + e, W) - loss(R - e, W)) / (2 * h)
        assert abs(d - float(drows[i, j])) <= 2 * U * abs(d) + 2.0 ** -50 * size / h
        t, k = int(rng.integers(T)), int(rng.integers(K))
        e = np.zeros_like(W)
        e[t, k] = h
        d = (loss(R, W + e) - loss(R, W - e)) / (2 * h)
        assert abs(d - float(dw[t, k])) <= 2 * C * U * size + 2.0 ** -50 * size / h


def test_dispatch_and_combine_are_transposed():
    """<dispatch(x), r> = <x, combine(r)> on whole numbers: exact."""
    T, K, E, C = 50, 4, 9, 136
    _, row_of, _, dr, _ = _maps(_routing(T, K, E, 0.1, 15), E)
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.integers(-8, 9, (T, C))).to(torch.bfloat16).cuda()
    r = torch.from_numpy(rng.integers(-8, 9, (T * K, C))).to(torch.float32).cuda()
    a = (_np(fb.moe_dispatch(x, dr)) * _np(r)).sum()
    b = (_np(x) * _np(fb.moe_combine(r, dr, out_dtype=torch.float32))).sum()
    assert a == b


def test_infinite_and_nan_rows_reach_only_their_token():
    T, K, E, C = 8, 2, 4, 64
    off, row_of, _, dr, _ = _maps(_routing(T, K, E, 0.0, 16), E)
    rows = _matrix(T * K, C, torch.bfloat16, 3)
    rows[int(row_of[3, 1]), 5] = float("inf")
    rows[int(row_of[6, 0]), 9] = float("nan")
    y = fb.moe_combine(rows, dr)
    bad = ~torch.isfinite(y.float())
    assert bad.nonzero().tolist() == [[3, 5], [6, 9]] and torch.isinf(y[3, 5])


def test_maps_out_of_range_are_skipped():
    """A row outside [0, T*K) is neither read nor written."""
    T, K, C = 3, 2, 64
    row_of = torch.tensor([[0, 6], [2, 2 ** 31 - 1], [-(2 ** 31), 1]], dtype=torch.int32, device="cuda")
    x = _matrix(T, C, torch.bfloat16, 4)
    out = torch.full((T * K, C), 7.0, dtype=torch.bfloat16, device="cuda")
    fb.moe_dispatch(x, row_of, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[2], x[1]) and torch.equal(out[1], x[2])
    assert (out[3:] == 7.0).all()
    y = fb.moe_combine(out, row_of)
    assert torch.equal(y, x)


def test_long_row_offsets():
    """Rows past 2^31 elements from the start of the matrix."""
    T, K, C = 8, 1, 2 ** 17
    P = 2 ** 14 + 9   # rows: P * C = 2^31 + 9 * 2^17 elements, 4.3 GB of BF16
    rows = torch.zeros(P, C, dtype=torch.bfloat16, device="cuda")
    row_of = torch.full((P, 1), -1, dtype=torch.int32, device="cuda")
    row_of[:, 0] = torch.arange(P - 1, -1, -1, dtype=torch.int32, device="cuda")
    x = torch.zeros(P, C, dtype=torch.bfloat16, device="cuda")
    x[0] = _matrix(1, C, torch.bfloat16, 1)[0]
    x[5] = _matrix(1, C, torch.bfloat16, 2)[0]
    fb.moe_dispatch(x, row_of, out=rows)
    assert torch.equal(rows[P - 1], x[0]) and torch.equal(rows[P - 6], x[5])
    y = fb.moe_combine(rows, row_of)
    assert torch.equal(y[0], x[0]) and torch.equal(y[5], x[5]) and not y[6].any()


def test_rows_feed_the_grouped_gemm():
    """Quantized tokens dispatched to their experts, through the grouped GEMM
    and back: each token gets the weighted sum of its experts' products."""
    T, K, E, C, N = 40, 3, 6, 256, 128
    ids = torch.from_numpy(_routing(T, K, E, 0.1, 17)).cuda()
    off, row_of, slot_of = fb.moe_sort(ids, E)
    x = _matrix(T, C, torch.bfloat16, 5)
    q, s = fb.quantize_1x128(x)
    qr, sr = fb.moe_dispatch_fp8(q, s, row_of, slot_of)
    W = torch.randn(E, C, N, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    codes = [fb.quantize_block128(W[e].cuda()) for e in range(E)]
    qw, sw = torch.stack([c[0] for c in codes]), torch.stack([c[1] for c in codes])
    h = fb.grouped_gemm_fp8_blockscaled(off, qr, sr, qw, sw)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(7)).cuda()
    y = _np(fb.moe_combine(h, row_of, w, out_dtype=torch.float32))
    X = oracle.dequantize_1x128(q.cpu().numpy(), s.cpu().numpy()).astype(np.float64)
    want = np.zeros((T, N))
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            if 0 <= e < E:
                We = oracle.dequantize_block128(qw[e].cpu().numpy(), sw[e].cpu().numpy()).astype(np.float64)
                want[t] += float(w[t, k]) * (X[t] @ We)
    # the GEMM's own gate, 1e-3 of the largest magnitude
    assert np.max(np.abs(y - want)) <= 1e-3 * np.max(np.abs(want))
