"""GPU tests of the global gradient norm and clipping, against 64-bit sums.

The squares are summed in FP64, so the norm is the exact one rounded to FP32
(relative error at most 2 U, one U from the final rounding and far less from
the sum); the coefficient adds three FP32 operations, the product one, and a
BF16 output its rounding.
"""
import math

import numpy as np
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from tests.layer_ref import U, UB

pytestmark = pytest.mark.gpu


def _tensor(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def _np(t):
    return t.detach().cpu().double().numpy()


def _norm(ts):
    return math.sqrt(sum(float((_np(t) ** 2).sum()) for t in ts))


def _list(kind):
    """Shapes of every kind of gradient; sizes around the work chunk of 8192."""
    n = [1, 7, 8, 63, 4096, 8191, 8192, 8193, 16385, 50001]
    if kind == "mixed":
        ts = [_tensor((m,), torch.bfloat16 if i % 2 else torch.float32, i) for i, m in enumerate(n)]
        return ts + [_tensor((3, 5, 7), torch.float32, 90), _tensor((), torch.bfloat16, 91),
                     _tensor((0, 4), torch.float32, 92)]
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    return [_tensor((m,), dt, i) for i, m in enumerate(n)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("factor", [0.25, 4.0])
def test_clip_in_place(kind, factor):
    print(f"[layer] clip {kind} {factor}", flush=True)
    ts = _list(kind)
    before = [t.clone() for t in ts]
    want = _norm(ts)
    got = fb.grad_norm(ts)
    assert got.shape == () and abs(float(got) - want) <= 2 * U * want
    norm = fb.clip_grad_norm(ts, factor * want)
    assert torch.equal(norm, got)
    c = min(1.0, factor * want / (want + 1e-6))
    for t, b in zip(ts, before):
        if factor > 1:
            assert torch.equal(t, b)
        else:
            w = _np(b) * c
            assert np.all(np.abs(_np(t) - w) <= (6 * U + (UB if t.dtype == torch.bfloat16 else 0)) * np.abs(w))


@pytest.mark.parametrize("out_dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("factor", [0.25, 4.0])
def test_clip_into_a_flat_buffer(out_dt, factor):
    """Outputs packed back to back: aligned to their element only."""
    ts = _list("mixed")
    sizes = [t.numel() for t in ts]
    flat = torch.full((sum(sizes) + 2,), 5.0, dtype=out_dt, device="cuda")
    outs = [o.view(t.shape) for o, t in zip(torch.split(flat[1:-1], sizes), ts)]
    before = [t.clone() for t in ts]
    want = _norm(ts)
    table = fb.grad_table(ts, outs)
    norm = fb.clip_grad_norm(table, factor * want)
    c = min(1.0, factor * want / (want + 1e-6))
    for t, b, o in zip(ts, before, outs):
        assert torch.equal(t, b)
        w = _np(b) * c
        assert np.all(np.abs(_np(o) - w) <= (6 * U + (UB if out_dt == torch.bfloat16 else 0)) * np.abs(w))
    assert float(flat[0]) == 5.0 and float(flat[-1]) == 5.0
    fb.grad_clip(table, norm, factor * want)  # by a given norm: the same
    assert abs(float(norm) - want) <= 2 * U * want


def test_strided_gradients():
    base = _tensor((300, 250), torch.float32, 1)
    ts = [base[:, 3:200], _tensor((200, 123), torch.bfloat16, 2).t(), _tensor((5, 40, 72), torch.float32, 3)[:, 1:39, :65],
          _tensor((4000,), torch.bfloat16, 4)[::2]]
    keep = base.clone()
    before = [t.clone() for t in ts]
    want = _norm(ts)
    fb.clip_grad_norm(ts, 0.5 * want)
    for t, b in zip(ts, before):
        w = _np(b) * 0.5 * want / (want + 1e-6)
        assert np.all(np.abs(_np(t) - w) <= (6 * U + (UB if t.dtype == torch.bfloat16 else 0)) * np.abs(w))
    assert torch.equal(base[:, :3], keep[:, :3]) and torch.equal(base[:, 200:], keep[:, 200:])
    # a transposed gradient into a dense output, a pitched output from a dense gradient
    src = [_tensor((60, 90), torch.float32, 5).t(), _tensor((70, 33), torch.bfloat16, 6)]
    outs = [torch.zeros(90, 60, device="cuda"), torch.full((70, 40), 9.0, device="cuda")[:, :33]]
    fb.clip_grad_norm(fb.grad_table(src, outs), 1e9)
    assert all(torch.equal(o, t.float()) for o, t in zip(outs, src))


def test_pieces_past_2_31_elements():
    n = 2 ** 31 + 12345
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[5], t[n - 1], t[2 ** 31 + 3] = 3.0, 4.0, 12.0
    assert float(fb.clip_grad_norm([t], 6.5)) == 13.0
    c = np.float32(6.5) / (np.float32(13.0) + np.float32(1e-6))
    for i, v in ((5, 3.0), (n - 1, 4.0), (2 ** 31 + 3, 12.0)):
        assert abs(float(t[i]) - v * float(c)) <= UB * v
    assert int((t != 0).sum()) == 3


@pytest.mark.parametrize("value", [1e30, 1e-30])
def test_extreme_magnitudes(value):
    """Squares far outside the FP32 range still count."""
    t = torch.full((10000,), value, device="cuda")
    want = 100.0 * float(np.float32(value))
    assert abs(float(fb.grad_norm([t])) - want) <= 2 * U * want


def test_non_finite():
    t = [_tensor((5000,), torch.float32, 1), _tensor((50,), torch.bfloat16, 2)]
    t[0][77] = float("inf")
    norm = fb.clip_grad_norm(t, 1.0)
    assert math.isinf(float(norm)) and not t[1].any() and torch.isnan(t[0][77]) and not t[0][78:].any()
    t = [_tensor((5000,), torch.float32, 1), _tensor((50,), torch.bfloat16, 2)]
    t[1][3] = float("nan")
    assert math.isnan(float(fb.clip_grad_norm(t, 1.0))) and torch.isnan(t[0]).all() and torch.isnan(t[1]).all()


def test_nothing_to_clip():
    assert float(fb.grad_norm([])) == 0.0 and float(fb.clip_grad_norm([], 1.0)) == 0.0
    z = [torch.zeros(100, device="cuda"), torch.empty(0, device="cuda")]
    assert float(fb.clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()


def test_many_tensors():
    """More tensors than one search step of 64, and than 64 * 64."""
    for n in (64, 65, 4097, 5000):
        ts = list(torch.split(_tensor((n * 3,), torch.float32, n), 3))
        want = _norm([torch.cat(ts)])
        before = torch.cat(ts)
        assert abs(float(fb.clip_grad_norm(ts, want / 2)) - want) <= 2 * U * want
        w = _np(before) * (want / 2) / (want + 1e-6)
        assert np.all(np.abs(_np(torch.cat(ts)) - w) <= 6 * U * np.abs(w))


def test_refuses():
    t = torch.zeros(8, device="cuda")
    with pytest.raises(TypeError):
        fb.grad_norm([t.double()])
    with pytest.raises(ValueError):
        fb.grad_table([t], [t, t])
    with pytest.raises(ValueError):
        fb.grad_table([t], [torch.zeros(9, device="cuda")])
    with pytest.raises(ValueError):
        fb.grad_table([torch.zeros(1, device="cuda").expand(8)])
    with pytest.raises(ValueError):
        fb.grad_norm([torch.zeros(8)])
    with pytest.raises(fb.Fp8BlkError):
        fb.clip_grad_norm([t], -1.0)
    with pytest.raises(fb.Fp8BlkError):
        fb.clip_grad_norm([t], float("nan"))
