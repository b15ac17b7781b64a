"""The memory that the optimizer's tables and the gated products' outputs name:
what changed since it was checked, and what two of them share, is refused on the
host before anything is enqueued.

CPU only: every call is refused, or asked on the host alone.
"""
import pytest
import torch

import fp8_fine_grained_quantize_amd as fb
from fp8_fine_grained_quantize_amd import train

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def _state(n=100, dtype=torch.float32, copies=True):
    p = torch.nn.Parameter(torch.zeros(n))
    return p, fb.AdamWState([p], dtype=dtype, copies=[torch.zeros(n, dtype=BF)] if copies else None)


# --- a state that changed after it was checked ----------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, BF, E4])
def test_parameter_of_another_size(dtype):
    for n in (100000, 129, 99):
        p, s = _state(dtype=dtype, copies=False)
        p.data = torch.zeros(n)
        with pytest.raises(ValueError, match="parameter 0"):
            train._entries(s, [torch.zeros(n)])


def _swapped(dtype, name, t):
    p, s = _state(dtype=dtype)
    getattr(s, name)[0] = t
    return lambda: train._entries(s, [torch.zeros(100)])


@pytest.mark.parametrize("name", ["ms", "vs"])
def test_moments_replaced(name):
    for dtype, kind in ((torch.float32, torch.float32), (BF, BF), (E4, torch.uint8)):
        for t in (torch.zeros(3, dtype=kind), torch.zeros(200, dtype=kind)[::2], torch.zeros(100, dtype=kind, device="meta")):
            with pytest.raises(ValueError, match="moments of parameter 0"):
                _swapped(dtype, name, t)()
        with pytest.raises(TypeError, match="moments"):
            _swapped(dtype, name, torch.zeros(100, dtype=torch.float64))()
        with pytest.raises(TypeError, match="tensor"):
            _swapped(dtype, name, None)()


@pytest.mark.parametrize("name", ["m_scales", "v_scales"])
def test_scales_replaced(name):
    for t in (torch.zeros(2), torch.zeros(0), torch.zeros(1, device="meta")):
        with pytest.raises(ValueError, match="scales of parameter 0"):
            _swapped(E4, name, t)()
    with pytest.raises(TypeError, match="scales of parameter 0"):
        _swapped(E4, name, torch.zeros(1, dtype=torch.float64))()
    with pytest.raises(TypeError, match="tensor"):
        _swapped(E4, name, None)()


def test_copies_replaced():
    for t in (torch.zeros(3, dtype=BF), torch.zeros(1, dtype=BF).expand(100), torch.zeros(100, dtype=BF, device="meta")):
        with pytest.raises(ValueError, match="copy"):
            _swapped(E4, "copies", t)()
    with pytest.raises(TypeError, match="copy 0 must be bfloat16"):
        _swapped(E4, "copies", torch.zeros(100))()


def test_lists_of_another_length():
    for name in ("params", "ms", "vs", "m_scales", "v_scales", "copies"):
        for change in (lambda v: v.pop(), lambda v: v.append(torch.zeros(100))):
            p, s = _state(dtype=E4)
            change(getattr(s, name))
            with pytest.raises(ValueError):
                train._entries(s, [torch.zeros(100)])


def test_state_unchanged():
    for dtype in (torch.float32, BF, E4):
        p, s = _state(dtype=dtype)
        p.data = torch.ones(100)  # other memory of the same kind
        s.ms[0] = s.ms[0].clone()
        e, = train._entries(s, [torch.zeros(100)])
        assert e.param == p.data_ptr() and e.m == s.ms[0].data_ptr()
