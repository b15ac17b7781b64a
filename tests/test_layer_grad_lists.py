"""Gradients of a list that share memory, on the CPU: which lists clipping must
refuse, against the sets of bytes that their tensors hold.
"""
import random

import pytest
import torch

from fp8_fine_grained_quantize_amd import layer


def _shared(ts, outs=None):
    entries, first = [], [0]
    for t, o in zip(ts, ts if outs is None else outs):
        flags = (1 if t.dtype == torch.float32 else 0) | (2 if o.dtype == torch.float32 else 0)
        layer._grad_entries(t, o, flags, entries)
        first.append(len(entries))
    return layer._shared((layer._Grad * max(1, len(entries)))(*entries), first)


def test_lists_that_share_nothing():
    t = torch.zeros(12, 20)
    assert _shared([]) is None and _shared([t]) is None and _shared([torch.zeros(0, 3), t]) is None
    assert _shared([t[:5], t[5:]]) is None and _shared([t[5:], t[:5]]) is None
    assert _shared([t[:, :7], t[:, 7:13], t[:, 13:]]) is None           # rows between rows
    assert _shared([t[::2], t[1::2, ::3], t[1::2, 1::3]]) is None
    assert _shared([t.view(-1)[0::2], t.view(-1)[1::2]]) is None
    assert _shared(list(torch.split(t.view(-1), 7))) is None
    o, p = torch.zeros(12, 20), torch.zeros(12, 20, dtype=torch.bfloat16)
    assert _shared([t, t], [o, p]) is None                               # only read
    assert _shared([t, o], [t, p]) is None and _shared([t], [t.view(12, 20)]) is None
    assert _shared([t, o], [torch.zeros(12, 20), o]) is None


def test_lists_that_share_memory():
    t, o = torch.zeros(12, 12), torch.zeros(12, 12)
    assert _shared([t, t]) == (0, 1) and _shared([o, t, t]) == (1, 2)    # a tied weight listed twice
    assert _shared([t, t.t()]) == (0, 1) and _shared([t, t[3:5]]) == (0, 1)
    assert _shared([t[:, :7], t[:, 6:]]) == (0, 1) and _shared([t.view(-1)[::2], t.view(-1)[::3]]) == (0, 1)
    assert _shared([t, o], [torch.zeros(12, 12), t]) == (0, 1)           # an output that is another's gradient
    assert _shared([t, t], [o, o]) == (0, 1) and _shared([t, t], [t, o]) == (0, 1)
    assert _shared([t, o], [torch.zeros(12, 12), torch.zeros(13, 12)[:12]]) is None
    assert _shared([t], [t.t()]) == (0, 0)                               # its own, but not in place
    b = torch.zeros(50)
    assert _shared([b[:40]], [b[1:41]]) == (0, 0) and _shared([b[:20]], [b[20:40]]) is None
    assert _shared([b[:20].view(torch.bfloat16)[:20]], [b[:20]]) == (0, 0)
    assert _shared([b[:20].view(torch.bfloat16)[:20]], [b[10:30]]) is None


@pytest.mark.parametrize("shape,expanded", [((1, 0), (3, 0)), ((0, 1), (0, 4)), ((1, 0, 5), (4, 0, 5))])
def test_expanded_tensors_without_elements(shape, expanded):
    t = torch.zeros(shape).expand(expanded)
    assert not layer._overlaps(t) and _shared([t, t]) is None


def _elements(t):
    """The addresses of t's elements, in order."""
    at = torch.zeros(t.shape, dtype=torch.int64)
    for d, (n, st) in enumerate(zip(t.shape, t.stride())):
        at = at + (torch.arange(n) * st).view([-1 if i == d else 1 for i in range(t.dim())])
    return (at * t.element_size() + t.data_ptr()).reshape(-1).tolist()


def _bytes(t):
    return {a + i for a in _elements(t) for i in range(t.element_size())}


def _own_race(t, o):
    """Whether an element of o lies on another element of t, or on its own but not the same way."""
    T, O = _elements(t), _elements(o)
    return any(a < q + o.element_size() and q < a + t.element_size() and not (i == j and a == q and t.dtype == o.dtype)
               for i, a in enumerate(T) for j, q in enumerate(O))


@pytest.mark.parametrize("seed", range(6))
def test_random_views_of_one_buffer(seed):
    rng = random.Random(seed)
    buf = torch.zeros(600)
    found = [0, 0]

    def view(shape=None):
        while True:
            base = buf if rng.random() < 0.5 else buf.view(torch.bfloat16)
            dims = shape or tuple(rng.randint(1, 5) for _ in range(rng.randint(1, 3)))
            t = base.as_strided(dims, [rng.choice([1, 2, 3, 5, 7, 11, 16, 20, 33]) for _ in dims], rng.randint(0, 150))
            if not layer._overlaps(t):
                return t

    while min(found) < 60:
        n = rng.randint(1, 3)
        ts = [view() for _ in range(n)]
        outs = [t if rng.random() < 0.4 else view(t.shape) for t in ts]
        G, O = [_bytes(t) for t in ts], [_bytes(t) for t in outs]
        two = {(min(i, j), max(i, j)) for i in range(n) for j in range(n) if i != j and (O[i] & G[j] or O[i] & O[j])}
        race = {(i, i) for i in range(n) if _own_race(ts[i], outs[i])}
        got = _shared(ts, outs)
        if two or race:
            assert got is not None, (ts, outs)
        # part of a tensor in place and the rest elsewhere may be refused too
        assert got is None or got in two or (got[0] == got[1] and outs[got[0]] is not ts[got[0]] and O[got[0]] & G[got[0]])
        found[got is not None] += 1
