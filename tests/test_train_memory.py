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


# --- gated products: what they write shares no memory ---------------------------

M, H, K = 8, 256, 384
U8 = torch.uint8


def _operands(N, G=None):
    of = [] if G is None else [G]
    return dict(A=torch.zeros(M, K, dtype=U8), sA=torch.zeros(K // 128, M), B=torch.zeros(*of, K, N, dtype=U8),
                sB=torch.zeros(*of, K // 128, N // 128))


def _outputs(**width):
    """u, h, q, s or du, h, q, s of the given widths, a lent workspace too."""
    d = {k: torch.zeros(M, n, dtype=U8 if k == "q" else BF) for k, n in width.items()}
    return dict(d, s=torch.zeros(d["q"].shape[1] // 128, M), workspace=torch.zeros(4096))


def _forward(offsets=None, **kw):
    if offsets is None:
        return fb.gated_gemm_fp8_blockscaled(quantize=True, **kw)
    kw.pop("workspace")
    return fb.grouped_gated_gemm_fp8_blockscaled(offsets, quantize=True, **kw)


def _backward(offsets=None, **kw):
    if offsets is None:
        return fb.gated_gemm_backward_fp8_blockscaled(quantize=True, opB=0, **kw)
    kw.pop("workspace")
    return fb.grouped_gated_gemm_backward_fp8_blockscaled(offsets, quantize=True, opB=0, **kw)


CALLS = [(_forward, 2 * H, dict(u=2 * H, h=H, q=H)), (_backward, H, dict(du=2 * H, h=H, q=2 * H))]


def _call(f, N, widths, G):
    kw = dict(_operands(N, G), **_outputs(**widths))
    if f is _backward:
        kw["u"] = torch.zeros(M, 2 * H, dtype=BF)
    offsets = None if G is None else torch.zeros(G + 1, dtype=torch.int32)
    return kw, offsets


@pytest.mark.parametrize("f,N,widths", CALLS)
@pytest.mark.parametrize("G", [None, 3])
def test_outputs_share_memory(f, N, widths, G):
    """Each output in each other one's, each operand's and the workspace's memory, at its first byte."""
    kw, offsets = _call(f, N, widths, G)
    with pytest.raises(ValueError, match="current GPU"):  # nothing shared: refused as CPU tensors only
        f(offsets, **kw)
    inputs = ["A", "sA", "B", "sB"] + (["u"] if f is _backward else []) + ([] if G is None else ["offsets"])
    outputs = [*widths, "s"] + (["workspace"] if G is None else [])
    for o in outputs:
        for other in inputs + outputs:
            if o == other or {o, other} == {"du", "u"}:
                continue
            kw, offsets = _call(f, N, widths, G)
            room = torch.zeros(1 << 21, dtype=U8)
            for k in (o, other):
                t = offsets if k == "offsets" else kw[k]
                t = room.view(t.dtype).as_strided(t.shape, t.stride())
                if k == "offsets":
                    offsets = t
                else:
                    kw[k] = t
            with pytest.raises(ValueError, match=f"^({o} shares memory with {other}|{other} shares memory with {o})$"):
                f(offsets, **kw)


@pytest.mark.parametrize("f,N,widths", CALLS)
def test_outputs_that_only_touch(f, N, widths):
    """Rows between rows, one after another in one buffer, and the last byte."""
    kw, _ = _call(f, N, widths, None)
    first, wide = list(widths)[0], torch.zeros(M, 3 * H, dtype=BF)
    kw[first], kw["h"] = wide[:, :2 * H], wide[:, 2 * H:]
    with pytest.raises(ValueError, match="current GPU"):
        f(**kw)
    kw["h"] = wide[:, 2 * H - 1:3 * H - 1]
    with pytest.raises(ValueError, match=f"^h shares memory with {first}$"):
        f(**kw)
    # experts' weights whose matrices lie apart, an output in the space between them, and one byte too far
    kw, _ = _call(f, N, widths, 3)
    room = torch.zeros(3, K * N + M * H * 2, dtype=U8)
    kw["B"] = room[:, :K * N].as_strided((3, K, N), (room.stride(0), N, 1))
    gap = room[1].view(BF)[K * N // 2:].view(M, H)
    offsets = torch.zeros(4, dtype=torch.int32)
    kw["h"] = gap
    with pytest.raises(ValueError, match="current GPU"):
        f(offsets, **kw)
    kw["h"] = room.view(-1).view(BF)[(room.stride(0) + K * N) // 2 - 1:][:M * H].view(M, H)
    with pytest.raises(ValueError, match="^h shares memory with B$"):
        f(offsets, **kw)


def test_gradient_in_place():
    kw, _ = _call(*CALLS[1], None)
    for du in (kw["u"], kw["u"].view(M, 2 * H)):  # u itself
        with pytest.raises(ValueError, match="current GPU"):
            _backward(**dict(kw, du=du))
    room = torch.zeros(2 * M + 1, 2 * H, dtype=BF)
    kw["u"] = room[:M]
    for du in (room[1:M + 1], room[:2 * M:2], room[:M].view(torch.float16)):
        with pytest.raises(ValueError, match="^du shares memory with u$"):
            _backward(**dict(kw, du=du))
    with pytest.raises(ValueError, match="^h shares memory with "):  # in place, and h there too
        _backward(**dict(kw, du=kw["u"], h=kw["u"][:, :H]))


def test_workspace_that_is_not_used():
    """A call that is not split leaves its workspace alone."""
    kw, _ = _call(*CALLS[0], None)
    kw["workspace"] = kw["h"]
    with pytest.raises(ValueError, match="current GPU"):
        _forward(**kw, split_k=False)


# --- a table whose tensors have other memory by now -----------------------------

def _held(dtype=E4):
    p, s = _state(dtype=dtype)
    g = [torch.zeros(100)]
    return p, s, g, train._hold(s, g)


def _step(held):
    """A step refused as one of CPU tensors, unless what it holds has moved."""
    return train._ext().adamw_step(torch.zeros(64, dtype=torch.int64), 1, 1, 2, 1e-3, 1, 0.9, 0.95, 1e-8, None, None, 1e-6,
                                   None, held, None)


def test_step_after_memory_moved():
    def set_data(t, n=100):
        t.data = torch.zeros(n, dtype=t.dtype)

    changes = {"parameter 0": lambda p, s, g: set_data(p), "gradient 0": lambda p, s, g: set_data(g[0]),
               "first moment 0": lambda p, s, g: s.ms[0].untyped_storage().resize_(0),
               "second moment 0": lambda p, s, g: s.vs[0].resize_(1 << 20),
               "first moment's scales 0": lambda p, s, g: set_data(s.m_scales[0], 1),
               "second moment's scales 0": lambda p, s, g: set_data(s.v_scales[0], 1),
               "copy 0": lambda p, s, g: set_data(s.copies[0])}
    for what, change in changes.items():
        p, s, g, held = _held()
        with pytest.raises(ValueError, match="current GPU"):
            _step(held)
        change(p, s, g)
        with pytest.raises(ValueError, match=f"^{what} "):
            _step(held)


def test_table_keeps_its_memory():
    """Lists that change after the table was built: it goes on with the tensors that it was built of."""
    p, s, g, held = _held()
    at, kept = s.ms[0].data_ptr(), [s.ms[0].data_ptr(), g[0].data_ptr()]
    s.ms[0], g[0] = torch.ones(100, dtype=torch.uint8), torch.ones(100)
    fresh = [torch.zeros(100, dtype=torch.uint8) for _ in range(64)] + [torch.zeros(100) for _ in range(64)]
    assert not {t.data_ptr() for t in fresh} & set(kept) and at == kept[0]
    with pytest.raises(ValueError, match="current GPU"):
        _step(held)


def test_written_clone_on_write():
    """A tensor that shares its memory with a clone until either is written gets its own: the table is another one's."""
    p, s, g, held = _held(torch.float32)
    clone = torch._lazy_clone(s.ms[0])
    with pytest.raises(ValueError, match="^first moment 0 "):
        _step(held)
    assert clone.numel() == 100
