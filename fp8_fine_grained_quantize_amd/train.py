"""The gated feed-forward block in FP8 and the optimizer step.

Argument marshalling only, in C++ as for the operators of ``layer.py``
(``csrc/train_binding.cpp``).  Names and argument meanings follow
``include/libfp8blk_train.h``.  Matrices are row-major with a 16-byte row pitch
(``empty_pitched`` / ``as_pitched``); missing outputs and workspaces are
allocated through torch on the current stream.  TypeError and ValueError refuse
arguments, Fp8BlkError reports a failed call.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

import fp8_fine_grained_quantize_amd as _fb

from .layer import _ext, _is_f32, _overlaps, _stream

_i64, _u32, _vp, _sz, _int, _f32 = (ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                                    ctypes.c_float)

SIGNATURES = {
    "fp8blk_train_abi_version": (_int, []),
    "fp8blk_gated_gemm_fp8_blockscaled": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _int, _vp, _int, _vp, _i64,
                                                 _vp, _i64, _vp, _i64, _vp, _u32, _vp, _sz, _vp]),
    "fp8blk_gated_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8blk_grouped_gated_gemm_fp8_blockscaled": (_int, [_i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64,
                                                         _int, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _u32,
                                                         _vp]),
    "fp8blk_gated_gemm_backward_fp8_blockscaled": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _int, _vp, _int, _vp,
                                                          _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _u32, _vp, _sz, _vp]),
    "fp8blk_gated_gemm_backward_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8blk_grouped_gated_gemm_backward_fp8_blockscaled": (_int, [_i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp,
                                                                  _i64, _i64, _int, _vp, _i64, _int, _vp, _i64, _vp, _i64,
                                                                  _vp, _i64, _vp, _i64, _vp, _u32, _vp]),
    "fp8blk_adamw_table_bytes": (_sz, [_i64]),
    "fp8blk_adamw_table_build": (_int, [_vp, _i64, _int, _vp, _sz, _vp]),
    "fp8blk_adamw_step": (_int, [_vp, _i64, _i64, _int, _vp, _vp]),
}
TRAIN_SYMBOLS = tuple(SIGNATURES)

_PARAM_F32, _GRAD_F32 = 0x1, 0x2
_STATES = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}


def train_abi_version() -> int:
    return _fb.lib().fp8blk_train_abi_version()


# --------------------------------------------------------------------------
# the gated feed-forward block
# --------------------------------------------------------------------------
_ACTS = {"silu": 0, "gelu": 1}


class GatedGemm(NamedTuple):
    """u: the projections, kept for the gradient; h: act(gate) * up; (q, s): its 1x128 codes and scales."""
    u: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    s: Optional[torch.Tensor]


class GatedGemmGrad(NamedTuple):
    """du: gradient of u; (q, s): its 1x128 codes and scales; h: act(gate) * up of the u given."""
    du: Optional[torch.Tensor]
    h: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    s: Optional[torch.Tensor]


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}, got {act!r}")
    return _ACTS[act]


def gated_gemm_fp8_blockscaled(A, sA, B, sB, act: str = "silu", opB: int = 0, pow2_scales: bool = False,
                               quantize: bool = False, pow2: bool = False, want_h: bool = True, want_u: bool = True,
                               split_k: bool = True, workspace=None, u=None, h=None, q=None, s=None) -> GatedGemm:
    """Gate and up projection, activation and product in one GEMM: u = A B (A uint8 codes [M][K], B [K][2H]
    for OP_N or [2H][K] for OP_T, its first H columns the gate's; scales, opB and pow2_scales as in
    gemm_fp8_blockscaled), h = act(u[:, :H]) * u[:, H:] with act "silu" or "gelu" (tanh form).  Returns u
    bf16 [M][2H] unless want_u is False, h bf16 [M][H], and with quantize (q uint8 [M][H], s float32
    [H/128][M]) = quantize_1x128(h, pow2); want_h=False then leaves h out.  H and K are multiples of 128.
    split_k: a product of few rows is split over the GPU, with a workspace allocated here unless given (which
    no other work, a captured graph's neither, may use at the same time; one that is too small or not 16-byte
    aligned leaves the call to one launch).  Outputs and the workspace share no memory with each other or with
    inputs; a given output counts as modified in place."""
    return GatedGemm(*_ext().gated_gemm(None, A, sA, B, sB, _act(act), opB, pow2_scales, None, quantize, pow2, want_h,
                                        want_u, split_k, workspace, u, h, q, s, _stream(A)))


def grouped_gated_gemm_fp8_blockscaled(offsets, A, sA, B, sB, act: str = "silu", opB: int = 0,
                                       max_group_rows: Optional[int] = None, pow2_scales: bool = False,
                                       quantize: bool = False, pow2: bool = False, want_h: bool = True,
                                       want_u: bool = True, u=None, h=None, q=None, s=None) -> GatedGemm:
    """The same for the experts of a mixture: offsets int32 [G+1] on the device, B [G][K][2H] or [G][2H][K],
    sB [G][...], as in grouped_gemm_fp8_blockscaled.  Rows past the last expert's are not written."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a tensor")
    return GatedGemm(*_ext().gated_gemm(offsets, A, sA, B, sB, _act(act), opB, pow2_scales, max_group_rows, quantize, pow2,
                                        want_h, want_u, False, None, u, h, q, s, _stream(A)))


def gated_gemm_backward_fp8_blockscaled(A, sA, B, sB, u, act: str = "silu", opB: int = 1, pow2_scales: bool = False,
                                        quantize: bool = False, pow2: bool = False, want_h: bool = True,
                                        want_du: bool = True, split_k: bool = True, workspace=None, du=None, h=None,
                                        q=None, s=None) -> GatedGemmGrad:
    """Gradient of h = act(u[:, :H]) * u[:, H:] and of the down projection that reads it, in one GEMM: dh = A B
    with A the codes of the gradient of the projection's output [M][K] and B its weights, [H][K] as the
    forward stored them (OP_T) or [K][H] (OP_N).  Returns du bf16 [M][2H] (du may be u itself, which it
    replaces; nothing else that is written shares memory with another argument; a given output counts as
    modified in place), h bf16 [M][H] for the weights' gradient unless want_h is False (from the u given, in BF16;
    the forward's h is from FP32 products, so that the two lie apart by u's rounding), and with quantize
    (q uint8 [M][2H], s float32 [2H/128][M]) = quantize_1x128(du, pow2); want_du=False then leaves du out."""
    return GatedGemmGrad(*_ext().gated_gemm_backward(None, A, sA, B, sB, _act(act), opB, pow2_scales, None, u, quantize, pow2,
                                                     want_h, want_du, split_k, workspace, du, h, q, s, _stream(A)))


def grouped_gated_gemm_backward_fp8_blockscaled(offsets, A, sA, B, sB, u, act: str = "silu", opB: int = 1,
                                                max_group_rows: Optional[int] = None, pow2_scales: bool = False,
                                                quantize: bool = False, pow2: bool = False, want_h: bool = True,
                                                want_du: bool = True, du=None, h=None, q=None, s=None) -> GatedGemmGrad:
    """The same for the experts of a mixture (see grouped_gated_gemm_fp8_blockscaled)."""
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a tensor")
    return GatedGemmGrad(*_ext().gated_gemm_backward(offsets, A, sA, B, sB, _act(act), opB, pow2_scales, max_group_rows, u,
                                                     quantize, pow2, want_h, want_du, False, None, du, h, q, s, _stream(A)))


# --------------------------------------------------------------------------
# AdamW
# --------------------------------------------------------------------------
class _Tensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp),
                ("copy", _vp), ("rows", _i64), ("cols", _i64), ("ldp", _i64), ("ldg", _i64), ("ldc", _i64),
                ("decay", _f32), ("flags", _u32), ("index", _u32), ("reserved", _u32)]


def _order(t: torch.Tensor):
    """Dimensions of more than one element, outermost in memory first."""
    return sorted((d for d in range(t.dim()) if t.shape[d] != 1), key=lambda d: -t.stride(d))


def _rows(t: torch.Tensor, order):
    """(rows, cols, pitch) of t's elements in that order of its dimensions, None if they are not evenly spaced rows."""
    merged = []  # innermost first: (stride, size)
    for d in reversed(order):
        st, n = t.stride(d), t.shape[d]
        if merged and st == merged[-1][0] * merged[-1][1]:
            merged[-1] = (merged[-1][0], merged[-1][1] * n)
        else:
            merged.append((st, n))
    if not merged or merged[0][0] != 1:
        merged.insert(0, (1, 1))
    if len(merged) == 1:
        return 1, merged[0][1], merged[0][1]
    (_, cols), (ld, rows) = merged[0], merged[1]
    return (rows, cols, ld) if len(merged) == 2 and ld >= cols else None


def _same_rows(spans):
    """(rows, cols, pitches) that describe every tensor, None if their rows end at different places."""
    rows, cols = next(((r, c) for r, c, _ in spans if r > 1), spans[0][:2])
    pitches = []
    for r, c, ld in spans:
        if r == 1 and rows > 1:  # dense: rows of any length that divides it
            ld = cols
        elif (r, c) != (rows, cols):
            return None
        pitches.append(ld)
    return rows, cols, pitches


def _per_tensor(ts, n: int, what: str):
    ts = list(ts)
    if len(ts) != n:
        raise ValueError(f"{n} parameters, {len(ts)} {what}")
    for i, t in enumerate(ts):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what} {i} must be a tensor")
    return ts


class AdamWState:
    """Parameters (bf16 or float32) with their AdamW moments.

    ms, vs: the moments, one contiguous tensor of as many elements as the
    parameter for each, in the parameter's order in memory; all of one type:
    float32, bfloat16, or uint8 E4M3 codes (of m and of sqrt(v)) with
    m_scales, v_scales, float32 vectors of one scale for 128 elements.  None:
    zeros of ``dtype`` (float32, bfloat16 or torch.float8_e4m3fn).  They are
    what a checkpoint has to hold, with the number of steps.
    copies: bf16 tensors that receive the new parameters (for FP32 parameters
    whose products run in BF16 or are quantized from it).
    decay: weight decay, one number or one for each parameter."""

    def __init__(self, params: Sequence[torch.Tensor], ms=None, vs=None, m_scales=None, v_scales=None, copies=None,
                 decay=0.0, dtype=torch.float32):
        self.params = list(params)
        n = len(self.params)
        self.params = _per_tensor(self.params, n, "parameter")
        for i, p in enumerate(self.params):
            _is_f32(p, f"parameter {i}")
            if p.device != self.params[0].device:
                raise ValueError(f"parameter {i} is on {p.device}, the first one on {self.params[0].device}")
            if _overlaps(p):
                raise ValueError(f"elements of parameter {i} share memory")
        if (ms is None) != (vs is None):
            raise ValueError("ms and vs go together")
        if ms is None:
            if dtype not in _STATES:
                raise TypeError(f"moments must be float32, bfloat16 or float8_e4m3fn, got {dtype}")
            if m_scales is not None or v_scales is not None:
                raise ValueError("scales without moments")
            codes = dtype == torch.float8_e4m3fn
            stored = torch.uint8 if codes else dtype
            ms, vs = ([torch.zeros(p.numel(), dtype=stored, device=p.device) for p in self.params] for _ in "mv")
            if codes:
                m_scales, v_scales = ([torch.ones(-(-p.numel() // 128), device=p.device) for p in self.params] for _ in "mv")
        self.ms, self.vs = _per_tensor(ms, n, "first moments"), _per_tensor(vs, n, "second moments")
        kinds = {t.dtype for t in self.ms + self.vs} or {dtype if dtype != torch.float8_e4m3fn else torch.uint8}
        if len(kinds) != 1 or not kinds <= {torch.float32, torch.bfloat16, torch.uint8}:
            raise TypeError(f"moments must all be float32, bfloat16 or uint8 codes, got {sorted(map(str, kinds))}")
        codes = kinds == {torch.uint8}
        self.state = 2 if codes else _STATES[kinds.pop()]
        if codes != (m_scales is not None) or codes != (v_scales is not None):
            raise ValueError("m_scales and v_scales go with codes" if codes else "scales without codes")
        self.m_scales = _per_tensor(m_scales, n, "scales") if codes else [None] * n
        self.v_scales = _per_tensor(v_scales, n, "scales") if codes else [None] * n
        self.copies = [None] * n if copies is None else _per_tensor(copies, n, "copies")
        try:
            self.decay = [float(decay)] * n
        except TypeError:
            self.decay = [float(d) for d in decay]
        if len(self.decay) != n:
            raise ValueError(f"{n} parameters, {len(self.decay)} decays")
        self._check()
        for i, c in enumerate(self.copies):
            if c is not None and _overlaps(c):
                raise ValueError(f"copy {i} must have memory for every element")

    def _check(self):
        """That the tensors still fit each other: sizes, types, devices (ValueError or TypeError)."""
        _ext().adamw_check(self.params, self.ms, self.vs, self.m_scales, self.v_scales, self.copies, self.state)


def _entries(state: AdamWState, grads):
    """The table entries of a state and its gradients; empty tensors have none."""
    state._check()
    entries = []
    for i, (p, g) in enumerate(zip(state.params, grads)):
        if g.shape != p.shape:
            raise ValueError(f"gradient {i} has shape {tuple(g.shape)}, its parameter {tuple(p.shape)}")
        flags = (_PARAM_F32 if _is_f32(p, f"parameter {i}") else 0) | (_GRAD_F32 if _is_f32(g, f"gradient {i}") else 0)
        if p.numel() == 0:
            continue
        c = state.copies[i]
        if p.is_contiguous() and g.is_contiguous() and (c is None or c.is_contiguous()):
            same = 1, p.numel(), (p.numel(),) * 3
        else:
            order = _order(p)
            spans = [_rows(t, order) for t in (p, g, c) if t is not None]
            same = _same_rows(spans) if None not in spans else None
        if same is None:
            raise ValueError(f"parameter {i}, its gradient and its copy must lie in memory in the same order, in rows")
        rows, cols, ld = same
        ptr = [t.data_ptr() if t is not None else None for t in (state.m_scales[i], state.v_scales[i], c)]
        entries.append(_Tensor(p.data_ptr(), g.data_ptr(), state.ms[i].data_ptr(), state.vs[i].data_ptr(), *ptr, rows, cols,
                               ld[0], ld[1], ld[2] if c is not None else cols, state.decay[i], flags, i, 0))
    return entries


def _shared(array, n: int, state: int):
    """What two tensors of the entries a step must not take together (see train_binding.cpp), None without such."""
    got = _ext().adamw_shared(ctypes.addressof(array), n, state)
    if got is None:
        return None
    i, a, j, b = got
    return f"the {a} of parameter {array[i].index} and the {b} of parameter {array[j].index}"


def _hold(state: AdamWState, grads):
    """The tensors of a table and the memory that it names, which it keeps."""
    return _ext().adamw_hold(state.params, grads, state.ms, state.vs, state.m_scales, state.v_scales, state.copies)


class AdamWTable:
    """An AdamWState and its gradients laid out on the device for adamw_step.
    It names the tensors' memory and holds the tensors and that memory: a
    training loop that keeps its gradient buffers builds it once (and before a
    graph is captured), one whose gradients are new tensors every step builds
    one a step.  A step is refused once a tensor has other memory than the table
    names (p.data replaced, a storage resized); a captured one does not look.
    A parameter's gradient and copy lie in memory in the order of its dimensions
    (any row pitch each); tensors that a step writes share no memory with any
    other.  The state's tensors are checked anew for every table, since a
    parameter's memory may have changed with its module."""

    def __init__(self, state: AdamWState, grads: Sequence[torch.Tensor]):
        if not isinstance(state, AdamWState):
            raise TypeError("state must be an AdamWState")
        self.state, self.grads = state, _per_tensor(grads, len(state.params), "gradients")
        self.device = state.params[0].device if state.params else torch.device("cuda", torch.cuda.current_device())
        here = not state.params or _stream(state.params[0]) is not None
        for t in (*state.params, *self.grads):
            if t.device != self.device or not here:
                raise ValueError(f"expected tensors on the current GPU, got {t.device}")
        entries = _entries(state, self.grads)
        self.kind = state.state  # the table's layout, whatever becomes of the state
        self.held = _hold(state, self.grads)
        L = _fb.lib()
        self.n = len(entries)
        array = (_Tensor * max(self.n, 1))(*entries)
        shared = _shared(array, self.n, self.kind)
        if shared is not None:
            raise ValueError(f"{shared} share memory that the step would write")
        nbytes = L.fp8blk_adamw_table_bytes(self.n)
        host = torch.empty(nbytes // 8, dtype=torch.int64)
        chunks = _i64(0)
        _fb._check(L.fp8blk_adamw_table_build(ctypes.cast(array, _vp), self.n, self.kind, host.data_ptr(), nbytes,
                                              ctypes.cast(ctypes.pointer(chunks), _vp)), "adamw_table")
        self.chunks = chunks.value
        self.device_table = host.to(self.device)
        self._stream = torch._C._cuda_getCurrentRawStream(self.device.index)


def adamw_table(state: AdamWState, grads) -> AdamWTable:
    """The device table of a state and its gradients (bf16 or float32, one for each parameter)."""
    return AdamWTable(state, grads)


def adamw_step(table: AdamWTable, lr, step, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8,
               norm: Optional[torch.Tensor] = None, max_norm: Optional[float] = None, clip_eps: float = 1e-6,
               seed=None) -> None:
    """One AdamW step on every parameter of the table, in place; step counts
    from 1.  norm (a float32 scalar on the device, as grad_norm returns it)
    with max_norm: gradients are scaled by min(1, max_norm / (norm + clip_eps))
    as they are read, and stay as they are.  seed: round BF16 and E4M3 values at
    random by this integer, another one every step (None: to nearest).  lr, step
    and seed may be one-element tensors on the device (float32, int64, int64),
    which a captured step reads anew at every replay; the graph reads the table
    too, which has to live as long as it is replayed.  Parameters, copies and
    moments count as modified in place: a graph that still needs the old values
    refuses its backward (a replay does not count)."""
    if not isinstance(table, AdamWTable):
        raise TypeError("table must be an AdamWTable")
    t = table.device_table
    stream = _stream(t)
    if stream is not None and stream != table._stream:  # the table's memory must outlive this stream's work too
        t.record_stream(torch.cuda.current_stream())
    _ext().adamw_step(t, table.n, table.chunks, table.kind, lr, step, beta1, beta2, eps, norm, max_norm, clip_eps,
                      seed, table.held, stream)
