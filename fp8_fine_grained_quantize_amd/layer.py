"""The operators around the FP8 GEMMs of a mixture-of-experts layer: tokens
into expert order and back, the norms around a block, gradient clipping.

Argument marshalling only, as in the rest of the package, here in C++
(``csrc/layer_binding.cpp``, ``_layer_ext.so``): a small call costs its launch
and little more.  Names and argument meanings follow
``include/libfp8blk_layer.h``.  Matrices are row-major with a 16-byte row pitch
(``empty_pitched`` / ``as_pitched``); missing outputs and workspaces are
allocated through torch on the current stream.  TypeError and ValueError refuse
arguments, Fp8BlkError reports a failed call.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence

import torch

import fp8_fine_grained_quantize_amd as _fb

_i64, _u32, _vp, _sz, _int, _f32 = (ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                                    ctypes.c_float)

SIGNATURES = {
    "fp8blk_layer_abi_version": (_int, []),
    "fp8blk_moe_sort": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _u32, _vp]),
    "fp8blk_moe_sort_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "fp8blk_moe_dispatch": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp]),
    "fp8blk_moe_dispatch_fp8": (_int, [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp]),
    "fp8blk_moe_combine": (_int, [_vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _u32, _vp]),
    "fp8blk_moe_combine_backward": (_int, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _u32,
                                           _vp]),
    "fp8blk_residual_norm": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _f32, _vp, _f32, _vp, _i64, _vp,
                                    _i64, _vp, _i64, _vp, _vp, _vp, _u32, _vp]),
    "fp8blk_residual_norm_backward": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp,
                                             _vp, _vp, _i64, _f32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _sz,
                                             _u32, _vp]),
    "fp8blk_residual_norm_backward_workspace_bytes": (_sz, [_i64, _i64]),
    "fp8blk_grad_table_bytes": (_sz, [_i64]),
    "fp8blk_grad_table_build": (_int, [_vp, _i64, _vp, _sz, _vp]),
    "fp8blk_grad_norm": (_int, [_vp, _i64, _i64, _vp, _vp, _sz, _vp]),
    "fp8blk_grad_clip": (_int, [_vp, _i64, _i64, _vp, _f32, _f32, _vp]),
    "fp8blk_grad_clip_norm": (_int, [_vp, _i64, _i64, _f32, _f32, _vp, _vp, _sz, _vp]),
}
LAYER_SYMBOLS = tuple(SIGNATURES)

_GRAD_F32, _GRAD_OUT_F32 = 0x1, 0x2


def layer_abi_version() -> int:
    return _fb.lib().fp8blk_layer_abi_version()


_EXT = None


def _ext():
    """The binding's C++ part (csrc/layer_binding.cpp): checks, allocates and
    calls the library."""
    global _EXT
    if _EXT is None:
        _fb.lib()
        try:
            from . import _layer_ext
        except ImportError as e:
            raise _fb.Fp8BlkError("_layer_ext.so is missing or was built for another torch: build it with "
                                  f"`python -m fp8_fine_grained_quantize_amd.build` ({e})") from e
        _layer_ext.set_error(_fb.Fp8BlkError)
        _EXT = _layer_ext
    return _EXT


def _stream(first: torch.Tensor):
    """Handle of the current stream; None unless the first tensor is on the
    current GPU (where the library works), which is then refused."""
    try:
        i = first.get_device()
    except AttributeError:  # no tensor: refused by its name
        return None
    return torch._C._cuda_getCurrentRawStream(i) if i >= 0 and i == torch._C._cuda_getDevice() else None


def _is_f32(t: torch.Tensor, what: str) -> bool:
    if t.dtype == torch.float32:
        return True
    if t.dtype == torch.bfloat16:
        return False
    raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")


# --------------------------------------------------------------------------
# tokens by expert
# --------------------------------------------------------------------------
def moe_sort(expert_ids: torch.Tensor, num_experts: int, offsets=None, row_of=None, slot_of=None, workspace=None):
    """Sort the (token, choice) pairs of expert_ids [T][K] (int32 or int64, as
    a top-k returns them) by expert, token order kept inside an expert; an id
    outside [0, num_experts) drops its pair.  Returns (offsets int32 [E+1],
    row_of int32 [T][K], slot_of int32 [T*K]): expert e owns rows
    offsets[e]:offsets[e+1]; row_of holds each pair's row, -1 - row for dropped
    pairs (their rows follow offsets[E]); slot_of holds each row's pair."""
    return _ext().moe_sort(expert_ids, num_experts, offsets, row_of, slot_of, workspace, _stream(expert_ids))


def moe_dispatch(x: torch.Tensor, row_of: torch.Tensor, out=None) -> torch.Tensor:
    """x [T][C] bf16 into expert order: out[row_of[t][k]] = x[t], zeros in the
    rows of dropped pairs.  Returns out bf16 [T*K][C]."""
    return _ext().moe_dispatch(x, row_of, out, _stream(x))


def moe_dispatch_fp8(q: torch.Tensor, s: torch.Tensor, row_of: torch.Tensor, slot_of: torch.Tensor, qr=None, sr=None):
    """Codes q uint8 [T][C] and 1x128 scales s [ceil(C/128)][T] into expert
    order, as the grouped GEMM takes them: returns (qr uint8 [T*K][C],
    sr float32 [ceil(C/128)][T*K])."""
    return _ext().moe_dispatch_fp8(q, s, row_of, slot_of, qr, sr, _stream(q))


def moe_combine(rows: torch.Tensor, row_of: torch.Tensor, weights: Optional[torch.Tensor] = None,
                out_dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """Expert rows [T*K][C] (bf16 or float32) back to their tokens: out[t] =
    sum over k of weights[t][k] * rows[row_of[t][k]] over the pairs not dropped
    (weights None: all one, the gradient of moe_dispatch).  out [T][C] in
    out_dtype (bfloat16 or float32)."""
    return _ext().moe_combine(rows, row_of, weights, out_dtype, out, _stream(rows))


def moe_combine_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, weights: torch.Tensor,
                         drows_dtype=None, drows=None, dweights=None):
    """Gradient of moe_combine(rows, row_of, weights) for dy [T][C] (bf16 or
    float32): returns (drows [T*K][C] in drows_dtype, rows' type by default,
    zeros in the rows of dropped pairs; dweights float32 [T][K])."""
    return _ext().moe_combine_backward(dy, rows, row_of, weights, drows_dtype, drows, dweights, _stream(dy))


# --------------------------------------------------------------------------
# norms around a block
# --------------------------------------------------------------------------
class ResidualNorm(NamedTuple):
    """x: the residual stream after the sum (the given x where there is no f);
    n, (q, s): the normalized rows; rstd_post, rstd_pre: kept for the gradient."""
    x: torch.Tensor
    n: Optional[torch.Tensor]
    q: Optional[torch.Tensor]
    s: Optional[torch.Tensor]
    rstd_post: Optional[torch.Tensor]
    rstd_pre: Optional[torch.Tensor]


class ResidualNormGrad(NamedTuple):
    dx: torch.Tensor
    df: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


def residual_norm(x: torch.Tensor, w_pre=None, f=None, w_post=None, gate=None, alpha: float = 1.0, eps: float = 1e-6,
                  quantize: bool = False, pow2: bool = False, want_n: bool = True, x_out=None, n=None, q=None,
                  s=None) -> ResidualNorm:
    """The end of a block and the start of the next: x' = x + alpha * gate *
    RMSNorm(f; w_post), n = RMSNorm(x'; w_pre), each part only where its
    arguments are given (f without w_post is added as it is).  x [M][C] bf16 or
    float32; f bf16; gate [C], or bf16 [M][C] per token; weights and gate [C]
    bf16 or float32.  quantize: also n's 1x128 E4M3 codes and scales (powers of
    two with pow2), quantized from the FP32 values; want_n=False then leaves n
    out.  x_out may be x."""
    return ResidualNorm(*_ext().residual_norm(x, w_pre, f, w_post, gate, alpha, eps, quantize, pow2, want_n, x_out, n,
                                              q, s, _stream(x)))


def residual_norm_backward(x_out: torch.Tensor, dx_out=None, dn=None, rstd_pre=None, w_pre=None, f=None,
                           rstd_post=None, w_post=None, gate=None, alpha: float = 1.0, dx=None, df=None,
                           workspace=None) -> ResidualNormGrad:
    """Gradient of residual_norm: x_out, rstd_pre and rstd_post from the
    forward, dx_out the gradient into its x (or None), dn the one into n.
    Without w_pre the gradient of x is dx_out itself, which is returned."""
    return ResidualNormGrad(*_ext().residual_norm_backward(x_out, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post,
                                                           gate, alpha, dx, df, workspace, _stream(x_out)))


# --------------------------------------------------------------------------
# gradient norm and clipping
# --------------------------------------------------------------------------
class _Grad(ctypes.Structure):
    _fields_ = [("grad", _vp), ("out", _vp), ("rows", _i64), ("cols", _i64), ("ld", _i64), ("ldo", _i64),
                ("flags", _u32), ("reserved", _u32)]


def _as_rows(shape, stride):
    """(rows, cols, pitch) of elements that form evenly spaced rows, else None."""
    dims = sorted(((st, n) for n, st in zip(shape, stride) if n != 1), reverse=True)
    merged = []
    for st, n in reversed(dims):  # dimensions that continue each other are one
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


def _overlaps(t: torch.Tensor) -> bool:
    """Whether two elements may share memory (expanded tensors, sliding windows)."""
    if t.numel() == 0:
        return False
    reach = 0
    for st, n in sorted((st, n) for n, st in zip(t.shape, t.stride()) if n > 1):
        if st <= reach:
            return True
        reach += (n - 1) * st
    return False


def _row_major(t: torch.Tensor) -> bool:
    st = [st for n, st in zip(t.shape, t.stride()) if n != 1]
    return st == sorted(st, reverse=True)


def _grad_entries(t: torch.Tensor, o: torch.Tensor, flags: int, out: list) -> None:
    """Appends the table entries of one gradient and its output."""
    if t.numel() == 0:
        return
    if t.stride() == o.stride():  # any order of the dimensions, the same in both
        a = b = _as_rows(t.shape, t.stride())
    else:
        a = b = None
        if _row_major(t) and _row_major(o):
            a, b = _as_rows(t.shape, t.stride()), _as_rows(o.shape, o.stride())
        if a and b and a[0] == 1 and b[0] > 1:
            a = (b[0], b[1], b[1])
        elif a and b and b[0] == 1 and a[0] > 1:
            b = (a[0], a[1], a[1])
    if a and b and a[:2] == b[:2]:
        out.append(_Grad(t.data_ptr(), o.data_ptr(), a[0], a[1], a[2], b[2], flags, 0))
        return
    for i in range(t.shape[0]):  # piece by piece along the first dimension
        _grad_entries(t[i], o[i], flags, out)


def _shared(array, first):
    """The first two tensors of a list of entries that clipping must not take
    together (see layer_binding.cpp), None without such; first: where each
    tensor's entries start, and their number."""
    starts = (_i64 * len(first))(*first)
    return _ext().grad_shared(ctypes.addressof(array), ctypes.addressof(starts), len(first) - 1)


class GradTable:
    """A list of gradients (and, where clipped values go elsewhere, their
    outputs) laid out on the device for grad_norm and clip_grad_norm.  It names
    the tensors' memory and holds the tensors: a training loop that keeps its
    gradient buffers builds it once (and before a graph is captured), one whose
    gradients are new tensors every step passes the list instead.  Gradients
    may share memory (a tied weight listed twice) for grad_norm, which counts
    them each time; clipping refuses outputs that share memory with another
    tensor of the list, or with their own gradient other than in place."""

    def __init__(self, tensors: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None):
        self.tensors = list(tensors)
        self.outs = None if outs is None else list(outs)
        for what, ts in (("gradient", self.tensors), ("output", self.outs or ())):
            for i, t in enumerate(ts):
                if not isinstance(t, torch.Tensor):
                    raise TypeError(f"{what} {i} must be a tensor")
        if self.outs is not None and len(self.outs) != len(self.tensors):
            raise ValueError(f"{len(self.tensors)} gradients, {len(self.outs)} outputs")
        if not self.tensors:
            self.device = torch.device("cuda", torch.cuda.current_device())
        else:
            self.device = self.tensors[0].device
            for t in (*self.tensors, *(self.outs or ())):
                if t.device != self.device or _stream(t) is None:
                    raise ValueError(f"expected tensors on the current GPU, got {t.device}")
        entries, first = [], [0]
        for i, t in enumerate(self.tensors):
            o = t if self.outs is None else self.outs[i]
            if o.shape != t.shape:
                raise ValueError(f"output {i} has shape {tuple(o.shape)}, its gradient {tuple(t.shape)}")
            if _overlaps(t) or (o is not t and _overlaps(o)):
                raise ValueError(f"elements of gradient {i} or of its output share memory")
            flags = (_GRAD_F32 if _is_f32(t, f"gradient {i}") else 0) | (_GRAD_OUT_F32 if _is_f32(o, f"output {i}") else 0)
            _grad_entries(t, o, flags, entries)
            first.append(len(entries))
        L = _fb.lib()
        self.n = len(entries)
        nbytes = L.fp8blk_grad_table_bytes(self.n)
        host = torch.empty(nbytes // 8, dtype=torch.int64)
        chunks = _i64(0)
        array = (_Grad * max(self.n, 1))(*entries)
        self.shared = _shared(array, first)
        _fb._check(L.fp8blk_grad_table_build(ctypes.cast(array, _vp), self.n, host.data_ptr(), nbytes,
                                             ctypes.cast(ctypes.pointer(chunks), _vp)), "grad_table")
        self.chunks = chunks.value
        self.device_table = host.to(self.device)
        self._stream = torch._C._cuda_getCurrentRawStream(self.device.index)


def grad_table(tensors, outs=None) -> GradTable:
    """The device table of a list of gradients (bf16 or float32); outs: where
    clipped values go (same shapes, either type; None: in place)."""
    return GradTable(tensors, outs)


def _table(grads):
    """(table, current stream) of a GradTable or a list of tensors."""
    t = grads if isinstance(grads, GradTable) else GradTable(grads)
    stream = _stream(t.device_table)
    if stream is not None and stream != t._stream:  # the table's memory must outlive this stream's work too
        t.device_table.record_stream(torch.cuda.current_stream())
    return t, stream


def _clippable(grads):
    """_table of gradients that can be clipped together."""
    t, stream = _table(grads)
    if t.shared is not None:
        raise ValueError("gradients {} and {}, or their outputs, share memory that clipping would write".format(*t.shared))
    return t, stream


def grad_norm(grads) -> torch.Tensor:
    """Global 2-norm over all gradients (a GradTable or a list of tensors): a
    float32 scalar on the device."""
    t, stream = _table(grads)
    return _ext().grad_norm(t.device_table, t.n, t.chunks, stream)


def grad_clip(grads, norm: torch.Tensor, max_norm: float, eps: float = 1e-6) -> None:
    """Scale every gradient by min(1, max_norm / (norm + eps)), norm a float32
    scalar on the device (e.g. reduced over ranks): in place, or into the
    table's outputs."""
    t, stream = _clippable(grads)
    _ext().grad_clip(t.device_table, t.n, t.chunks, norm, max_norm, eps, stream)


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """grad_norm and grad_clip by it; returns the norm before clipping."""
    t, stream = _clippable(grads)
    return _ext().clip_grad_norm(t.device_table, t.n, t.chunks, max_norm, eps, stream)
