"""The operators around the FP8 GEMMs of a mixture-of-experts layer: tokens
into expert order and back, the norms around a block, gradient clipping.

Argument marshalling only, as in the rest of the package; names and argument
meanings follow ``include/libfp8blk_layer.h``.  Matrices are row-major with a
16-byte row pitch (``empty_pitched`` / ``as_pitched``); missing outputs and
workspaces are allocated through torch on the current stream.
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

_IDS_I64 = 0x1
_ROWS_F32, _TOKENS_F32, _DROWS_F32 = 0x1, 0x2, 0x4
_NORM_RES_F32, _NORM_PARAM_F32, _NORM_GATE_ROW = 0x10, 0x20, 0x40
_GRAD_F32, _GRAD_OUT_F32 = 0x1, 0x2
_GRAD_WORKSPACE_BYTES = 16384


def layer_abi_version() -> int:
    return _fb.lib().fp8blk_layer_abi_version()


def _is_f32(t: torch.Tensor, what: str) -> bool:
    if t.dtype == torch.float32:
        return True
    if t.dtype == torch.bfloat16:
        return False
    raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")


def _need(t: torch.Tensor, dtype, what: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")


def _shape(t: torch.Tensor, shape, what: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _dense(t: torch.Tensor, dtype, shape, what: str) -> None:
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _need(t, dtype, what)
        _shape(t, shape, what)
        raise ValueError(f"{what} must be contiguous")


def _current_stream(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The current stream's handle.  The library works on the current device:
    every tensor has to be there.  (The handle is taken directly: a small call
    spends more time building torch.cuda.Stream objects than in its kernel.)"""
    i = first.get_device()
    if i < 0 or i != torch._C._cuda_getDevice():
        raise ValueError(f"expected tensors on the current GPU, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != i:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    return torch._C._cuda_getCurrentRawStream(i)


def _addr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _ld(t: Optional[torch.Tensor]) -> int:
    """Row pitch (elements) of a row-major matrix; 0 without one."""
    if t is None:
        return 0
    rows, cols = t.shape
    ld, step = t.stride()
    if rows == 0 or cols == 0:
        return _fb._pad16(cols, t.element_size())
    if (step != 1 and cols != 1) or (ld < cols and rows != 1):
        raise ValueError(f"expected a row-major matrix of separate rows, got strides {(ld, step)}")
    return ld if ld >= cols else cols


def _mat(t: torch.Tensor, dtype, shape, what: str) -> int:
    """Row pitch of a matrix argument, checked."""
    if t.dtype != dtype or t.shape != shape:
        _need(t, dtype, what)
        _shape(t, shape, what)
    ld, step = t.stride()
    return ld if step == 1 and ld >= shape[1] else _ld(t)


def _out(t: Optional[torch.Tensor], rows: int, cols: int, dtype, like: torch.Tensor, what: str):
    """(t, its pitch): the given output, checked, or a new one beside `like`."""
    if t is not None:
        return t, _mat(t, dtype, (rows, cols), what)
    per = 16 // dtype.itemsize
    if cols % per == 0:
        if like.dtype == dtype and like.shape == (rows, cols) and like.is_contiguous():
            return torch.empty_like(like), cols  # fewer arguments to parse than torch.empty
        return torch.empty(rows, cols, dtype=dtype, device=like.device), cols
    ld = (cols // per + 1) * per
    return torch.empty(rows, ld, dtype=dtype, device=like.device)[:, :cols], ld


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
    if expert_ids.dtype not in (torch.int32, torch.int64) or expert_ids.dim() != 2:
        raise TypeError("expert_ids must be an int32 or int64 matrix [T][K]")
    stream = _current_stream(expert_ids, offsets, row_of, slot_of, workspace)
    T, K = expert_ids.shape
    if (K > 1 and expert_ids.stride(1) != 1) or (T > 1 and expert_ids.stride(0) < K):
        expert_ids = expert_ids.contiguous()
    dev = expert_ids.device
    E = int(num_experts)
    new = torch.empty
    if offsets is None:
        offsets = new(max(E, 0) + 1, dtype=torch.int32, device=dev)
    else:
        _dense(offsets, torch.int32, (E + 1,), "offsets")
    if row_of is None:
        row_of = new(T, K, dtype=torch.int32, device=dev)
    else:
        _dense(row_of, torch.int32, (T, K), "row_of")
    if slot_of is None:
        slot_of = new(T * K, dtype=torch.int32, device=dev)
    else:
        _dense(slot_of, torch.int32, (T * K,), "slot_of")
    L = _fb.lib()
    need = L.fp8blk_moe_sort_workspace_bytes(T, K, E)
    if need and workspace is None:
        workspace = new(need // 4, dtype=torch.int32, device=dev)
    _fb._check(L.fp8blk_moe_sort(_addr(expert_ids), T, K, expert_ids.stride(0) if T > 1 else K, E,
                                 _addr(offsets), _addr(row_of), _addr(slot_of), _addr(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                 _IDS_I64 if expert_ids.dtype == torch.int64 else 0, stream), "moe_sort")
    return offsets, row_of, slot_of


def _pairs(row_of: torch.Tensor, T: int):
    if row_of.dim() != 2 or row_of.shape[0] != T:
        raise ValueError(f"row_of must be [T][K] with T = {T}, got {tuple(row_of.shape)}")
    _dense(row_of, torch.int32, row_of.shape, "row_of")
    return row_of.shape[1]


def moe_dispatch(x: torch.Tensor, row_of: torch.Tensor, out=None) -> torch.Tensor:
    """x [T][C] bf16 into expert order: out[row_of[t][k]] = x[t], zeros in the
    rows of dropped pairs.  Returns out bf16 [T*K][C]."""
    _need(x, torch.bfloat16, "x")
    stream = _current_stream(x, row_of, out)
    T, C = x.shape
    K = _pairs(row_of, T)
    out, ldo = _out(out, T * K, C, torch.bfloat16, x, "out")
    _fb._check(_fb.lib().fp8blk_moe_dispatch(_addr(x), T, C, _ld(x), K, _addr(row_of), _addr(out), ldo, stream),
               "moe_dispatch")
    return out


def moe_dispatch_fp8(q: torch.Tensor, s: torch.Tensor, row_of: torch.Tensor, slot_of: torch.Tensor, qr=None, sr=None):
    """Codes q uint8 [T][C] and 1x128 scales s [ceil(C/128)][T] into expert
    order, as the grouped GEMM takes them: returns (qr uint8 [T*K][C],
    sr float32 [ceil(C/128)][T*K])."""
    _need(q, torch.uint8, "q")
    stream = _current_stream(q, s, row_of, slot_of, qr, sr)
    T, C = q.shape
    K = _pairs(row_of, T)
    G = (C + 127) // 128
    _dense(s, torch.float32, (G, T), "s")
    _dense(slot_of, torch.int32, (T * K,), "slot_of")
    qr, ldqr = _out(qr, T * K, C, torch.uint8, q, "qr")
    if sr is None:
        sr = torch.empty(G, T * K, dtype=torch.float32, device=q.device)
    else:
        _dense(sr, torch.float32, (G, T * K), "sr")
    _fb._check(_fb.lib().fp8blk_moe_dispatch_fp8(_addr(q), T, C, _ld(q), _addr(s), K, _addr(row_of),
                                                 _addr(slot_of), _addr(qr), ldqr, _addr(sr),
                                                 stream), "moe_dispatch_fp8")
    return qr, sr


def moe_combine(rows: torch.Tensor, row_of: torch.Tensor, weights: Optional[torch.Tensor] = None,
                out_dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """Expert rows [T*K][C] (bf16 or float32) back to their tokens: out[t] =
    sum over k of weights[t][k] * rows[row_of[t][k]] over the pairs not dropped
    (weights None: all one, the gradient of moe_dispatch).  out [T][C] in
    out_dtype (bfloat16 or float32)."""
    T = row_of.shape[0]
    K = _pairs(row_of, T)
    stream = _current_stream(rows, row_of, weights, out)
    C = rows.shape[1]
    _shape(rows, (T * K, C), "rows")
    if weights is not None:
        _dense(weights, torch.float32, (T, K), "weights")
    flags = _ROWS_F32 if _is_f32(rows, "rows") else 0
    out, ldo = _out(out, T, C, out_dtype if out is None else out.dtype, rows, "out")
    if _is_f32(out, "out"):
        flags |= _TOKENS_F32
    _fb._check(_fb.lib().fp8blk_moe_combine(_addr(rows), T, K, C, _ld(rows), _addr(row_of),
                                            _addr(weights), _addr(out), ldo, flags, stream),
               "moe_combine")
    return out


def moe_combine_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, weights: torch.Tensor,
                         drows_dtype=None, drows=None, dweights=None):
    """Gradient of moe_combine(rows, row_of, weights) for dy [T][C] (bf16 or
    float32): returns (drows [T*K][C] in drows_dtype, rows' type by default,
    zeros in the rows of dropped pairs; dweights float32 [T][K])."""
    T, C = dy.shape
    K = _pairs(row_of, T)
    stream = _current_stream(dy, rows, row_of, weights, drows, dweights)
    _shape(rows, (T * K, C), "rows")
    _dense(weights, torch.float32, (T, K), "weights")
    flags = (_TOKENS_F32 if _is_f32(dy, "dy") else 0) | (_ROWS_F32 if _is_f32(rows, "rows") else 0)
    dt = drows.dtype if drows is not None else rows.dtype if drows_dtype is None else drows_dtype
    drows, lddr = _out(drows, T * K, C, dt, rows, "drows")
    if _is_f32(drows, "drows"):
        flags |= _DROWS_F32
    if dweights is None:
        dweights = torch.empty(T, K, dtype=torch.float32, device=dy.device)
    else:
        _dense(dweights, torch.float32, (T, K), "dweights")
    _fb._check(_fb.lib().fp8blk_moe_combine_backward(
        _addr(dy), _ld(dy), _addr(rows), _ld(rows), T, K, C, _addr(row_of), _addr(weights),
        _addr(drows), lddr, _addr(dweights), flags, stream), "moe_combine_backward")
    return drows, dweights


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


def _params(C: int, w_pre, w_post, gate) -> int:
    """The flag of the parameters' common type, checked."""
    flag = None
    for t in (w_pre, w_post, gate):
        if t is None:
            continue
        if t.shape != (C,) or not t.is_contiguous():
            raise ValueError(f"w_pre, w_post and a gate per channel must be contiguous vectors of {C}, got {tuple(t.shape)}")
        f = _NORM_PARAM_F32 if _is_f32(t, "w_pre, w_post and a gate per channel") else 0
        if flag is not None and f != flag:
            raise TypeError("w_pre, w_post and a gate per channel must have one type")
        flag = f
    return flag or 0


def _gate(gate, M: int, C: int):
    """(gate per channel or None, flag, pitch)."""
    if gate is None or gate.dim() == 1:
        return gate, 0, 0
    return None, _NORM_GATE_ROW, _mat(gate, torch.bfloat16, (M, C), "a gate per token")


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
    M, C = x.shape
    stream = _current_stream(x, w_pre, f, w_post, gate, x_out, n, q, s)
    gate_c, flags, ldg = _gate(gate, M, C)
    flags |= _params(C, w_pre, w_post, gate_c)
    if _is_f32(x, "x"):
        flags |= _NORM_RES_F32
    dev = x.device
    if (w_post is not None or gate is not None) and f is None:
        raise ValueError("w_post and gate need f")
    if f is None and w_pre is None:
        raise ValueError("nothing to do: neither f nor w_pre is given")
    if w_pre is None and (quantize or n is not None):
        raise ValueError("n and its quantization need w_pre")
    rstd_post = rstd_pre = None
    ldf = ldxo = ldn = ldq = 0
    if f is not None:
        ldf = _mat(f, torch.bfloat16, (M, C), "f")
        x_out, ldxo = _out(x_out, M, C, x.dtype, x, "x_out")
        if w_post is not None:
            rstd_post = torch.empty(M, dtype=torch.float32, device=dev)
    elif x_out is not None:
        raise ValueError("x_out without f: x would not change")
    if w_pre is not None:
        rstd_pre = torch.empty(M, dtype=torch.float32, device=dev)
        if n is not None or want_n or not quantize:
            n, ldn = _out(n, M, C, torch.bfloat16, x if f is None else f, "n")
        if quantize:
            q, ldq = _out(q, M, C, torch.uint8, x, "q")
            if s is None:
                s = torch.empty((C + 127) // 128, M, dtype=torch.float32, device=dev)
            else:
                _dense(s, torch.float32, ((C + 127) // 128, M), "s")
            if pow2:
                flags |= _fb.SCALE_POW2
        else:
            q = s = None
    _fb._check(_fb.lib().fp8blk_residual_norm(
        M, C, x.data_ptr(), _ld(x), _addr(f), ldf, _addr(w_post), _addr(gate), ldg, alpha, _addr(w_pre), eps,
        _addr(x_out), ldxo, _addr(n), ldn, _addr(q), ldq, _addr(s), _addr(rstd_post), _addr(rstd_pre), flags, stream),
        "residual_norm")
    return ResidualNorm(x if f is None else x_out, n, q, s, rstd_post, rstd_pre)


def residual_norm_backward(x_out: torch.Tensor, dx_out=None, dn=None, rstd_pre=None, w_pre=None, f=None,
                           rstd_post=None, w_post=None, gate=None, alpha: float = 1.0, dx=None, df=None,
                           workspace=None) -> ResidualNormGrad:
    """Gradient of residual_norm: x_out, rstd_pre and rstd_post from the
    forward, dx_out the gradient into its x (or None), dn the one into n.
    Without w_pre the gradient of x is dx_out itself, which is returned."""
    M, C = x_out.shape
    stream = _current_stream(x_out, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post, gate, dx, df, workspace)
    gate_c, flags, ldg = _gate(gate, M, C)
    flags |= _params(C, w_pre, w_post, gate_c)
    if _is_f32(x_out, "x_out"):
        flags |= _NORM_RES_F32
    dev = x_out.device
    if dx_out is None and dn is None:
        raise ValueError("neither dx_out nor dn is given")
    if (w_post is not None or gate is not None) and f is None:
        raise ValueError("w_post and gate need f")
    mat = (M, C)
    lddxo = lddn = lddx = ldf = lddf = lddg = 0
    if dx_out is not None:
        lddxo = _mat(dx_out, x_out.dtype, mat, "dx_out")
    if (dn is None) != (w_pre is None) or (rstd_pre is None) != (w_pre is None):
        raise ValueError("dn, rstd_pre and w_pre go together")
    if (rstd_post is None) != (w_post is None):
        raise ValueError("rstd_post and w_post go together")
    dw_pre = dw_post = dgate = None
    new = torch.empty
    if w_pre is not None:
        lddn = _mat(dn, torch.bfloat16, mat, "dn")
        _dense(rstd_pre, torch.float32, (M,), "rstd_pre")
        dw_pre = new(C, dtype=torch.float32, device=dev)
    if w_pre is not None or dx is not None:
        dx, lddx = _out(dx, M, C, x_out.dtype, x_out, "dx")
    if f is not None:
        ldf = _mat(f, torch.bfloat16, mat, "f")
        df, lddf = _out(df, M, C, torch.bfloat16, f, "df")
        if w_post is not None:
            _dense(rstd_post, torch.float32, (M,), "rstd_post")
            dw_post = new(C, dtype=torch.float32, device=dev)
        if gate_c is not None:
            dgate = new(C, dtype=torch.float32, device=dev)
        elif gate is not None:
            dgate, lddg = _out(None, M, C, torch.bfloat16, f, "dgate")
    L = _fb.lib()
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
    elif dw_pre is not None or dw_post is not None or (dgate is not None and dgate.dim() == 1):
        ws_bytes = L.fp8blk_residual_norm_backward_workspace_bytes(M, C)
        workspace = new((ws_bytes + 3) // 4, dtype=torch.float32, device=dev)
    if dx is not None or f is not None:
        _fb._check(L.fp8blk_residual_norm_backward(
            M, C, x_out.data_ptr(), _ld(x_out), _addr(dx_out), lddxo, _addr(dn), lddn, _addr(rstd_pre),
            _addr(w_pre), _addr(f), ldf, _addr(rstd_post), _addr(w_post), _addr(gate), ldg, alpha, _addr(dx), lddx,
            _addr(df), lddf, _addr(dw_pre), _addr(dw_post), _addr(dgate), lddg, _addr(workspace), ws_bytes, flags,
            stream), "residual_norm_backward")
    return ResidualNormGrad(dx_out if dx is None else dx, df, dw_pre, dw_post, dgate)


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


class GradTable:
    """A list of gradients (and, where clipped values go elsewhere, their
    outputs) laid out on the device for grad_norm and clip_grad_norm.  It names
    the tensors' memory and holds the tensors: a training loop that keeps its
    gradient buffers builds it once (and before a graph is captured), one whose
    gradients are new tensors every step passes the list instead."""

    def __init__(self, tensors: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None):
        self.tensors = list(tensors)
        self.outs = None if outs is None else list(outs)
        if self.outs is not None and len(self.outs) != len(self.tensors):
            raise ValueError(f"{len(self.tensors)} gradients, {len(self.outs)} outputs")
        if not self.tensors:
            self.device = torch.device("cuda", torch.cuda.current_device())
        else:
            self.device = self.tensors[0].device
            _current_stream(self.tensors[0], *self.tensors, *(self.outs or ()))
        entries = []
        for i, t in enumerate(self.tensors):
            o = t if self.outs is None else self.outs[i]
            if o.shape != t.shape:
                raise ValueError(f"output {i} has shape {tuple(o.shape)}, its gradient {tuple(t.shape)}")
            if _overlaps(t) or (o is not t and _overlaps(o)):
                raise ValueError(f"elements of gradient {i} or of its output share memory")
            flags = (_GRAD_F32 if _is_f32(t, f"gradient {i}") else 0) | (_GRAD_OUT_F32 if _is_f32(o, f"output {i}") else 0)
            _grad_entries(t, o, flags, entries)
        L = _fb.lib()
        self.n = len(entries)
        nbytes = L.fp8blk_grad_table_bytes(self.n)
        host = torch.empty(nbytes // 8, dtype=torch.int64)
        chunks = _i64(0)
        array = (_Grad * max(self.n, 1))(*entries)
        _fb._check(L.fp8blk_grad_table_build(ctypes.cast(array, _vp), self.n, _addr(host), nbytes,
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
    if t.device.index != torch._C._cuda_getDevice():
        raise ValueError(f"expected gradients on the current GPU, got {t.device}")
    stream = torch._C._cuda_getCurrentRawStream(t.device.index)
    if stream != t._stream:  # the table's memory must outlive this stream's work too
        t.device_table.record_stream(torch.cuda.current_stream())
    return t, stream


def _grad_workspace(t: GradTable) -> torch.Tensor:
    return torch.empty(_GRAD_WORKSPACE_BYTES // 8, dtype=torch.float64, device=t.device)


def grad_norm(grads) -> torch.Tensor:
    """Global 2-norm over all gradients (a GradTable or a list of tensors): a
    float32 scalar on the device."""
    t, stream = _table(grads)
    norm = torch.empty((), dtype=torch.float32, device=t.device)
    ws = _grad_workspace(t)
    _fb._check(_fb.lib().fp8blk_grad_norm(_addr(t.device_table), t.n, t.chunks, _addr(norm),
                                          _addr(ws), _GRAD_WORKSPACE_BYTES, stream),
               "grad_norm")
    return norm


def grad_clip(grads, norm: torch.Tensor, max_norm: float, eps: float = 1e-6) -> None:
    """Scale every gradient by min(1, max_norm / (norm + eps)), norm a float32
    scalar on the device (e.g. reduced over ranks): in place, or into the
    table's outputs."""
    t, stream = _table(grads)
    _need(norm, torch.float32, "norm")
    if norm.numel() != 1 or norm.device != t.device:
        raise ValueError("norm must be one value on the gradients' device")
    _fb._check(_fb.lib().fp8blk_grad_clip(_addr(t.device_table), t.n, t.chunks, _addr(norm), max_norm, eps,
                                          stream), "grad_clip")


def clip_grad_norm(grads, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """grad_norm and grad_clip by it; returns the norm before clipping."""
    t, stream = _table(grads)
    norm = torch.empty((), dtype=torch.float32, device=t.device)
    ws = _grad_workspace(t)
    _fb._check(_fb.lib().fp8blk_grad_clip_norm(_addr(t.device_table), t.n, t.chunks, max_norm, eps, _addr(norm),
                                               _addr(ws), _GRAD_WORKSPACE_BYTES, stream),
               "clip_grad_norm")
    return norm
