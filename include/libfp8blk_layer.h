/*
 * libfp8blk — the operators around the FP8 GEMMs of a mixture-of-experts
 * layer, for AMD Instinct MI355X (gfx950):
 *
 *   tokens into expert order and back, with the router's weights, and the
 *   gradients (the grouped GEMMs of libfp8blk.h work on rows ordered by
 *   expert; the pages route each token to 8 of 256 experts [p5¶3] and quantize
 *   MoE activations before they are dispatched [p2¶4]);
 *   the norm after a block with its gate and residual scale, the residual sum
 *   and the norm before the next block, optionally quantized on store to the
 *   1x128 E4M3 tiles that the next FP8 GEMM reads [p1¶3, p2¶4], and the
 *   gradients;
 *   the global norm over many gradient tensors, and clipping by it.
 *
 * Citations [pN¶k] as in libfp8blk.h.  Status codes, streams, ownership and
 * the host-side validation of arguments are those of libfp8blk.h: device
 * pointers, everything asynchronous on `stream`, nothing allocated, filled or
 * copied, an invalid call returns FP8BLK_ERR_INVALID_ARG and touches nothing,
 * sizes of zero are valid.  Matrix pointers are 16-byte aligned and row
 * pitches multiples of 16 bytes; unlike the GEMMs, these operators neither
 * read nor write the padding between a row's length and its pitch.
 * Results do not depend on the run: no floating-point sum is formed by atomics
 * (the sort counts pairs with them, in whole numbers).
 */
#ifndef LIBFP8BLK_LAYER_H
#define LIBFP8BLK_LAYER_H

#include "libfp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ABI version of this header: 1. */
int fp8blk_layer_abi_version(void);

/* ------------------------------------------------------------------------
 * Tokens by expert.  T tokens, K expert choices ("pairs") each, E experts;
 * pair p = t*K + k.  T*K at most 2^31 - 1 - 2^20, C at most 2^40, E at most
 * 960, and a launch has fewer than 2^32 lanes (FP8BLK_ERR_UNSUPPORTED
 * otherwise): a token's row takes one for 8 channels (4 where either matrix
 * is FP32; 16 codes) in workgroups of 64 to 256, for codes always 256, of
 * which the scales take more for every 256 rows and 8 groups; in the gradient
 * of the combine every token has one workgroup, of 64 to 512 lanes whatever C.
 * ------------------------------------------------------------------------ */

/* Flag: the expert ids are int64 (as a top-k over router scores returns
 * them); int32 without it. */
#define FP8BLK_MOE_IDS_I64 0x1u
/* Flags of the combine and its gradient: element types, BF16 without them. */
#define FP8BLK_MOE_ROWS_F32 0x1u   /* the expert rows */
#define FP8BLK_MOE_TOKENS_F32 0x2u /* the token matrix (y, dy) */
#define FP8BLK_MOE_DROWS_F32 0x4u  /* the gradient of the expert rows */

/*
 * Sorts the pairs by expert, keeping token order inside an expert.
 *   expert_ids  [T][K], pitch ld >= K elements; aligned to their own size.
 *               An id outside [0, E) drops the pair (a masked token, a full
 *               expert): no expert owns it.
 *   offsets     int32 [E+1], what the grouped entry points take: expert e
 *               owns rows [offsets[e], offsets[e+1]); offsets[E] is the
 *               number of pairs not dropped.
 *   row_of      int32 [T][K], dense: the row of pair (t, k) in expert order.
 *               Dropped pairs take the rows from offsets[E] on, in pair
 *               order, and are marked by storing -1 - row.
 *   slot_of     int32 [T*K]: the pair of every row, -1 - pair for the rows of
 *               dropped pairs.
 *   workspace   fp8blk_moe_sort_workspace_bytes(T, K, E) bytes, 4-byte
 *               aligned (may be NULL where that is 0).
 * With T*K = 0 the offsets are still written (all zero).
 */
fp8blk_status_t fp8blk_moe_sort(const void* expert_ids, int64_t T, int64_t K, int64_t ld, int64_t E,
                                int32_t* offsets, int32_t* row_of, int32_t* slot_of, void* workspace,
                                size_t workspace_bytes, uint32_t flags, void* stream);
size_t fp8blk_moe_sort_workspace_bytes(int64_t T, int64_t K, int64_t E);

/*
 * Token rows into expert order: out[row_of[t][k]] = x[t] for every pair not
 * dropped, zeros in the rows of dropped pairs (so that all T*K rows are
 * defined).  Also the gradient of an unweighted combine.
 *   x    [T][C] BF16, pitch ldx >= C;  out [T*K][C] BF16, pitch ldo >= C.
 *   row_of  as fp8blk_moe_sort writes it: its rows are a permutation of
 *           [0, T*K).  (A row outside that range is skipped, not written.)
 */
fp8blk_status_t fp8blk_moe_dispatch(const uint16_t* x, int64_t T, int64_t C, int64_t ldx, int64_t K,
                                    const int32_t* row_of, uint16_t* out, int64_t ldo, void* stream);

/*
 * The same for activations already quantized, by fp8blk_quantize_1x128 or by
 * fp8blk_residual_norm: E4M3 codes and their 1x128 scales.
 *   q   [T][C] codes, pitch ldq;  s  [ceil(C/128)][T] FP32.
 *   qr  [T*K][C] codes, pitch ldqr;  sr [ceil(C/128)][T*K] FP32: what the
 *   grouped GEMM takes as A and sA.  Rows of dropped pairs get code 0 and
 *   scale 1, as the quantizers write a tile of zeros.
 */
fp8blk_status_t fp8blk_moe_dispatch_fp8(const uint8_t* q, int64_t T, int64_t C, int64_t ldq, const float* s,
                                        int64_t K, const int32_t* row_of, const int32_t* slot_of, uint8_t* qr,
                                        int64_t ldqr, float* sr, void* stream);

/*
 * Expert rows back to their tokens:
 *   y[t] = sum over k ascending, not dropped, of weights[t][k] * rows[row_of[t][k]],
 * summed in FP32 and rounded once.  weights NULL: all one (the gradient of
 * dispatch).  A token whose pairs are all dropped gets zeros; rows of dropped
 * pairs are not read.
 *   rows [T*K][C] BF16 (FP32 with FP8BLK_MOE_ROWS_F32), pitch ldr >= C.
 *   weights FP32 [T][K], dense.
 *   y    [T][C] BF16 (FP32 with FP8BLK_MOE_TOKENS_F32), pitch ldy >= C.
 */
fp8blk_status_t fp8blk_moe_combine(const void* rows, int64_t T, int64_t K, int64_t C, int64_t ldr,
                                   const int32_t* row_of, const float* weights, void* y, int64_t ldy,
                                   uint32_t flags, void* stream);

/*
 * Gradient of the weighted combine:
 *   drows[row_of[t][k]] = weights[t][k] * dy[t]        (zeros for dropped pairs)
 *   dweights[t][k] = sum over c of dy[t][c] * rows[row_of[t][k]][c]   (0 for dropped pairs)
 *   dy    [T][C] BF16 (FP32 with FP8BLK_MOE_TOKENS_F32), pitch lddy.
 *   rows  [T*K][C] BF16 (FP32 with FP8BLK_MOE_ROWS_F32), pitch ldr.
 *   drows [T*K][C] BF16 (FP32 with FP8BLK_MOE_DROWS_F32), pitch lddr.
 *   dweights FP32 [T][K], dense.
 */
fp8blk_status_t fp8blk_moe_combine_backward(const void* dy, int64_t lddy, const void* rows, int64_t ldr, int64_t T,
                                            int64_t K, int64_t C, const int32_t* row_of, const float* weights,
                                            void* drows, int64_t lddr, float* dweights, uint32_t flags,
                                            void* stream);

/* ------------------------------------------------------------------------
 * Norms around a block.
 * ------------------------------------------------------------------------ */
#define FP8BLK_NORM_RES_F32 0x10u    /* x, x_out, dx_out, dx are FP32 (BF16 without) */
#define FP8BLK_NORM_PARAM_F32 0x20u  /* w_post, w_pre and a gate per channel are FP32 (BF16 without) */
#define FP8BLK_NORM_GATE_ROW 0x40u   /* gate is [M][C] BF16, one per token and channel (per channel without) */

/*
 * The end of one block and the start of the next, for M tokens of C channels:
 *   u  = f * r_post * w_post,  r_post = (mean_c f^2 + eps)^(-1/2)   (u = f if w_post is NULL)
 *   x' = x + alpha * gate * u                                       (x' = x if f is NULL; gate 1 if NULL)
 *   n  = x' * r_pre * w_pre,   r_pre = (mean_c x'^2 + eps)^(-1/2)   (only if w_pre is given)
 *   (q, s) = 1x128 E4M3 quantization of n                           (only if q is given)
 * All in FP32; x' enters the second norm, and n the quantizer, before being
 * rounded for storage.  A tile's scale is fl32(amax / 448) of its FP32 values
 * (the smallest power of two not below amax / 448 with FP8BLK_SCALE_POW2 in
 * flags; 1 for a tile of zeros) and its codes are E4M3(n / s), the quotient
 * within one unit in the last place of FP32.
 *   x      [M][C] BF16 or FP32, pitch ldx.
 *   f      [M][C] BF16, pitch ldf, or NULL.
 *   w_post, w_pre  [C], element aligned, or NULL.
 *   gate   [C] (element aligned) or, with FP8BLK_NORM_GATE_ROW, [M][C] with
 *          pitch ldg; or NULL.  w_post and gate need f.
 *   x_out  [M][C] as x, pitch ldxo; required with f, NULL without.  It may be
 *          x itself (same pitch).
 *   n      [M][C] BF16, pitch ldn, or NULL; q [M][C] codes, pitch ldq, with
 *          s [ceil(C/128)][M] FP32, or both NULL.  With w_pre at least one of
 *          n and q is given, without it neither.
 *   rstd_post, rstd_pre  [M] FP32, r_post and r_pre for the gradient, or NULL.
 *   C at most 16384 (FP8BLK_ERR_UNSUPPORTED otherwise).
 */
fp8blk_status_t fp8blk_residual_norm(int64_t M, int64_t C, const void* x, int64_t ldx, const uint16_t* f, int64_t ldf,
                                     const void* w_post, const void* gate, int64_t ldg, float alpha,
                                     const void* w_pre, float eps, void* x_out, int64_t ldxo, uint16_t* n, int64_t ldn,
                                     uint8_t* q, int64_t ldq, float* s, float* rstd_post, float* rstd_pre,
                                     uint32_t flags, void* stream);

/*
 * Its gradient, from dx_out (into x') and dn (into n):
 *   g  = dx_out + r_pre * (v - h * mean_c(v * h)),   v = dn * w_pre, h = x' * r_pre
 *   dx = g;  dw_pre = sum_m dn * h;  d = alpha * gate * g
 *   df = r_post * (v' - h' * mean_c(v' * h')),       v' = d * w_post, h' = f * r_post   (df = d if w_post is NULL)
 *   dw_post = sum_m d * h';  dgate = alpha * g * u   (summed over m for a gate per channel)
 *   x_out  the x' that the forward stored (x where f is NULL); may be NULL
 *          without w_pre.
 *   dx_out may be NULL (zeros); dn, rstd_pre, dw_pre go with w_pre: all or
 *          none.  f, df: both or neither; rstd_post, dw_post go with w_post;
 *          dgate with gate.  At least one of dx_out and dn is given.
 *   dx     [M][C] as x, pitch lddx; NULL if not wanted.
 *   df     [M][C] BF16, pitch lddf.
 *   dgate  FP32 [C], or BF16 [M][C] with pitch lddg for FP8BLK_NORM_GATE_ROW.
 *   dw_pre, dw_post  FP32 [C].
 *   workspace  fp8blk_residual_norm_backward_workspace_bytes(M, C) bytes,
 *          16-byte aligned; needed only where a sum over m is asked for.
 *   With M = 0 the sums over m are zeros.
 */
fp8blk_status_t fp8blk_residual_norm_backward(
    int64_t M, int64_t C, const void* x_out, int64_t ldx, const void* dx_out, int64_t lddxo, const uint16_t* dn,
    int64_t lddn, const float* rstd_pre, const void* w_pre, const uint16_t* f, int64_t ldf, const float* rstd_post,
    const void* w_post, const void* gate, int64_t ldg, float alpha, void* dx, int64_t lddx, uint16_t* df, int64_t lddf,
    float* dw_pre, float* dw_post, void* dgate, int64_t lddg, void* workspace, size_t workspace_bytes, uint32_t flags,
    void* stream);
size_t fp8blk_residual_norm_backward_workspace_bytes(int64_t M, int64_t C);

/* ------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping.
 * ------------------------------------------------------------------------ */
#define FP8BLK_GRAD_F32 0x1u     /* grad is FP32 (BF16 without) */
#define FP8BLK_GRAD_OUT_F32 0x2u /* out is FP32 (BF16 without) */

/* One gradient: rows x cols elements, rows ld (ldo) elements apart; pointers
 * aligned to their element.  out may be grad itself with the same type and
 * pitch (clipped in place); it must not overlap any other tensor. */
typedef struct {
  const void* grad;
  void* out;
  int64_t rows, cols;
  int64_t ld, ldo;
  uint32_t flags;
  uint32_t reserved; /* 0 */
} fp8blk_grad_t;

/*
 * The table of n gradients that the calls below read, built on the host: the
 * caller copies its fp8blk_grad_table_bytes(n) bytes to the device once and
 * uses it for as long as the tensors stay where they are.
 * fp8blk_grad_table_build checks the list and fills `table` (HOST memory,
 * 8-byte aligned); *chunks receives the number of work chunks, which the
 * calls take.
 */
size_t fp8blk_grad_table_bytes(int64_t n);
fp8blk_status_t fp8blk_grad_table_build(const fp8blk_grad_t* list, int64_t n, void* table, size_t table_bytes,
                                        int64_t* chunks);

/* Workspace of the calls below: constant, 8-byte aligned. */
#define FP8BLK_GRAD_WORKSPACE_BYTES ((size_t)16384)

/*
 * *norm = (sum over all elements of all gradients of g^2)^(1/2), FP32 on the
 * device, the sum held in FP64 (it neither overflows nor loses small values).
 *   table  DEVICE copy of what fp8blk_grad_table_build filled, with its n and
 *   chunks.  n = 0 gives 0.  NaN or infinite elements give a NaN or infinite norm.
 */
fp8blk_status_t fp8blk_grad_norm(const void* table, int64_t n, int64_t chunks, float* norm, void* workspace,
                                 size_t workspace_bytes, void* stream);
/*
 * out = grad * c for every gradient, c = min(1, max_norm / (*norm + eps)),
 * multiplied in FP32 and rounded once.  A gradient clipped in place is not
 * touched where c = 1.  A NaN norm makes c NaN, an infinite one 0.  `norm` is
 * read on the device (e.g. after a reduction over ranks).
 */
fp8blk_status_t fp8blk_grad_clip(const void* table, int64_t n, int64_t chunks, const float* norm, float max_norm,
                                 float eps, void* stream);
/* Both: fp8blk_grad_norm into *norm, then fp8blk_grad_clip by it. */
fp8blk_status_t fp8blk_grad_clip_norm(const void* table, int64_t n, int64_t chunks, float max_norm, float eps,
                                      float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBFP8BLK_LAYER_H */
