/*
 * libfp8blk — the gated feed-forward block in FP8 and the optimizer step, for
 * AMD Instinct MI355X (gfx950):
 *
 *   gate and up projection, the activation and the product in one GEMM, with
 *   the block's gradient (the pages' experts have gate, up and down
 *   projections, all three in FP8 in every direction [p1¶3, p5¶3], and
 *   quantize what the next projection reads [p2¶4]);
 *   one AdamW step over many tensors, with moments in FP32, BF16 or E4M3 (the
 *   pages keep optimizer states in low precision [p2¶4]).
 *
 * Citations [pN¶k] as in libfp8blk.h.  Status codes, streams, ownership and
 * the host-side validation of arguments are those of libfp8blk.h: device
 * pointers, everything asynchronous on `stream`, nothing allocated, filled or
 * copied, an invalid call returns FP8BLK_ERR_INVALID_ARG and touches nothing,
 * sizes of zero are valid.  Matrix pointers are 16-byte aligned and row
 * pitches multiples of 16 bytes.  Results do not depend on the run: no
 * floating-point sum is formed by atomics.
 */
#ifndef LIBFP8BLK_TRAIN_H
#define LIBFP8BLK_TRAIN_H

#include "libfp8blk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ABI version of this header: 1. */
int fp8blk_train_abi_version(void);

/* ------------------------------------------------------------------------
 * The gated feed-forward block: u = X W_up with the gate projection in W_up's
 * first H columns and the up projection in its last H, h = act(u_g) * u_u, and
 * what follows is a plain product of h with the down projection.
 * H and K multiples of 128, M arbitrary.
 *
 * Definitions, from the FP32 products u and dh that fp8blk_gemm_fp8_blockscaled
 * defines, all in FP32 and rounded for storage only:
 *   act(g) = g p,  p = 1 / (1 + e^-z),
 *     z = g (SILU) or (8/pi)^(1/2) (g + 0.044715 g^3) (GELU, its tanh form)
 *   h = act(u_g) u_u
 *   du_u = dh act(u_g),  du_g = dh u_u (p + g p (1 - p) dz/dg)
 * and (q, s) = fp8blk_quantize_1x128 of h, or of du, as stored in BF16, with
 * flags qflags, whether or not h or du itself is asked for.
 *
 * A product of few rows is split along K over the GPU and joined in a second
 * launch if `workspace` (DEVICE, 16-byte aligned, contents irrelevant, not used
 * by other work during the call) has the bytes that the call's _workspace_bytes
 * gives; without it, one launch computes it all.  Either form gives the same
 * bits on every run.
 *
 * Outputs and the workspace overlap neither each other nor an input; only du
 * may be u.  (The Python binding refuses such calls, this interface does not see
 * the memory's owners.)
 * ------------------------------------------------------------------------ */
enum { FP8BLK_ACT_SILU = 0, FP8BLK_ACT_GELU = 1 };

/*
 * Both projections, the activation and the product.
 *   A  [M][K] codes, sA [K/128][M]; B [K][2H] (FP8BLK_OP_N) or [2H][K]
 *   (FP8BLK_OP_T), block scales; FP8BLK_GEMM_POW2_SCALES allowed in opB: as in
 *   fp8blk_gemm_fp8_blockscaled with N = 2H.
 *   u  [M][2H] BF16, pitch ldu, kept for the gradient, or NULL.
 *   h  [M][H] BF16, pitch ldh, or NULL; q [M][H] codes, pitch ldq, with
 *   s [H/128][M] FP32, or both NULL.  At least one of h and q is given.
 *   FP8BLK_ERR_UNSUPPORTED for FP8BLK_OP_T where (H + 128) * ldb reaches 2^31.
 */
fp8blk_status_t fp8blk_gated_gemm_fp8_blockscaled(int64_t M, int64_t H, int64_t K, const uint8_t* A, int64_t lda,
                                                  const float* sA, const uint8_t* B, int64_t ldb, int opB,
                                                  const float* sB, int act, uint16_t* u, int64_t ldu, uint16_t* h,
                                                  int64_t ldh, uint8_t* q, int64_t ldq, float* s, uint32_t qflags,
                                                  void* workspace, size_t workspace_bytes, void* stream);
size_t fp8blk_gated_gemm_workspace_bytes(int64_t M, int64_t H, int64_t K);

/*
 * The same for every expert's rows: group_offsets, M_total, max_group_rows,
 * strideB and stride_sB as in fp8blk_grouped_gemm_fp8_blockscaled; s
 * [H/128][M_total].  Rows from group_offsets[G] on are not written.
 */
fp8blk_status_t fp8blk_grouped_gated_gemm_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t H, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, int act, uint16_t* u, int64_t ldu, uint16_t* h, int64_t ldh, uint8_t* q,
    int64_t ldq, float* s, uint32_t qflags, void* stream);

/*
 * The gradient: the down projection's input gradient dh = dO W_down^T, and the
 * activation's from it.
 *   A  [M][K] codes of dO, sA [K/128][M].
 *   B  W_down, [H][K] (FP8BLK_OP_T: as the forward's product h W_down reads it
 *      with FP8BLK_OP_N) or [K][H] (FP8BLK_OP_N), block scales.
 *   u  [M][2H] BF16 that the forward kept.
 *   du [M][2H] BF16, pitch lddu, or NULL; it may be u itself (same pitch).
 *   h  [M][H] BF16, act(u_g) u_u for the down projection's weight gradient, or
 *      NULL.  It is formed from u as given, the forward's h from the FP32
 *      products: the two lie apart by what u's rounding to BF16 makes of h.
 *   q  [M][2H] codes of du, what the up projection's gradients read, with
 *      s [2H/128][M], or both NULL.  At least one of du and q is given.
 */
fp8blk_status_t fp8blk_gated_gemm_backward_fp8_blockscaled(
    int64_t M, int64_t H, int64_t K, const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb,
    int opB, const float* sB, int act, const uint16_t* u, int64_t ldu, uint16_t* du, int64_t lddu, uint16_t* h,
    int64_t ldh, uint8_t* q, int64_t ldq, float* s, uint32_t qflags, void* workspace, size_t workspace_bytes,
    void* stream);
size_t fp8blk_gated_gemm_backward_workspace_bytes(int64_t M, int64_t H, int64_t K);

/* The same for every expert's rows; rows from group_offsets[G] on are neither read nor written. */
fp8blk_status_t fp8blk_grouped_gated_gemm_backward_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t H, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, int act, const uint16_t* u, int64_t ldu, uint16_t* du, int64_t lddu,
    uint16_t* h, int64_t ldh, uint8_t* q, int64_t ldq, float* s, uint32_t qflags, void* stream);

/* ------------------------------------------------------------------------
 * AdamW over many tensors.  For every element, t steps taken with this one:
 *   g = grad * c,  c = min(1, max_norm / (*norm + clip_eps))   (c = 1 without norm)
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in FP32; p uses m and v before they are rounded for storage.
 * ------------------------------------------------------------------------ */

/* How the moments are stored, one for a whole table:
 *   F32, BF16  m and v as they are;
 *   E4M3       codes of m / s_m and of sqrt(v) / s_v, with one FP32 scale
 *              (amax times 1 / 448, both in FP32; 1 where all are zero) for
 *              every 128 consecutive elements of a tensor.  A v that is not zero keeps at least the
 *              smallest code, so that no moment is divided by a rounded-off
 *              zero.  A NaN or an infinity spoils its 128 elements' moments. */
enum { FP8BLK_ADAMW_F32 = 0, FP8BLK_ADAMW_BF16 = 1, FP8BLK_ADAMW_E4M3 = 2 };

#define FP8BLK_ADAMW_PARAM_F32 0x1u /* param is FP32 (BF16 without) */
#define FP8BLK_ADAMW_GRAD_F32 0x2u  /* grad is FP32 (BF16 without) */

/* One tensor: rows x cols elements, rows ldp (ldg, ldc) elements apart in
 * param (grad, copy); pointers aligned to their element.  The moments are
 * dense, in the same order: rows*cols elements of the table's kind, for E4M3
 * codes with 4-byte aligned m and v and ceil(rows*cols / 128) scales each.
 * copy: BF16, receives the new param rounded to nearest, or NULL.  No tensor
 * may overlap another one that is written. */
typedef struct {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale; /* E4M3 only, NULL otherwise */
  float* v_scale;
  uint16_t* copy;
  int64_t rows, cols;
  int64_t ldp, ldg, ldc;
  float decay;
  uint32_t flags;
  uint32_t index;    /* of the tensor in the caller's list: varies its random bits */
  uint32_t reserved; /* 0 */
} fp8blk_adamw_t;

/*
 * The table of n tensors that the step reads, built on the host as
 * fp8blk_grad_table_build builds its table: checks the list, fills `table`
 * (HOST memory, 8-byte aligned, fp8blk_adamw_table_bytes(n) bytes), which the
 * caller copies to the device once; *chunks receives the number of work chunks.
 */
size_t fp8blk_adamw_table_bytes(int64_t n);
fp8blk_status_t fp8blk_adamw_table_build(const fp8blk_adamw_t* list, int64_t n, int state, void* table,
                                         size_t table_bytes, int64_t* chunks);

/* Rounding of BF16 params, BF16 moments and E4M3 moments: to nearest, or at
 * random with FP8BLK_ADAMW_RANDOM in flags: up with the probability of the
 * distance, so that small changes are kept on average (an E4M3 moment that
 * decays by 5 % a step never leaves its code otherwise, nor a BF16 param whose
 * update is below 2^-9 of it).  The bits depend on `seed`, the tensor's index
 * and the element's place alone:
 *   i = place, k = (seed + index * 0x27D4EB2F) mod 2^32
 *   h = (i * 0x9E3779B1 xor i >> 32) + k;  h = (h xor h >> 16) * 0x85EBCA6B;
 *   h = (h xor h >> 13) * 0xC2B2AE35;  r = h xor h >> 16          (all mod 2^32)
 * (the last two lines are the 32-bit finalizer of MurmurHash3, a published one).
 * m takes the low half of r, v the high half, a BF16 param the low half of
 * the r of k xor 0x5BD1E995: 16 bits, added below the kept ones (16 dropped
 * ones of BF16, 20 of E4M3, the upper 16 of those) before they are dropped.
 * E4M3 values below 2^-6 take the codes' spacing there, 2^-9. */
#define FP8BLK_ADAMW_RANDOM 0x1u

/* What a step depends on.  Values that change from step to step may come from
 * device memory, read when the kernel runs, so that a captured graph can be
 * replayed: lr_at, step_at, seed_at non-NULL replace lr, step and seed.  They
 * are not checked: below 1 step a moment's correction is not finite. */
typedef struct {
  double lr, beta1, beta2, eps; /* FP64: 1 - 0.999 in FP32 is off by 5e-5 of itself */
  int64_t step;                 /* t, at least 1 */
  uint32_t seed, flags;
  const float* lr_at;
  const int64_t* step_at;
  const int64_t* seed_at; /* its low 32 bits */
  const float* norm;      /* clipping: a norm on the device, or NULL */
  float max_norm, clip_eps;
} fp8blk_adamw_step_t;

/*
 * One step.  table: DEVICE copy of what fp8blk_adamw_table_build filled, with
 * its n, chunks and state.  0 <= beta1, beta2 < 1, eps >= 0, lr finite.  A NaN
 * norm makes c NaN, an infinite one 0.
 */
fp8blk_status_t fp8blk_adamw_step(const void* table, int64_t n, int64_t chunks, int state,
                                  const fp8blk_adamw_step_t* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBFP8BLK_TRAIN_H */
