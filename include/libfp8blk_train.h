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
 * m takes the low half of r, v the high half, a BF16 param the low half of
 * the r of k xor 0x5BD1E995: 16 bits, added below the kept ones (16 dropped
 * ones of BF16, 20 of E4M3, the upper 16 of those) before they are dropped.
 * E4M3 values below 2^-6 take the codes' spacing there, 2^-9. */
#define FP8BLK_ADAMW_RANDOM 0x1u

/* What a step depends on.  Values that change from step to step may come from
 * device memory, read when the kernel runs, so that a captured graph can be
 * replayed: lr_at, step_at, seed_at non-NULL replace lr, step and seed. */
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
