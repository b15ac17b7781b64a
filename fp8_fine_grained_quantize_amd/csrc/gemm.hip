// Block-scaled FP8 GEMM for gfx950: dense and grouped (per-expert).
//
//   C[m][n] = sum_g sA[g][m] * sB(g, n) * P_g[m][n],
//   P_g     = the 128-deep K group g's FP8 product.
//
// The pages apply one scale per 128-element group along K, multiply the
// scales in during dequantization [p2¶4] and promote the matrix-core partial
// sums into full-precision FP32 accumulators at a fixed K interval [p2¶3].
// Here the interval is the scale group itself: each 16x16 output tile gets one
// v_mfma_scale_f32_16x16x128_f8f6f4 per group (K = 128 in one instruction,
// starting from zero), and the FP32 result is folded into a separate FP32
// accumulator with one FMA by fl32(sA * sB).  Fprop, Dgrad and Wgrad all use
// this kernel family [p1¶3, Figure 6; p5¶4].
//
// When every scale is a power of two (the pages' choice for some activations
// [p2¶4]; FP8BLK_GEMM_POW2_SCALES), the scales are exact E8M0 block scales:
// the MFMA applies them to its operands and adds the group's product to the
// FP32 accumulator itself (srcC, round to nearest even), so the promotion
// needs no vector-ALU work.
// Citations [pN¶k]: N-th page of the source collection, k-th paragraph
// (p1 = xn--9g3bo1gtkw0l8ubf92bgle.kr wr_id 85187, p2 = inprokorea.com wr_id
// 735329, p5 = inprokorea.com wr_id 890463).
// The tile code is in gemm_tile.h.
#include <atomic>
#include <mutex>

#include "gemm_tile.h"

namespace fp8blk {

template <class CFG, bool OPB_T, bool ROW128, bool P2, int OM>
__global__ __launch_bounds__(CFG::NT) void k_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* __restrict__ A,
                                                   int64_t lda, const float* __restrict__ sA,
                                                   const uint8_t* __restrict__ B, int64_t ldb,
                                                   const float* __restrict__ sB, int64_t sB_ld,
                                                   void* __restrict__ C, int64_t ldc, int64_t tiles_m,
                                                   int64_t tiles_n, float* __restrict__ partials, int groups_per_split,
                                                   float* __restrict__ sQ) {
  FP8BLK_DECLARE_STAGES(CFG);
  int64_t tm, tn;
  tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn);
  // Split K: workgroup row blockIdx.y computes the partial product of K
  // groups [y*groups_per_split, ...) into its own [M][N] slice of `partials`.
  const int G = (int)(K / 128);
  // (Only FP32-output kernels are split: a split GEMM writes FP32 partials
  // and the reduction writes BF16 when asked to.)
  const int split = blockIdx.y;
  if (gridDim.y > 1) {  // partial slices of pitch N rounded up to 4 floats (16-byte rows)
    const int64_t Np = (N + 3) & ~int64_t(3);
    C = partials + (int64_t)split * M * Np;
    ldc = Np;
  }
  const int64_t m0 = tm * CFG::BM;
  TileArgs t;
  t.A = A + m0 * lda;
  t.lda = lda;
  t.rows = (M - m0) < CFG::BM ? (M - m0) : CFG::BM;
  t.sA = sA + m0;
  t.sA_ld = M;
  t.B = B;
  t.ldb = ldb;
  t.n0 = tn * CFG::BN;
  t.N = N;
  t.sB = sB;
  t.sB_ld = sB_ld;
  t.C = out_row(C, ldc, m0, out_elem_bytes(OM));
  t.ldc = ldc;
  t.sQ = sQ;
  t.sQ_ld = M;
  t.m0 = m0;
  t.K = K;
  t.g0 = split * groups_per_split;
  t.g1 = t.g0 + groups_per_split < G ? t.g0 + groups_per_split : G;
  gemm_tile<CFG, OPB_T, ROW128, P2, OM>(t, s_ops0, s_ops1, s_sc0, s_sc1);
}

// Partial row tiles of the grouped GEMM: waves whose rows all lie past the
// expert's last row skip their MFMAs and folds, and A copies of such rows
// are not issued.  Measured (interleaved, one box, bitwise identical): MoE
// up 3.26 -> 3.23 ms, down 2.055 -> 2.025 ms, down Dgrad 1.69 -> 1.68 ms.
// An L2 prefetch of each tile's weight slab 2-4 groups ahead (4-byte copies
// into a dummy LDS area) made all three 10-13 % slower and was dropped.
// Balancing the real tiles over the 8 XCDs (k_grouped_gemm, in place of a
// remap over the whole upper-bound grid, which left the MoE shapes' tiles to
// six XCDs, 1.27x the balanced share on the busiest): MoE up 3.35 ->
// 2.94 ms, down 2.15 -> 1.81 ms, down Dgrad 1.72 -> 1.45 ms (interleaved, one
// box, bitwise identical), so a grouped tile now takes within a few percent of
// a dense tile's time (2.94 ms over 25.2 tiles per CU).
#ifndef FP8BLK_GROUPED_SKIP
#define FP8BLK_GROUPED_SKIP 1
#endif
// Every expert's rows times its own matrix (grouped_tile says which tile a workgroup takes).
template <class CFG, bool OPB_T, bool P2, int OM>
__global__ __launch_bounds__(CFG::NT) void k_grouped_gemm(int64_t G, const int32_t* __restrict__ offsets,
                                                           int64_t M_total, int64_t N, int64_t K,
                                                           const uint8_t* __restrict__ A, int64_t lda,
                                                           const float* __restrict__ sA,
                                                           const uint8_t* __restrict__ B, int64_t ldb,
                                                           int64_t strideB, const float* __restrict__ sB,
                                                           int64_t stride_sB, int64_t sB_ld,
                                                           void* __restrict__ C, int64_t ldc, int64_t tiles_n) {
  FP8BLK_DECLARE_STAGES(CFG);
  int64_t e, tn, m0, rows;
  if (!grouped_tile<CFG>(offsets, G, tiles_n, e, tn, m0, rows)) return;
  TileArgs t;
  t.A = A + m0 * lda;
  t.lda = lda;
  t.rows = rows;
  t.sA = sA + m0;
  t.sA_ld = M_total;
  t.B = B + e * strideB;
  t.ldb = ldb;
  t.n0 = tn * CFG::BN;
  t.N = N;
  t.sB = sB + e * stride_sB;
  t.sB_ld = sB_ld;
  t.C = out_row(C, ldc, m0, out_elem_bytes(OM));
  t.ldc = ldc;
  t.K = K;
  t.g0 = 0;
  t.g1 = (int)(K / 128);
  gemm_tile<CFG, OPB_T, false, P2, OM, FP8BLK_GROUPED_SKIP != 0>(t, s_ops0, s_ops1, s_sc0, s_sc1);
}

// Grouped Wgrad of MoE experts: dW_e = X_e^T dY_e for every expert e, both
// operands 128x1-quantized along tokens inside each expert (ragged token
// groups, token_groups.h) and stored transposed, so that expert e's K range
// is its own group slots [PG[e], PG[e] + n_e) of the shared code matrices.
// Every expert's output has the same M x N tiles; tiles are enumerated expert
// by expert, column tile by column tile, row tiles innermost.  An expert
// without tokens gets dW_e = 0.
// One LDS stage: an expert's tiles have only 2-3 K groups on average, so the
// second stage bought little overlap and held the kernel to two workgroups
// per compute unit by LDS; with one stage (35 KB) three are resident (by
// registers) and one workgroup's stores overlap another's loads.  Measured
// (interleaved, one box, bitwise identical) on the MoE down projection's
// Wgrad: FP32 output 4.95 -> 4.63 ms, BF16 3.74 -> 3.41 ms.  Holding the
// kernel to 128 VGPRs for four workgroups per compute unit spills.
#ifndef FP8BLK_WGRAD_STAGES
#define FP8BLK_WGRAD_STAGES 1
#endif
template <class CFG, bool P2, int OM>
__global__ __launch_bounds__(CFG::NT) void k_grouped_wgrad(const int32_t* __restrict__ offsets, int64_t M, int64_t N,
                                                            const uint8_t* __restrict__ A, int64_t lda,
                                                            const float* __restrict__ sA,
                                                            const uint8_t* __restrict__ B, int64_t ldb,
                                                            const float* __restrict__ sB, void* __restrict__ C,
                                                            int64_t ldc, int64_t strideC, int64_t tiles_m,
                                                            int64_t tiles_n) {
#if FP8BLK_WGRAD_STAGES == 1
  __shared__ __align__(16) uint8_t s_ops0[CFG::BUF_BYTES];
  __shared__ __align__(16) float s_sc0[CFG::SC_FLOATS];
  uint8_t* s_ops1 = s_ops0;
  float* s_sc1 = s_sc0;
#else
  FP8BLK_DECLARE_STAGES(CFG);
#endif
  __shared__ int64_t s_red[CFG::NT];
  const int64_t per = tiles_m * tiles_n;
  const int64_t lin = blockIdx.x;
  // Column tiles fastest: consecutive workgroups write one 128-row band of
  // dW_e side by side (rows of 7168 FP32 are 28 KB apart), and with ids dealt
  // round-robin over the 8 XCDs each XCD keeps reading the same eighth of the
  // expert's B tiles.  Measured 14 % faster than row tiles fastest, whose
  // in-flight tiles write 512-byte pieces spread over the whole dW_e.
  const int64_t e = lin / per, rem = lin % per;
  const int64_t tm = rem / tiles_n, tn = rem % tiles_n;
  const int64_t pg = token_group_start<CFG::NT>(offsets, e, s_red);
  const int64_t ng = token_groups_of(offsets, e);
  const int64_t m0 = tm * CFG::BM;
  TileArgs t;
  t.A = A + m0 * lda;
  t.lda = lda;
  t.rows = (M - m0) < CFG::BM ? (M - m0) : CFG::BM;
  t.sA = sA + m0;
  t.sA_ld = M;
  t.B = B;
  t.ldb = ldb;
  t.n0 = tn * CFG::BN;
  t.N = N;
  t.sB = sB;
  t.sB_ld = N;
  t.C = out_row(out_row(C, strideC, e, out_elem_bytes(OM)), ldc, m0, out_elem_bytes(OM));
  t.ldc = ldc;
  t.K = 128 * (pg + ng);
  t.g0 = (int)pg;
  t.g1 = (int)(pg + ng);
  gemm_tile<CFG, true, true, P2, OM, false, FP8BLK_WGRAD_STAGES == 1>(t, s_ops0, s_ops1, s_sc0, s_sc1);
}

// Split-K reduction: C[m][n] = sum over s = 0 .. S-1, in that order, of the
// partial products partials[s][m][n] (FP32 additions).  The partial slices
// have row pitch Np = N rounded up to 4 floats, so every thread reads four
// consecutive columns as 16-byte words (columns from N to Np are padding,
// read but never stored).
__global__ __launch_bounds__(256) void k_splitk_reduce(const float* __restrict__ partials, int S, int64_t M,
                                                       int64_t N, void* __restrict__ Cv, int64_t ldc, int out_bf16) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;  // index of a 4-column chunk
  const int64_t Np = (N + 3) & ~int64_t(3);
  const int64_t cpr = Np / 4;
  const int64_t m = q / cpr, n = (q % cpr) * 4;
  if (m >= M) return;
  const int64_t MN = M * Np;
  const float* src = partials + m * Np + n;
  float4 a = *reinterpret_cast<const float4*>(src);
  for (int s = 1; s < S; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(src + s * MN);
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  const float acc[4] = {a.x, a.y, a.z, a.w};
  if (out_bf16) {
    uint16_t* dst = static_cast<uint16_t*>(Cv) + m * ldc + n;
    if (n + 4 <= N)
      *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pack(acc[0], acc[1]), bf16_pack(acc[2], acc[3]));
    else
      for (int r = 0; r < 4 && n + r < N; ++r) dst[r] = (uint16_t)(bf16_pack(acc[r], 0.0f) & 0xFFFFu);
  } else {
    float* dst = static_cast<float*>(Cv) + m * ldc + n;
    if (n + 4 <= N)
      *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    else
      for (int r = 0; r < 4 && n + r < N; ++r) dst[r] = acc[r];
  }
}

// K splits for a dense GEMM: only when its 128 x 128 tiles cannot fill the
// compute units and K is long enough (at least FP8BLK_SPLITK_MIN_GROUPS
// groups) for the split to save more than the reduction's launch costs; each
// split keeps at least eight K groups, at most FP8BLK_SPLITK_MAX splits.
// Measured on 1024 x 1024 x K (one box): K = 4096 with 2 / 4 / 8 splits
// 27.6 / 22.0 / 24.4 us, K = 8192 40.7 / 28.8 / 28.9 us, K = 16384
// 70.7 / 44.7 / 38.9 us.
#ifndef FP8BLK_SPLITK_MIN_GROUPS
#define FP8BLK_SPLITK_MIN_GROUPS 16
#endif
#ifndef FP8BLK_SPLITK_MAX
#define FP8BLK_SPLITK_MAX 16
#endif
static int64_t splitk_count(int64_t M, int64_t N, int64_t K) {
  const int64_t big_tiles = ceil_div(M, BigCfg::BM) * ceil_div(N, BigCfg::BN);
  if (big_tiles >= 128) return 1;
  const int64_t G = K / 128;
  if (G < FP8BLK_SPLITK_MIN_GROUPS) return 1;
  const int64_t tiles = ceil_div(M, SmallCfg::BM) * ceil_div(N, SmallCfg::BN);
  const int64_t slots = 2 * (int64_t)device_cus();  // two 128 x 128 workgroups fit per CU
  int64_t S = ceil_div(slots, tiles);
  if (S > G / 8) S = G / 8;
  if (S > FP8BLK_SPLITK_MAX) S = FP8BLK_SPLITK_MAX;
  return S < 1 ? 1 : S;
}

// 224x256 tiles in place of 256x256 when they take fewer tile rows per CU:
// ceil(tiles / CUs) launch waves times the tile height.  On 256 CUs the
// 7168 x 2048 output (the Wgrad of a 7168-wide layer over a 2048-wide one)
// is 224 tiles of 256 rows, one launch wave with 32 CUs idle, or exactly 256
// tiles of 224 rows, each 7/8 of the MFMA work and 15/16 of the copies;
// square outputs such as 4096 x 4096 keep the 256-row tiles.  Measured
// (interleaved against 256-row tiles, one box, results bitwise identical):
// 7168 x 2048 x 4096 Wgrad 77.0 -> 73.8 us, power-of-two scales 70.8 -> 67.8;
// 4100 x 2050 x 7168 (153 -> 171 tiles) 104.5 -> 97.4 us, power-of-two
// 98.7 -> 101.6 (the one loss).
static bool use_tile224(int64_t M, int64_t N) {
  const int64_t cus = device_cus();
  const int64_t t256 = ceil_div(M, BigCfg::BM) * ceil_div(N, BigCfg::BN);
  const int64_t t224 = ceil_div(M, Big224Cfg::BM) * ceil_div(N, Big224Cfg::BN);
  return ceil_div(t224, cus) * Big224Cfg::BM < ceil_div(t256, cus) * BigCfg::BM;
}

static size_t splitk_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t S = splitk_count(M, N, K);
  const int64_t Np = (N + 3) & ~int64_t(3);
  return S > 1 ? (size_t)S * (size_t)M * (size_t)Np * sizeof(float) : 0;
}

template <class CFG, bool OPB_T, bool ROW128, bool P2>
static fp8blk_status_t launch_dense(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                                    const uint8_t* B, int64_t ldb, const float* sB, int64_t sB_ld, void* C,
                                    int64_t ldc, int out_bf16, float* partials, int64_t S, hipStream_t stream) {
  const int64_t tiles_m = ceil_div(M, CFG::BM), tiles_n = ceil_div(N, CFG::BN);
  const int64_t blocks = tiles_m * tiles_n;
  if (blocks > 0x7FFFFFFF) return FP8BLK_ERR_UNSUPPORTED;
  const int64_t G = K / 128;
  const int64_t per = ceil_div(G, S);
  S = ceil_div(G, per);  // no empty split
  if (out_bf16 && S == 1)
    hipLaunchKernelGGL((k_gemm<CFG, OPB_T, ROW128, P2, OUT_BF16>), dim3((unsigned)blocks), dim3(CFG::NT), 0, stream, M,
                       N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, tiles_m, tiles_n, partials, (int)per, nullptr);
  else
    hipLaunchKernelGGL((k_gemm<CFG, OPB_T, ROW128, P2, OUT_F32>), dim3((unsigned)blocks, (unsigned)S), dim3(CFG::NT), 0,
                       stream, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, tiles_m, tiles_n, partials, (int)per,
                       nullptr);
  if (S > 1) {
    if (hipGetLastError() != hipSuccess) return FP8BLK_ERR_LAUNCH;
    const int64_t chunks = M * ceil_div(N, 4);  // N rounded up to 4 floats, in chunks of 4
    hipLaunchKernelGGL(k_splitk_reduce, dim3((unsigned)ceil_div(chunks, 256)), dim3(256), 0, stream, partials, (int)S,
                       M, N, C, ldc, out_bf16);
  }
  return launch_status();
}

template <class CFG, bool ROW128>
static fp8blk_status_t dispatch_dense(bool t, bool p2, int64_t M, int64_t N, int64_t K, const uint8_t* A,
                                      int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, const float* sB,
                                      int64_t sB_ld, void* C, int64_t ldc, int ob, float* partials, int64_t S,
                                      hipStream_t st) {
  if (p2) {
    if (t) return launch_dense<CFG, true, ROW128, true>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
    return launch_dense<CFG, false, ROW128, true>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
  }
  if (t) return launch_dense<CFG, true, ROW128, false>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
  return launch_dense<CFG, false, ROW128, false>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
}

}  // namespace fp8blk

using namespace fp8blk;

// Per-lane copy offsets are 32-bit: operand pitches stay below 2^23 bytes.
static constexpr int64_t kMaxPitch = int64_t(1) << 23;

// Workspace that lets the dense GEMM split K (0: it never splits this
// shape); the grouped GEMM needs none.
extern "C" size_t fp8blk_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t G) {
  if (G > 1 || M <= 0 || N <= 0 || K <= 0 || K % 128 != 0) return 0;
  return splitk_bytes(M, N, K);
}

// Argument checks and tile/split choice shared by the dense entry points.
// `workspace` is the split-K partials buffer (S slices of M x N rounded up
// to 4 floats); with too small a workspace the GEMM runs in one pass, or,
// with `strict`, the call fails with FP8BLK_ERR_UNSUPPORTED.
static fp8blk_status_t gemm_dense(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                                  const uint8_t* B, int64_t ldb, int opB, const float* sB, int bscale_mode, void* C,
                                  int64_t ldc, void* workspace, size_t workspace_bytes, bool strict, void* stream) {
  if (M < 0 || N < 0 || K < 0) return FP8BLK_ERR_INVALID_ARG;
  const bool p2 = (opB & FP8BLK_GEMM_POW2_SCALES) != 0;
  const int ob = (opB & FP8BLK_GEMM_OUT_BF16) != 0;
  opB &= ~(FP8BLK_GEMM_POW2_SCALES | FP8BLK_GEMM_OUT_BF16);
  if (opB != FP8BLK_OP_N && opB != FP8BLK_OP_T) return FP8BLK_ERR_INVALID_ARG;
  if (bscale_mode != FP8BLK_BSCALE_BLOCK128 && bscale_mode != FP8BLK_BSCALE_ROW128) return FP8BLK_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BLK_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return FP8BLK_OK;
  if (K == 0) return FP8BLK_ERR_INVALID_ARG;
  if (!matrix_ok(A, M, K, lda, 1) || !matrix_ok(C, M, N, ldc, ob ? 2 : 4)) return FP8BLK_ERR_INVALID_ARG;
  if (opB == FP8BLK_OP_N ? !matrix_ok(B, K, N, ldb, 1) : !matrix_ok(B, N, K, ldb, 1)) return FP8BLK_ERR_INVALID_ARG;
  if (lda >= kMaxPitch || ldb >= kMaxPitch) return FP8BLK_ERR_UNSUPPORTED;
  const int64_t G = K / 128;
  const int64_t NB = ceil_div(N, 128);
  if (!vec_ok(sA, G * M)) return FP8BLK_ERR_INVALID_ARG;
  int64_t sB_ld;
  if (bscale_mode == FP8BLK_BSCALE_ROW128) {
    if (!vec_ok(sB, G * N)) return FP8BLK_ERR_INVALID_ARG;
    sB_ld = N;
  } else {
    if (!vec_ok(sB, G * NB)) return FP8BLK_ERR_INVALID_ARG;
    sB_ld = opB == FP8BLK_OP_N ? NB : G;
  }
  hipStream_t st = as_stream(stream);
  const bool t = opB == FP8BLK_OP_T;
  // Split K when a large enough workspace is given and the tiles alone
  // cannot fill the GPU; otherwise one pass writes C directly.
  int64_t S = splitk_count(M, N, K);
  float* partials = nullptr;
  if (S > 1) {
    if (workspace != nullptr && workspace_bytes >= splitk_bytes(M, N, K) && aligned(workspace, 16))
      partials = static_cast<float*>(workspace);
    else if (strict)
      return FP8BLK_ERR_UNSUPPORTED;
    else
      S = 1;
  }
  // 256x256 tiles (or 224x256, see use_tile224) when they give at least
  // half a wave of workgroups over the 256 CUs, 128x128 tiles otherwise.
  const int64_t big_tiles = ceil_div(M, BigCfg::BM) * ceil_div(N, BigCfg::BN);
  const bool t224 = big_tiles >= 128 && use_tile224(M, N);
  if (bscale_mode == FP8BLK_BSCALE_ROW128) {
    if (t224)
      return dispatch_dense<Big224Cfg, true>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
    if (big_tiles >= 128)
      return dispatch_dense<BigCfg, true>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
    return dispatch_dense<SmallCfg, true>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
  }
  if (t224)
    return dispatch_dense<Big224Cfg, false>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
  if (big_tiles >= 128)
    return dispatch_dense<BigCfg, false>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
  return dispatch_dense<SmallCfg, false>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, C, ldc, ob, partials, S, st);
}

extern "C" fp8blk_status_t fp8blk_gemm_fp8_blockscaled(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
                                                       const float* sA, const uint8_t* B, int64_t ldb, int opB,
                                                       const float* sB, int bscale_mode, void* C, int64_t ldc,
                                                       void* workspace, size_t workspace_bytes, void* stream) {
  return gemm_dense(M, N, K, A, lda, sA, B, ldb, opB, sB, bscale_mode, C, ldc, workspace, workspace_bytes, false,
                    stream);
}

// ---- The same GEMM without any allocation --------------------------------
// For callers that cannot allocate (code under graph capture, serving loops,
// harnesses that forbid it): the split-K partials live in `scratch`, a
// file-scope device array of FP8BLK_NOALLOC_SCRATCH_BYTES that each GPU holds
// for the life of the process.  Its device address is looked up once per
// device (hipGetSymbolAddress with that device current) and kept; host code
// passes only that address to the kernels, never the array's name.
static __device__ __align__(256) float scratch[FP8BLK_NOALLOC_SCRATCH_BYTES / sizeof(float)];

static float* scratch_on_current_device() {
  static std::mutex mu;
  static std::atomic<float*> ptrs[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return nullptr;
  float* p = ptrs[dev].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  std::lock_guard<std::mutex> lock(mu);
  p = ptrs[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    void* q = nullptr;
    if (hipGetSymbolAddress(&q, HIP_SYMBOL(scratch)) != hipSuccess || q == nullptr) return nullptr;
    p = static_cast<float*>(q);
    ptrs[dev].store(p, std::memory_order_release);
  }
  return p;
}

extern "C" fp8blk_status_t fp8blk_gemm_fp8_blockscaled_noalloc(int64_t M, int64_t N, int64_t K, const uint8_t* A,
                                                               int64_t lda, const float* sA, const uint8_t* B,
                                                               int64_t ldb, int opB, const float* sB, int bscale_mode,
                                                               void* C, int64_t ldc, void* stream) {
  // Shapes whose partials would not fit are rejected before anything is
  // looked up or enqueued (the split count is the workspace entry point's).
  if (M > 0 && N > 0 && K > 0 && K % 128 == 0 && splitk_bytes(M, N, K) > FP8BLK_NOALLOC_SCRATCH_BYTES)
    return FP8BLK_ERR_UNSUPPORTED;
  float* ws = nullptr;
  if (M > 0 && N > 0 && K > 0 && K % 128 == 0 && splitk_bytes(M, N, K) > 0) {
    ws = scratch_on_current_device();
    if (ws == nullptr) return FP8BLK_ERR_LAUNCH;
  }
  return gemm_dense(M, N, K, A, lda, sA, B, ldb, opB, sB, bscale_mode, C, ldc, ws,
                    ws != nullptr ? (size_t)FP8BLK_NOALLOC_SCRATCH_BYTES : 0, true, stream);
}

// Dense GEMM with the output quantized on store (1x128 tiles along each row
// of the BF16-rounded result); block-scaled B only, never split.
template <class CFG, bool OPB_T, bool P2>
static fp8blk_status_t launch_q(int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda, const float* sA,
                                const uint8_t* B, int64_t ldb, const float* sB, int64_t sB_ld, uint8_t* Q, int64_t ldq,
                                float* sQ, bool qpow2, hipStream_t st) {
  const int64_t tiles_m = ceil_div(M, CFG::BM), tiles_n = ceil_div(N, CFG::BN);
  const int64_t blocks = tiles_m * tiles_n;
  if (blocks > 0x7FFFFFFF) return FP8BLK_ERR_UNSUPPORTED;
  const int per = (int)(K / 128);
  if (qpow2)
    hipLaunchKernelGGL((k_gemm<CFG, OPB_T, false, P2, OUT_Q_POW2>), dim3((unsigned)blocks), dim3(CFG::NT), 0, st, M, N,
                       K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, tiles_m, tiles_n, nullptr, per, sQ);
  else
    hipLaunchKernelGGL((k_gemm<CFG, OPB_T, false, P2, OUT_Q>), dim3((unsigned)blocks), dim3(CFG::NT), 0, st, M, N, K,
                       A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, tiles_m, tiles_n, nullptr, per, sQ);
  return launch_status();
}

template <class CFG>
static fp8blk_status_t dispatch_q(bool t, bool p2, int64_t M, int64_t N, int64_t K, const uint8_t* A, int64_t lda,
                                  const float* sA, const uint8_t* B, int64_t ldb, const float* sB, int64_t sB_ld,
                                  uint8_t* Q, int64_t ldq, float* sQ, bool qpow2, hipStream_t st) {
  if (p2) {
    if (t) return launch_q<CFG, true, true>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, sQ, qpow2, st);
    return launch_q<CFG, false, true>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, sQ, qpow2, st);
  }
  if (t) return launch_q<CFG, true, false>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, sQ, qpow2, st);
  return launch_q<CFG, false, false>(M, N, K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, sQ, qpow2, st);
}

extern "C" fp8blk_status_t fp8blk_gemm_fp8_blockscaled_q1x128(int64_t M, int64_t N, int64_t K, const uint8_t* A,
                                                              int64_t lda, const float* sA, const uint8_t* B,
                                                              int64_t ldb, int opB, const float* sB, uint8_t* Q,
                                                              int64_t ldq, float* sQ, uint32_t qflags, void* stream) {
  if (M < 0 || N < 0 || K < 0) return FP8BLK_ERR_INVALID_ARG;
  if (qflags & ~FP8BLK_SCALE_POW2) return FP8BLK_ERR_INVALID_ARG;
  const bool p2 = (opB & FP8BLK_GEMM_POW2_SCALES) != 0;
  opB &= ~FP8BLK_GEMM_POW2_SCALES;
  if (opB != FP8BLK_OP_N && opB != FP8BLK_OP_T) return FP8BLK_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BLK_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return FP8BLK_OK;
  if (K == 0) return FP8BLK_ERR_INVALID_ARG;
  if (!matrix_ok(A, M, K, lda, 1) || !matrix_ok(Q, M, N, ldq, 1)) return FP8BLK_ERR_INVALID_ARG;
  if (opB == FP8BLK_OP_N ? !matrix_ok(B, K, N, ldb, 1) : !matrix_ok(B, N, K, ldb, 1)) return FP8BLK_ERR_INVALID_ARG;
  if (lda >= kMaxPitch || ldb >= kMaxPitch) return FP8BLK_ERR_UNSUPPORTED;
  const int64_t G = K / 128, NB = ceil_div(N, 128);
  if (!vec_ok(sA, G * M) || !vec_ok(sB, G * NB) || !vec_ok(sQ, NB * M)) return FP8BLK_ERR_INVALID_ARG;
  const int64_t sB_ld = opB == FP8BLK_OP_N ? NB : G;
  const bool t = opB == FP8BLK_OP_T, qpow2 = (qflags & FP8BLK_SCALE_POW2) != 0;
  hipStream_t st = as_stream(stream);
  const int64_t big_tiles = ceil_div(M, BigCfg::BM) * ceil_div(N, BigCfg::BN);
  if (big_tiles >= 128) return dispatch_q<BigCfg>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, sQ, qpow2, st);
  return dispatch_q<SmallCfg>(t, p2, M, N, K, A, lda, sA, B, ldb, sB, sB_ld, Q, ldq, sQ, qpow2, st);
}

extern "C" fp8blk_status_t fp8blk_grouped_gemm_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t N, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, void* C, int64_t ldc, void* workspace, size_t workspace_bytes,
    void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  // 256 x 256 tiles on the row-pipelined loop.  With 256 experts of mean
  // 256 rows (skewed), 256-row tiles pad the experts' row ranges more than
  // 128-row tiles (64 % against 79 % useful rows), but each group's copies
  // feed four times the MFMA work, and the copies, not the matrix cores,
  // bound these kernels: measured against 128 x 128 tiles (interleaved, one
  // box, bitwise identical, both before the XCD balance of the kernel) MoE
  // up 3.32 / 3.50 ms, down 2.08 / 2.16 ms, down Dgrad 1.72 / 1.71 ms.
  using CFG = BigCfg;
  if (G < 0 || M_total < 0 || N < 0 || K < 0 || max_group_rows < 0) return FP8BLK_ERR_INVALID_ARG;
  const bool p2 = (opB & FP8BLK_GEMM_POW2_SCALES) != 0;
  const int ob = (opB & FP8BLK_GEMM_OUT_BF16) != 0;
  opB &= ~(FP8BLK_GEMM_POW2_SCALES | FP8BLK_GEMM_OUT_BF16);
  if (opB != FP8BLK_OP_N && opB != FP8BLK_OP_T) return FP8BLK_ERR_INVALID_ARG;
  if (K % 128 != 0) return FP8BLK_ERR_INVALID_ARG;
  if (G == 0 || M_total == 0 || N == 0) return FP8BLK_OK;
  if (K == 0 || group_offsets == nullptr || !aligned(group_offsets, 4)) return FP8BLK_ERR_INVALID_ARG;
  if (!matrix_ok(A, M_total, K, lda, 1) || !matrix_ok(C, M_total, N, ldc, ob ? 2 : 4)) return FP8BLK_ERR_INVALID_ARG;
  const int64_t Gk = K / 128, NB = ceil_div(N, 128);
  const int64_t brows = opB == FP8BLK_OP_N ? K : N, bcols = opB == FP8BLK_OP_N ? N : K;
  if (!matrix_ok(B, brows, bcols, ldb, 1)) return FP8BLK_ERR_INVALID_ARG;
  if (lda >= kMaxPitch || ldb >= kMaxPitch) return FP8BLK_ERR_UNSUPPORTED;
  if (strideB < brows * ldb || strideB % 16 != 0) return FP8BLK_ERR_INVALID_ARG;
  if (!vec_ok(sA, Gk * M_total) || !vec_ok(sB, Gk * NB)) return FP8BLK_ERR_INVALID_ARG;
  if (stride_sB < Gk * NB) return FP8BLK_ERR_INVALID_ARG;
  const int64_t sB_ld = opB == FP8BLK_OP_N ? NB : Gk;
  const int64_t tiles_n = ceil_div(N, CFG::BN);
  // Each expert adds at most one partial row tile.
  int64_t tiles_m = ceil_div(M_total, CFG::BM) + G;
  if (max_group_rows > 0) {
    const int64_t alt = G * ceil_div(max_group_rows, CFG::BM);
    if (alt < tiles_m) tiles_m = alt;
  }
  int64_t blocks = tiles_m * tiles_n;
  if (blocks == 0) return FP8BLK_OK;
  if (blocks % 8) blocks += 8 - blocks % 8;  // keep the XCD remap a bijection on the grid
  if (blocks > 0x7FFFFFFF) return FP8BLK_ERR_UNSUPPORTED;
  hipStream_t st = as_stream(stream);
#define FP8BLK_GROUPED_LAUNCH(T_, P2_, OB_)                                                                      \
  hipLaunchKernelGGL((k_grouped_gemm<CFG, T_, P2_, OB_>), dim3((unsigned)blocks), dim3(CFG::NT), 0, st, G,          \
                     group_offsets, M_total, N, K, A, lda, sA, B, ldb, strideB, sB, stride_sB, sB_ld, C, ldc, tiles_n)
#define FP8BLK_GROUPED_LAUNCH_OB(T_, P2_) \
  if (ob) FP8BLK_GROUPED_LAUNCH(T_, P2_, OUT_BF16); else FP8BLK_GROUPED_LAUNCH(T_, P2_, OUT_F32)
  if (opB == FP8BLK_OP_T) {
    if (p2) { FP8BLK_GROUPED_LAUNCH_OB(true, true); } else { FP8BLK_GROUPED_LAUNCH_OB(true, false); }
  } else {
    if (p2) { FP8BLK_GROUPED_LAUNCH_OB(false, true); } else { FP8BLK_GROUPED_LAUNCH_OB(false, false); }
  }
#undef FP8BLK_GROUPED_LAUNCH_OB
#undef FP8BLK_GROUPED_LAUNCH
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_grouped_wgrad_fp8_blockscaled(int64_t G, const int32_t* group_offsets, int64_t T,
                                                                int64_t M, int64_t N, const uint8_t* AT,
                                                                int64_t ldaT, const float* sA, const uint8_t* BT,
                                                                int64_t ldbT, const float* sB, uint32_t flags,
                                                                void* C, int64_t ldc, int64_t strideC,
                                                                void* stream) {
  // 128 x 128 tiles: the per-column scales of both operands (ROW128) need the
  // registers of the smaller tile.
  using CFG = RowCfg;
  if (G < 0 || T < 0 || M < 0 || N < 0) return FP8BLK_ERR_INVALID_ARG;
  if (flags & ~(uint32_t)(FP8BLK_GEMM_POW2_SCALES | FP8BLK_GEMM_OUT_BF16)) return FP8BLK_ERR_INVALID_ARG;
  const bool p2 = (flags & FP8BLK_GEMM_POW2_SCALES) != 0;
  const int ob = (flags & FP8BLK_GEMM_OUT_BF16) != 0;
  if (G == 0 || M == 0 || N == 0) return FP8BLK_OK;
  const int64_t slots = fp8blk_token_group_slots(T, G);
  if (group_offsets == nullptr || !aligned(group_offsets, 4)) return FP8BLK_ERR_INVALID_ARG;
  if (T > 0) {  // with no tokens the operands are not read (every dW_e = 0)
    if (!matrix_ok(AT, M, 128 * slots, ldaT, 1) || !matrix_ok(BT, N, 128 * slots, ldbT, 1))
      return FP8BLK_ERR_INVALID_ARG;
    if (!vec_ok(sA, slots * M) || !vec_ok(sB, slots * N)) return FP8BLK_ERR_INVALID_ARG;
  }
  if (!matrix_ok(C, M, N, ldc, ob ? 2 : 4) || strideC < M * ldc || strideC % (ob ? 8 : 4) != 0)
    return FP8BLK_ERR_INVALID_ARG;
  if (ldaT >= kMaxPitch || ldbT >= kMaxPitch || slots > 0x7FFFFFFF / 2) return FP8BLK_ERR_UNSUPPORTED;
  const int64_t tiles_m = ceil_div(M, CFG::BM), tiles_n = ceil_div(N, CFG::BN);
  const int64_t blocks = G * tiles_m * tiles_n;
  if (blocks > 0x7FFFFFFF) return FP8BLK_ERR_UNSUPPORTED;
  hipStream_t st = as_stream(stream);
#define FP8BLK_WGRAD_LAUNCH(P2_, OB_)                                                                             \
  hipLaunchKernelGGL((k_grouped_wgrad<CFG, P2_, OB_>), dim3((unsigned)blocks), dim3(CFG::NT), 0, st, group_offsets, M, \
                     N, AT, ldaT, sA, BT, ldbT, sB, C, ldc, strideC, tiles_m, tiles_n)
  if (p2) {
    if (ob) FP8BLK_WGRAD_LAUNCH(true, OUT_BF16); else FP8BLK_WGRAD_LAUNCH(true, OUT_F32);
  } else {
    if (ob) FP8BLK_WGRAD_LAUNCH(false, OUT_BF16); else FP8BLK_WGRAD_LAUNCH(false, OUT_F32);
  }
#undef FP8BLK_WGRAD_LAUNCH
  return launch_status();
}
