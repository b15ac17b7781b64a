// Gated feed-forward block in block-scaled FP8 (gfx950): gate and up projection,
// activation and product in one GEMM, and the gradient of the same.
//
//   u = A B (B's first H columns the gate, its last H the up projection),
//   h = act(u_g) u_u,   act(g) = g sigmoid(z(g)),
//   z = g (SiLU) or (8 / pi)^(1/2) (g + 0.044715 g^3) (GELU in its tanh form);
//   dh = A B (A the gradient of the down projection's output, B its weights),
//   p = sigmoid(z):  du_u = dh g p,   du_g = dh u_u (p + g p (1 - p) dz/dg).
//
// The GEMMs are those of gemm_tile.h, FP8 in every direction [p1¶3], and what
// the next one reads is quantized on the way out [p2¶4].
// Citations [pN¶k]: N-th page of the source collection, k-th paragraph
// (p1 = xn--9g3bo1gtkw0l8ubf92bgle.kr wr_id 85187, p2 = inprokorea.com wr_id
// 735329).
//
// Forward: a 256 x 256 tile holds 128 gate columns and the 128 up columns that
// go with them (GATED in gemm_tile.h), in such an order that a lane's four
// column tiles are two of gate and the two of up beside them: the product is
// formed in registers, and the 128 columns of h are one 1x128 scale group.
// Gradient: the plain tile of dh, whose lanes read u where their results lie.
// Both are bound as the GEMMs are, by moving operands; the FP32 results (u or
// dh, half a GB for 65536 rows of 2048) never reach memory.
//
// Measured, K = 7168 and H = 2048: forward with codes out, 8192 rows 220 us
// (2.19 PFLOP/s, the GEMMs' rate), 65536 rows of 256 experts with u and codes 2.83
// ms (the GEMM of the same operands alone, FP32 out, 2.84); gradient, 8192 rows
// 134 us (1.80 PFLOP/s), 65536 rows of 256 experts with codes 1.81 ms (plain GEMM
// 1.46).  The gradient's codes cost 24 us at 8192 rows, one round of tiles with
// nothing to cover its end (a quantizer of its own 19 and a launch), and 90 us for
// the experts (148).
#include <algorithm>
#include <cmath>

#include "../../include/libfp8blk_train.h"
#include "gemm_tile.h"
#include "layer_device.h"
#include "layer_host.h"

namespace fp8blk {

// The activation's sigmoid argument, and its derivative.
template <bool GELU>
__device__ __forceinline__ float act_arg(float g) {
  constexpr float k = 1.5957691216057308f;  // (8 / pi)^(1/2)
  return GELU ? k * __builtin_fmaf(0.044715f * g * g, g, g) : g;
}
template <bool GELU>
__device__ __forceinline__ float act_slope(float g) {
  constexpr float k = 1.5957691216057308f;
  return GELU ? k * __builtin_fmaf(0.134145f * g, g, 1.0f) : 1.0f;
}
// 1 / (1 + e^-z) by the hardware's 2^x and reciprocal, one unit in the last place
// (2^-23) each.  e^-z is off by that and by 2^-24 |z| for each of the two
// roundings before it, to which GELU's argument adds up to six; the sum and the
// reciprocal add 3 x 2^-24: within ((1 - p) (8 |z| + 2) + 3) 2^-24 of itself in all
// (BF16 has 2^-8), and 0 where e^-z passes FP32's range, z < -88.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// What a forward tile or row writes; each part may be missing.
struct GatedOut {
  uint16_t* u;  // [.][2H]
  int64_t ldu;
  uint16_t* h;  // [.][H]
  int64_t ldh;
  uint8_t* q;  // [.][H] codes of h
  int64_t ldq;
  float* s;  // [H / 128][s_ld]
  int64_t s_ld;
  int gelu, pow2;
};
// ... and a gradient's.
struct GatedGradOut {
  const uint16_t* u;
  int64_t ldu;
  uint16_t* du;  // [.][2H]; may be u
  int64_t lddu;
  uint16_t* h;
  int64_t ldh;
  uint8_t* q;  // [.][2H] codes of du
  int64_t ldq;
  float* s;  // [2H / 128][s_ld]
  int64_t s_ld;
  int gelu, pow2;
};

// E4M3 codes of BF16 values (two to a word), as quantize_1x128 makes them.
template <bool POW2, int N>
__device__ __forceinline__ void encode_bf16(const uint32_t (&w)[N], uint32_t amax, uint32_t (&codes)[N / 2], float& s) {
  const TileScale ts = make_scale<POW2, true>(amax << 16);
  s = ts.s;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float x[4] = {bf16_lo(w[2 * i]), bf16_hi(w[2 * i]), bf16_lo(w[2 * i + 1]), bf16_hi(w[2 * i + 1])};
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = quotient_fast<POW2, true>(x[r], ts);
    if (__builtin_expect(ts.slow, 0)) {
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = quotient_slow(x[r], ts.s);
    }
    codes[i] = pack4_e4m3(y[0], y[1], y[2], y[3]);
  }
}

template <bool GELU>
__device__ __forceinline__ float gated(float g, float v) { return g * sigmoid(act_arg<GELU>(g)) * v; }

// dg, du and h of one value.  Where the sigmoid is 0 or 1 in FP32 the term with
// its slope is nothing, also where the cubic's slope overflows.
template <bool GELU>
__device__ __forceinline__ void gated_grad(float dh, float g, float v, float& dg, float& dv, float& h) {
  const float p = sigmoid(act_arg<GELU>(g));
  const float a = g * p, t = a * (1.0f - p);
  const float slope = t == 0.0f ? p : __builtin_fmaf(t, act_slope<GELU>(g), p);
  dv = dh * a;
  dg = dh * v * slope;
  h = a * v;
}

// Stores of a gated tile (see GatedOut).
template <class CFG>
struct GatedStore {
  GatedOut o;

  template <bool GELU>
  __device__ __forceinline__ void products(const v4f (&acc)[CFG::TM][CFG::TN], uint32_t (&hw)[CFG::TM][4]) const {
#pragma unroll
    for (int i = 0; i < CFG::TM; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = gated<GELU>(acc[i][j][r], acc[i][j + 2][r]);
        hw[i][2 * j] = bf16_pack(v[0], v[1]);
        hw[i][2 * j + 1] = bf16_pack(v[2], v[3]);
      }
    }
  }

  template <bool POW2>
  __device__ __forceinline__ void quantized(const TileArgs& t, const uint32_t (&hw)[CFG::TM][4], uint32_t* red) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / CFG::WAVES_N, wn = wave % CFG::WAVES_N, l16 = lane & 15, lq = lane >> 4;
    const int64_t col = t.n0 + wn * (CFG::WTN / 2) + 16 * (lq & 1);
#pragma unroll
    for (int i = 0; i < CFG::TM; i += 2) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t m = 0;
        const int at = wm * CFG::WTM + 16 * (i + k) + l16;
#pragma unroll
        for (int w = 0; w < CFG::WAVES_N; ++w) m = max(m, red[w * CFG::BM + at]);
        uint32_t two[2];
        float s;
        encode_bf16<POW2>(hw[i + k], m, two, s);
        c[2 * k] = two[0];
        c[2 * k + 1] = two[1];
        if (wn == 0 && lq == 0 && at < t.rows) o.s[(t.n0 >> 7) * o.s_ld + t.m0 + at] = s;
      }
      // Two row tiles of two column tiles each: lane row lq stores 16 columns of row tile i + lq / 2.
      transpose_rows4(c);
      const int64_t row = wm * CFG::WTM + 16 * (i + (lq >> 1)) + l16;
      if (row < t.rows)
        *reinterpret_cast<uint4*>(o.q + (t.m0 + row) * o.ldq + col) = make_uint4(c[0], c[1], c[2], c[3]);
    }
  }

  __device__ __forceinline__ void operator()(const TileArgs& t, v4f (&acc)[CFG::TM][CFG::TN], uint8_t* lds) const {
    constexpr int TM = CFG::TM, TN = CFG::TN;
    static_assert(TN == 4 && TM % 2 == 0 && CFG::WAVES_N * CFG::WTN == 256, "two gate and two up column tiles a wave");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / CFG::WAVES_N, wn = wave % CFG::WAVES_N, l16 = lane & 15, lq = lane >> 4;
    if (o.u != nullptr) {  // lane row lq takes column tile lq: gate, gate, up, up
      const int64_t col = t.n0 + wn * (CFG::WTN / 2) + 16 * (lq & 1) + (lq >> 1) * t.H;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          lo[j] = bf16_pack(acc[i][j][0], acc[i][j][1]);
          hi[j] = bf16_pack(acc[i][j][2], acc[i][j][3]);
        }
        transpose_rows4(lo);
        transpose_rows4(hi);
        const int64_t row = wm * CFG::WTM + 16 * i + l16;
        if (row >= t.rows) continue;
        uint4* dst = reinterpret_cast<uint4*>(o.u + (t.m0 + row) * o.ldu + col);
        dst[0] = make_uint4(lo[0], hi[0], lo[1], hi[1]);
        dst[1] = make_uint4(lo[2], hi[2], lo[3], hi[3]);
      }
    }
    if (o.h == nullptr && o.q == nullptr) return;
    uint32_t hw[TM][4];
    if (o.gelu) products<true>(acc, hw);
    else products<false>(acc, hw);
    if (o.h != nullptr) {
      const int64_t col = t.n0 + wn * (CFG::WTN / 2) + 16 * (lq & 1);
#pragma unroll
      for (int i = 0; i < TM; i += 2) {
        uint32_t lo[4] = {hw[i][0], hw[i][2], hw[i + 1][0], hw[i + 1][2]};
        uint32_t hi[4] = {hw[i][1], hw[i][3], hw[i + 1][1], hw[i + 1][3]};
        transpose_rows4(lo);
        transpose_rows4(hi);
        const int64_t row = wm * CFG::WTM + 16 * (i + (lq >> 1)) + l16;
        if (row >= t.rows) continue;
        uint4* dst = reinterpret_cast<uint4*>(o.h + (t.m0 + row) * o.ldh + col);
        dst[0] = make_uint4(lo[0], hi[0], lo[1], hi[1]);
        dst[1] = make_uint4(lo[2], hi[2], lo[3], hi[3]);
      }
    }
    if (o.q == nullptr) return;
    uint32_t* red = reinterpret_cast<uint32_t*>(lds);  // the maximum of every row over each wave's columns
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) m = abs_max_bits(m, hw[i][k]);
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lq == 0) red[wn * CFG::BM + wm * CFG::WTM + 16 * i + l16] = m;
    }
    __syncthreads();
    if (o.pow2) quantized<true>(t, hw, red);
    else quantized<false>(t, hw, red);
  }
};

// Stores of a tile of dh (see GatedGradOut).
template <class CFG>
struct GatedGradStore {
  GatedGradOut o;

  struct Row {  // what a lane reads of u: 16 gate values and the 16 up values beside them
    uint4 g[2], v[2];
  };
  __device__ __forceinline__ Row read(const TileArgs& t, int64_t row, int64_t col) const {
    Row r{};
    if (row >= t.rows || col >= t.N) return r;
    const uint16_t* p = o.u + (t.m0 + row) * o.ldu + col;
    r.g[0] = reinterpret_cast<const uint4*>(p)[0];
    r.g[1] = reinterpret_cast<const uint4*>(p)[1];
    r.v[0] = reinterpret_cast<const uint4*>(p + t.H)[0];
    r.v[1] = reinterpret_cast<const uint4*>(p + t.H)[1];
    return r;
  }

  // Row tile i: du in BF16 pairs, dg[8] then dv[8], in place of the lane's 16 values of dh.
  template <bool GELU>
  __device__ __forceinline__ void gradients(const TileArgs& t, v4f (&acc)[CFG::TN], const Row& u, int64_t row,
                                            int64_t col) const {
    // Afterwards d[r][k] is column 4k + r of the 16 from col.
    uint32_t d[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int j = 0; j < 4; ++j) d[r][j] = __float_as_uint(acc[j][r]);
      transpose_rows4(d[r]);
    }
    const uint32_t g[8] = {u.g[0].x, u.g[0].y, u.g[0].z, u.g[0].w, u.g[1].x, u.g[1].y, u.g[1].z, u.g[1].w};
    const uint32_t v[8] = {u.v[0].x, u.v[0].y, u.v[0].z, u.v[0].w, u.v[1].x, u.v[1].y, u.v[1].z, u.v[1].w};
    uint32_t dg[8], dv[8], h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // columns 2k and 2k + 1
      float a[2], b[2], c[2];
      gated_grad<GELU>(__uint_as_float(d[2 * (k & 1)][k >> 1]), bf16_lo(g[k]), bf16_lo(v[k]), a[0], b[0], c[0]);
      gated_grad<GELU>(__uint_as_float(d[2 * (k & 1) + 1][k >> 1]), bf16_hi(g[k]), bf16_hi(v[k]), a[1], b[1], c[1]);
      dg[k] = bf16_pack(a[0], a[1]);
      dv[k] = bf16_pack(b[0], b[1]);
      h[k] = bf16_pack(c[0], c[1]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      acc[k >> 2][k & 3] = __uint_as_float(dg[k]);
      acc[2 + (k >> 2)][k & 3] = __uint_as_float(dv[k]);
    }
    if (row >= t.rows || col >= t.N) return;
    auto put = [](uint16_t* p, const uint32_t (&w)[8]) {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    };
    if (o.du != nullptr) {
      uint16_t* p = o.du + (t.m0 + row) * o.lddu + col;
      put(p, dg);
      put(p + t.H, dv);
    }
    if (o.h != nullptr) put(o.h + (t.m0 + row) * o.ldh + col, h);
  }

  template <bool POW2>
  __device__ __forceinline__ void quantized(const TileArgs& t, const v4f (&acc)[CFG::TM][CFG::TN], const uint32_t* red,
                                            int64_t col) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / CFG::WAVES_N, wn = wave % CFG::WAVES_N, l16 = lane & 15, lq = lane >> 4;
#pragma unroll
    for (int i = 0; i < CFG::TM; ++i) {
      const int at = wm * CFG::WTM + 16 * i + l16;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t* mine = red + half * CFG::WAVES_N * CFG::BM + at;
        uint32_t w[8], c[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(acc[i][2 * half + (k >> 2)][k & 3]);
        float s;
        encode_bf16<POW2>(w, max(mine[wn * CFG::BM], mine[(wn ^ 1) * CFG::BM]), c, s);
        if (at >= t.rows || col >= t.N) continue;
        const int64_t out = col + half * t.H;
        *reinterpret_cast<uint4*>(o.q + (t.m0 + at) * o.ldq + out) = make_uint4(c[0], c[1], c[2], c[3]);
        if ((wn & 1) == 0 && lq == 0) o.s[(out >> 7) * o.s_ld + t.m0 + at] = s;
      }
    }
  }

  __device__ __forceinline__ void operator()(const TileArgs& t, v4f (&acc)[CFG::TM][CFG::TN], uint8_t* lds) const {
    constexpr int TM = CFG::TM, TN = CFG::TN;
    static_assert(TN == 4 && CFG::WTN == 64, "a 128-column scale group spans two waves");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / CFG::WAVES_N, wn = wave % CFG::WAVES_N, l16 = lane & 15, lq = lane >> 4;
    const int64_t col = t.n0 + wn * CFG::WTN + 16 * lq, row0 = wm * CFG::WTM + l16;
    Row u = read(t, row0, col);
#pragma unroll
    for (int i = 0; i < TM; ++i) {  // the next rows of u are on their way while these are worked on
      const Row next = i + 1 < TM ? read(t, row0 + 16 * (i + 1), col) : u;
      if (o.gelu) gradients<true>(t, acc[i], u, row0 + 16 * i, col);
      else gradients<false>(t, acc[i], u, row0 + 16 * i, col);
      u = next;
    }
    if (o.q == nullptr) return;
    uint32_t* red = reinterpret_cast<uint32_t*>(lds);  // gate's, then up's row maxima over each wave's columns
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = abs_max_bits(m, __float_as_uint(acc[i][2 * half + (k >> 2)][k & 3]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lq == 0) red[(half * CFG::WAVES_N + wn) * CFG::BM + row0 + 16 * i] = m;
      }
    __syncthreads();
    if (o.pow2) quantized<true>(t, acc, red, col);
    else quantized<false>(t, acc, red, col);
  }
};

// Operands of either product, dense (G = 0) or one B for every expert.
struct GatedArgs {
  int64_t G;
  const int32_t* offsets;
  int64_t M, H, N, K;  // N: B's columns (2H forward, H in the gradient)
  const uint8_t* A;
  int64_t lda;
  const float* sA;
  const uint8_t* B;
  int64_t ldb, strideB;
  const float* sB;
  int64_t stride_sB, sB_ld;
  int64_t tiles_m, tiles_n;
};

// The workgroup's tile of BN columns of a tile row, or (GATED) BN / 2 of either half; false for none.
template <class CFG, bool GROUPED, bool GATED>
__device__ __forceinline__ bool gated_tile(const GatedArgs& a, TileArgs& t) {
  int64_t e = 0, tn, m0, rows;
  if (GROUPED) {
    if (!grouped_tile<CFG>(a.offsets, a.G, a.tiles_n, e, tn, m0, rows)) return false;
  } else {
    int64_t tm;
    tile_of(blockIdx.x, gridDim.x, a.tiles_m, a.tiles_n, tm, tn);
    m0 = tm * CFG::BM;
    rows = (a.M - m0) < CFG::BM ? (a.M - m0) : CFG::BM;
  }
  t.A = a.A + m0 * a.lda;
  t.lda = a.lda;
  t.rows = rows;
  t.sA = a.sA + m0;
  t.sA_ld = a.M;
  t.B = a.B + e * a.strideB;
  t.ldb = a.ldb;
  t.n0 = tn * (GATED ? CFG::BN / 2 : CFG::BN);
  t.N = a.N;
  t.sB = a.sB + e * a.stride_sB;
  t.sB_ld = a.sB_ld;
  t.m0 = m0;
  t.K = a.K;
  t.g0 = 0;
  t.g1 = (int)(a.K / 128);
  t.H = a.H;
  return true;
}

template <class CFG, bool GROUPED, bool OPB_T, bool P2>
__global__ __launch_bounds__(CFG::NT) void k_gated_gemm(GatedArgs a, GatedOut o) {
  FP8BLK_DECLARE_STAGES(CFG);
  TileArgs t;
  if (!gated_tile<CFG, GROUPED, true>(a, t)) return;
  gemm_tile<CFG, OPB_T, false, P2, OUT_OWN, GROUPED, false, true>(t, s_ops0, s_ops1, s_sc0, s_sc1, GatedStore<CFG>{o});
}

template <class CFG, bool GROUPED, bool OPB_T, bool P2>
__global__ __launch_bounds__(CFG::NT) void k_gated_gemm_backward(GatedArgs a, GatedGradOut o) {
  FP8BLK_DECLARE_STAGES(CFG);
  TileArgs t;
  if (!gated_tile<CFG, GROUPED, false>(a, t)) return;
  gemm_tile<CFG, OPB_T, false, P2, OUT_OWN, GROUPED, false, false>(t, s_ops0, s_ops1, s_sc0, s_sc1,
                                                                   GatedGradStore<CFG>{o});
}

// --- tiles of fewer rows --------------------------------------------------------
// With fewer than 256 rows a K group is worked on in less time than its
// successor needs to arrive, so these tiles keep three or four LDS stages, all
// but one of them on their way.  The matrix cores wait anyhow: power-of-two
// scales take the same path (the scaled product is exact, and so the sum is the
// MFMA's own).
template <class CFG_, int STAGES_>
struct Deep {
  using CFG = CFG_;
  static constexpr int STAGES = STAGES_;
  uint8_t ops[STAGES][CFG::BUF_BYTES];
  float sc[STAGES][CFG::SC_FLOATS];
  static_assert(STAGES * (CFG::BUF_BYTES + CFG::SC_FLOATS * 4) <= 160 * 1024, "LDS capacity");
};
using MidDeep = Deep<TileCfg<2, 4, 4, 4>, 3>;  // 128 x 256, 49 KB a stage
using LowDeep = Deep<TileCfg<2, 4, 2, 4>, 3>;  // 64 x 256, 41 KB
using FewDeep = Deep<TileCfg<1, 8, 2, 2>, 4>;  // 32 x 256, 37 KB

// All but the newest `groups` of at most MOST groups of L copies each have landed.
template <int MOST, int L>
__device__ __forceinline__ void wait_groups(int groups) {
  if constexpr (MOST == 0) {
    wait_vmcnt<0>();
  } else {
    if (groups >= MOST) wait_vmcnt<MOST * L>();
    else wait_groups<MOST - 1, L>(groups);
  }
}

template <class D, bool OPB_T, bool GATED, bool ONCE = false>
__device__ __forceinline__ void deep_loop(const TileArgs& t, D& lds, v4f (&acc)[D::CFG::TM][D::CFG::TN]) {
  using CFG = typename D::CFG;
  using Plan = CopyPlan<CFG, OPB_T, false, GATED>;
  constexpr int TM = CFG::TM, TN = CFG::TN, ST = D::STAGES;
  const int lane = threadIdx.x & 63, l16 = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / CFG::WAVES_N, wn = wave % CFG::WAVES_N;
  const int blk = wave < CFG::S_BLOCKS ? wave : 0;
  // Whether this wave copies rows of A (a partial copy iteration: only where it has valid rows).
  const bool with_a = !CFG::A_PARTIAL || (int)t.rows > wave * 8;
  static_assert(!CFG::A_PARTIAL || CFG::A_ITERS == 1, "the copies of a wave are counted");
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  Plan plan;
  plan.init(t);
  const uint32_t scoff = plan.sc_offset(t);
  GroupCursor<CFG, OPB_T, false, GATED> cur;
  cur.init(t, t.g0, blk * 64 < CFG::BMP);
  int into = 0;  // the stage of the next group to copy
  auto issue = [&]() {
    issue_copies<CFG, OPB_T, false, false, GATED, ONCE>(t, plan, scoff, cur.ra(true), cur.rb(true), cur.rs(true), 0,
                                                        Plan::LOADS, lds.ops[into], lds.sc[into], wave, blk);
    cur.advance();
    into = into + 1 < ST ? into + 1 : 0;
  };
  const int groups = t.g1 - t.g0;
  for (int g = 0; g < groups && g < ST; ++g) issue();
  int from = 0;
  for (int g = 0; g < groups; ++g) {
    // Groups g + 1 .. are still on their way: ST - 1 of them at first, then one fewer, as a
    // stage is filled again only once every wave has left it.
    const int newer = min(groups - 1 - g, g == 0 ? ST - 1 : ST - 2);
    if (with_a) wait_groups<ST - 1, Plan::LOADS>(newer);
    else wait_groups<ST - 1, Plan::LOADS - 1>(newer);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    if (g > 0 && g + ST - 1 < groups) issue();
    const uint8_t *As = lds.ops[from], *Bs = As + CFG::A_BYTES;
    const float* sc = lds.sc[from];
    from = from + 1 < ST ? from + 1 : 0;
    auto kmaj = [&](const uint8_t* base, int r) {
      const uint4 lo = *reinterpret_cast<const uint4*>(base + kmaj_off(r, 2 * lq));
      const uint4 hi = *reinterpret_cast<const uint4*>(base + kmaj_off(r, 2 * lq + 1));
      return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    v8i bf[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int ncol = wn * CFG::WTN + 16 * j;
      if (OPB_T) {
        bf[j] = kmaj(Bs, ncol + l16);
      } else {
        v2i part[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          part[r] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_v2i*)(Bs + nmaj_off<CFG::BN>(32 * lq + 8 * r + (l16 >> 1), ncol >> 4) + 8 * (l16 & 1)));
        bf[j] = v8i{part[0][0], part[0][1], part[1][0], part[1][1], part[2][0], part[2][1], part[3][0], part[3][1]};
      }
    }
    const float4 sa4 = *reinterpret_cast<const float4*>(sc + wm * CFG::WTMP + l16 * CFG::TMP);
    static_assert(TM <= 4, "four row scales");
    const float sa[4] = {sa4.x, sa4.y, sa4.z, sa4.w};
    const int block = wn * CFG::WTN / 128;
    const float sb[2] = {sc[CFG::BMP + (GATED ? 0 : block)], sc[CFG::BMP + (GATED ? 1 : block)]};
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const v8i af = kmaj(As, wm * CFG::WTM + 16 * i + l16);
      v4f p[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j)
        p[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bf[j], af, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 127, 0, 127);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const float f = sa[i] * sb[j < TN / 2 ? 0 : 1];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[j][r], f, acc[i][j][r]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Few rows, or experts of few rows: bound by the weights' way from memory.  128
// rows for 79 of 256 experts of 7168 x 4096 take 367 us for 2.3 GB (6.3 TB/s;
// reads alone reach 7.0); 777 rows of 2048 x 2816 16 us, a launch and 16 K groups
// of one tile after the other.
template <class D, bool GROUPED, bool OPB_T, bool ONCE>
__global__ __launch_bounds__(D::CFG::NT) void k_gated_gemm_deep(GatedArgs a, GatedOut o) {
  __shared__ __align__(16) D lds;
  TileArgs t;
  if (!gated_tile<typename D::CFG, GROUPED, true>(a, t)) return;
  v4f acc[D::CFG::TM][D::CFG::TN];
  deep_loop<D, OPB_T, true, ONCE>(t, lds, acc);
  GatedStore<typename D::CFG>{o}(t, acc, lds.ops[0]);
}

template <class D, bool GROUPED, bool OPB_T, bool ONCE>
__global__ __launch_bounds__(D::CFG::NT) void k_gated_gemm_backward_deep(GatedArgs a, GatedGradOut o) {
  __shared__ __align__(16) D lds;
  TileArgs t;
  if (!gated_tile<typename D::CFG, GROUPED, false>(a, t)) return;
  v4f acc[D::CFG::TM][D::CFG::TN];
  deep_loop<D, OPB_T, false, ONCE>(t, lds, acc);
  GatedGradStore<typename D::CFG>{o}(t, acc, lds.ops[0]);
}

// FP32 partial products [split][M][N] of K groups [split * per, ...): 16 rows of
// 7168 x 4096 in 14 parts take 7.6 us for 29 MB of weights (and the join 2.0, see
// below), of which the launch and the first copies' way are half.
template <class D, bool OPB_T, bool GATED>
__global__ __launch_bounds__(D::CFG::NT) void k_gated_partial(GatedArgs a, float* __restrict__ partials, int per) {
  using CFG = typename D::CFG;
  __shared__ __align__(16) D lds;
  TileArgs t;
  gated_tile<CFG, false, GATED>(a, t);
  t.g0 = blockIdx.y * per;
  t.g1 = min(t.g0 + per, (int)(a.K / 128));
  v4f acc[CFG::TM][CFG::TN];
  deep_loop<D, OPB_T, GATED>(t, lds, acc);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, lq = lane >> 4;
  const int wm = wave / CFG::WAVES_N, wn = wave % CFG::WAVES_N;
  float* out = partials + ((int64_t)blockIdx.y * a.M + t.m0) * a.N;
#pragma unroll
  for (int i = 0; i < CFG::TM; ++i) {
    const int64_t row = wm * CFG::WTM + 16 * i + l16;
    if (row >= t.rows) continue;
#pragma unroll
    for (int j = 0; j < CFG::TN; ++j) {
      const int c = wn * CFG::WTN + 16 * j;
      const int64_t col = t.n0 + (GATED ? gated_column<CFG>(c, t.H) : c) + 4 * lq;
      if (col < t.N) *reinterpret_cast<v4f*>(out + row * t.N + col) = acc[i][j];
    }
  }
}

// --- the join of partial products -------------------------------------------
// A lane has four columns of h, 32 lanes a scale group of one row, and SLICES
// times 32 lanes share its partial products: slice k adds k, k + SLICES, ..,
// in that order, and the first slice adds the slices' sums.  With many parts
// each lane loads few of them (16 parts in one lane, unrolled, took 7 us for
// 128 columns of one row, most of it fetching the instructions; 8 slices 4).
template <int SLICES>
struct Join {
  int64_t m, c;  // row, first column
  bool first;    // whether this lane holds the sums in the end
  int slice;
  __device__ __forceinline__ Join(int64_t H) {
    slice = SLICES > 1 ? (int)threadIdx.x >> 5 : 0;
    const int64_t at = SLICES > 1 ? (int64_t)blockIdx.x * 32 + (threadIdx.x & 31) : (int64_t)blockIdx.x * 64 + threadIdx.x;
    m = (int64_t)((uint32_t)at / (uint32_t)(H / 4));  // fewer than 2^31 lanes: few rows
    c = (int64_t)((uint32_t)at % (uint32_t)(H / 4)) * 4;
    first = slice == 0;
  }
  // The sums of N columns' parts at p, p + other.
  template <int N>
  __device__ __forceinline__ void sum(const float* __restrict__ p, int64_t other, int S, int64_t step, v4f (&x)[N]) const {
    __shared__ v4f part[N][SLICES][32];
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int s = slice; s < S; s += SLICES)
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] += *reinterpret_cast<const v4f*>(p + s * step + n * other);
    if (SLICES == 1) return;
#pragma unroll
    for (int n = 0; n < N; ++n) part[n][slice][threadIdx.x & 31] = x[n];
    __syncthreads();
    if (!first) return;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int k = 1; k < SLICES; ++k) x[n] += part[n][k][threadIdx.x & 31];
  }
};
// The codes of four values of a tile that 32 lanes hold, and its scale.
__device__ __forceinline__ void put_codes(uint2 w, bool pow2, uint8_t* q, float* s) {
  const uint32_t m = row16_max(abs_max_bits(abs_max_bits(0, w.x), w.y));
  const auto o = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  const uint32_t p[2] = {w.x, w.y};
  uint32_t c[1];
  float scale;
  if (pow2) encode_bf16<true>(p, max(o[0], o[1]), c, scale);
  else encode_bf16<false>(p, max(o[0], o[1]), c, scale);
  *reinterpret_cast<uint32_t*>(q) = c[0];
  if ((threadIdx.x & 31) == 0) *s = scale;
}
__device__ __forceinline__ uint2 pack4(const float (&x)[4]) { return make_uint2(bf16_pack(x[0], x[1]), bf16_pack(x[2], x[3])); }

template <int SLICES>
__global__ __launch_bounds__(SLICES > 1 ? 32 * SLICES : 64) void k_gated_join(const float* __restrict__ partials, int S,
                                                                              int64_t M, int64_t H, GatedOut o) {
  const Join<SLICES> j(H);
  const int64_t m = j.m, c = j.c;
  if (m >= M) return;
  v4f u[2];
  j.template sum<2>(partials + m * 2 * H + c, H, S, M * 2 * H, u);
  if (!j.first) return;
  const v4f g = u[0], v = u[1];
  if (o.u != nullptr) {
    *reinterpret_cast<uint2*>(o.u + m * o.ldu + c) = make_uint2(bf16_pack(g[0], g[1]), bf16_pack(g[2], g[3]));
    *reinterpret_cast<uint2*>(o.u + m * o.ldu + H + c) = make_uint2(bf16_pack(v[0], v[1]), bf16_pack(v[2], v[3]));
  }
  float x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = o.gelu ? gated<true>(g[k], v[k]) : gated<false>(g[k], v[k]);
  const uint2 w = pack4(x);
  if (o.h != nullptr) *reinterpret_cast<uint2*>(o.h + m * o.ldh + c) = w;
  if (o.q != nullptr) put_codes(w, o.pow2, o.q + m * o.ldq + c, o.s + (c >> 7) * o.s_ld + m);
}

template <int SLICES>
__global__ __launch_bounds__(SLICES > 1 ? 32 * SLICES : 64) void k_gated_join_backward(const float* __restrict__ partials,
                                                                                       int S, int64_t M, int64_t H,
                                                                                       GatedGradOut o) {
  const Join<SLICES> j(H);
  const int64_t m = j.m, c = j.c;
  if (m >= M) return;
  const uint2 ug = *reinterpret_cast<const uint2*>(o.u + m * o.ldu + c);
  const uint2 uv = *reinterpret_cast<const uint2*>(o.u + m * o.ldu + H + c);
  v4f d[1];
  j.template sum<1>(partials + m * H + c, 0, S, M * H, d);
  if (!j.first) return;
  const float g[4] = {bf16_lo(ug.x), bf16_hi(ug.x), bf16_lo(ug.y), bf16_hi(ug.y)};
  const float v[4] = {bf16_lo(uv.x), bf16_hi(uv.x), bf16_lo(uv.y), bf16_hi(uv.y)};
  float dg[4], dv[4], h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (o.gelu) gated_grad<true>(d[0][k], g[k], v[k], dg[k], dv[k], h[k]);
    else gated_grad<false>(d[0][k], g[k], v[k], dg[k], dv[k], h[k]);
  }
  const uint2 wg = pack4(dg), wv = pack4(dv);
  if (o.du != nullptr) {
    *reinterpret_cast<uint2*>(o.du + m * o.lddu + c) = wg;
    *reinterpret_cast<uint2*>(o.du + m * o.lddu + H + c) = wv;
  }
  if (o.h != nullptr) *reinterpret_cast<uint2*>(o.h + m * o.ldh + c) = pack4(h);
  if (o.q != nullptr) {
    put_codes(wg, o.pow2, o.q + m * o.ldq + c, o.s + (c >> 7) * o.s_ld + m);
    put_codes(wv, o.pow2, o.q + m * o.ldq + H + c, o.s + ((H + c) >> 7) * o.s_ld + m);
  }
}

// Tiles of a dense product: 256, 128, 64 or 32 rows by 256 columns of B, and
// into how many parts K is split (1: fused, more: partial products, joined).
struct GatedForm {
  int rows;
  int64_t splits;
};

// The form that takes least time by what the forms take per K group and round
// over the compute units, in ns: fitted to 252 products (1 to 4096 rows, K 512
// to 7168, H 512 to 2048, either direction) measured in every form on one box,
// within 0.5 % of the best form on average and 10 % at worst (as for 168 others, of
// up to 30000 rows and H 4096).  Both sides, forward of K = 7168 and
// H = 2048 in us: 16 rows 64 fused 50, 32 in 14 parts 11.5; 128 rows 64 fused
// 51, 64 in 8 parts 16; 1024 rows 64 fused 57, 128 70, 64 in 2 parts 67; 2048
// rows 128 fused 74, 256 100, 64 103; 4096 rows 256 fused 102, 128 139.
inline GatedForm gated_form(int64_t M, int64_t N, int64_t K, bool gradient, bool may_split) {
  const int64_t n = ceil_div(N, 256), cus = device_cus(), G = K / 128;
  GatedForm best{256, 1};
  double least = INFINITY;
  auto fused = [&](int rows, int group) {
    const int64_t rounds = ceil_div(std::min<int64_t>(ceil_div(M, rows), 1 << 20) * std::min<int64_t>(n, 1 << 20), cus);
    const double ns = (gradient ? 5200 : 3300) + (double)group * G * rounds;
    if (ns < least) least = ns, best = {rows, 1};
  };
  fused(256, 1330);
  if (ceil_div(M, 256) * n > 4 * cus) return best;  // many rounds: the largest tile
  fused(128, 930);
  fused(64, 580);
  if (!may_split) return best;
  for (const int rows : {64, 32}) {
    const int64_t tiles = ceil_div(M, rows) * n;
    for (int64_t s = 2; s <= 16 && s <= G; ++s) {
      const int64_t per = ceil_div(G, s), S = ceil_div(G, per);
      const double ns = 5200.0 + (rows == 64 ? 470 : 420) * per * ceil_div(tiles * S, cus) + S * M * N * 3 / 2000;
      if (ns < least) least = ns, best = {rows, S};
    }
  }
  return best;
}

// Rows of the experts' tiles, by the mean number of rows: the less of a tile an
// expert fills, the more of it is wasted.  128 experts of 7168 x 4096 (and of
// the down projection's 2048 x 7168), skewed as a router's top 8 of them, 64 /
// 128 / 256 rows in us: mean 2 439 / - / 528 (gradient 240 / - / 298), 32 730 /
// 724 / 809 (376 / 364 / 432), 96 977 / 902 / 942 (558 / 504 / 563), 192 1460 /
// 1244 / 1204 (802 / 721 / 729), 256 1833 / 1528 / 1434 (1006 / 859 / 874), 384
// 2569 / 2045 / 1879 (1397 / 1167 / 1090).  The limits are those of that size.
// 64 experts of 2048 x 2816 (2048 x 1408), 64 / 128 / 256 rows: mean 32 92 / 86 /
// 100 (43 / 51 / 62), 96 121 / 109 / 120 (82 / 70 / 89), 128 140 / 133 / 145 (89 /
// 97 / 109), 256 236 / 182 / 186 (151 / 136 / 162), 384 330 / 251 / 232 (211 / 190 /
// 214): there the gradient's choice costs up to 13 % at means of 128 and 384.
inline int expert_rows(int64_t G, int64_t M, bool gradient) {
  if (M <= (gradient ? 40 : 28) * G) return 64;
  return M <= (gradient ? 256 : 160) * G ? 128 : 256;
}

// Whether the weights pass by the caches: more of them than the Infinity Cache
// holds, and read by one tile, as almost all are with few rows an expert.  256
// experts of 7168 x 4096 (gradient: 2048 x 7168) in us, kept / passing by: 32 rows
// of 31 experts 178 / 162 (gradient 90 / 80), 2048 of 219 1083 / 987 (559 / 535),
// 4096 of 240 1240 / 1156 (637 / 625), 8192 of 251 1386 / 1372 (744 / 758); where
// they fit, called again and again, 8 of 8 53 / 66 (44 / 49).
inline bool read_once(const GatedArgs& a) {
  return a.M <= 20 * a.G && std::min(a.G, a.M) > kStreamBytes / a.K / a.N;
}

constexpr int64_t kGatedMaxPitch = int64_t(1) << 23;  // per-lane copy offsets are 32-bit
constexpr int64_t kGatedMost = int64_t(1) << 31;      // of M, H and K: products of two of them fit 64 bits

// The checks that all entry points share; N: B's columns.
inline fp8blk_status_t gated_check(int64_t M, int64_t H, int64_t K, int64_t N, const uint8_t* A, int64_t lda,
                                   const float* sA, const uint8_t* B, int64_t ldb, int opB, const float* sB, int act,
                                   uint32_t qflags) {
  if (M < 0 || H < 0 || K < 0 || H % 128 != 0 || K % 128 != 0) return FP8BLK_ERR_INVALID_ARG;
  if (act != FP8BLK_ACT_SILU && act != FP8BLK_ACT_GELU) return FP8BLK_ERR_INVALID_ARG;
  if (qflags & ~FP8BLK_SCALE_POW2) return FP8BLK_ERR_INVALID_ARG;
  opB &= ~FP8BLK_GEMM_POW2_SCALES;
  if (opB != FP8BLK_OP_N && opB != FP8BLK_OP_T) return FP8BLK_ERR_INVALID_ARG;
  if (M == 0 || H == 0) return FP8BLK_OK;
  if (K == 0) return FP8BLK_ERR_INVALID_ARG;
  if (M > kGatedMost || H > kGatedMost || K > kGatedMost) return FP8BLK_ERR_UNSUPPORTED;
  if (!matrix_ok(A, M, K, lda, 1)) return FP8BLK_ERR_INVALID_ARG;
  if (opB == FP8BLK_OP_N ? !matrix_ok(B, K, N, ldb, 1) : !matrix_ok(B, N, K, ldb, 1)) return FP8BLK_ERR_INVALID_ARG;
  if (!vec_ok(sA, K / 128 * M) || !vec_ok(sB, K / 128 * (N / 128))) return FP8BLK_ERR_INVALID_ARG;
  if (lda >= kGatedMaxPitch || ldb >= kGatedMaxPitch) return FP8BLK_ERR_UNSUPPORTED;
  // A gated tile's rows of [N][K] B reach over H rows from one resource of less than 2^31 bytes.
  if (opB == FP8BLK_OP_T && N > H && (H + 128) > INT32_MAX / ldb) return FP8BLK_ERR_UNSUPPORTED;
  return FP8BLK_OK;
}

inline bool quantized_ok(int64_t M, int64_t N, const uint8_t* q, int64_t ldq, const float* s) {
  if (q == nullptr) return s == nullptr;
  return matrix_ok(q, M, N, ldq, 1) && vec_ok(s, N / 128 * M);
}
inline bool rows_ok(int64_t M, int64_t N, const void* p, int64_t ld) { return p == nullptr || matrix_ok(p, M, N, ld, 2); }

inline bool forward_ok(int64_t M, int64_t H, const GatedOut& o) {
  return (o.h != nullptr || o.q != nullptr) && rows_ok(M, 2 * H, o.u, o.ldu) && rows_ok(M, H, o.h, o.ldh) &&
         quantized_ok(M, H, o.q, o.ldq, o.s);
}
inline bool backward_ok(int64_t M, int64_t H, const GatedGradOut& o) {
  return o.u != nullptr && (o.du != nullptr || o.q != nullptr) && (o.du != o.u || o.lddu == o.ldu) &&
         rows_ok(M, 2 * H, o.u, o.ldu) && rows_ok(M, 2 * H, o.du, o.lddu) && rows_ok(M, H, o.h, o.ldh) &&
         quantized_ok(M, 2 * H, o.q, o.ldq, o.s);
}

inline GatedArgs gated_args(int64_t M, int64_t H, int64_t K, int64_t N, const uint8_t* A, int64_t lda, const float* sA,
                            const uint8_t* B, int64_t ldb, int opB, const float* sB) {
  GatedArgs a{};
  a.M = M;
  a.H = H;
  a.N = N;
  a.K = K;
  a.A = A;
  a.lda = lda;
  a.sA = sA;
  a.B = B;
  a.ldb = ldb;
  a.sB = sB;
  a.sB_ld = (opB & FP8BLK_OP_T) ? K / 128 : N / 128;
  return a;
}

#define FP8BLK_GATED_BY_B(LAUNCH_)                                               \
  if (opB & FP8BLK_OP_T) {                                                       \
    if (opB & FP8BLK_GEMM_POW2_SCALES) LAUNCH_(true, true); else LAUNCH_(true, false);   \
  } else {                                                                       \
    if (opB & FP8BLK_GEMM_POW2_SCALES) LAUNCH_(false, true); else LAUNCH_(false, false); \
  }

// Grid of the grouped kernels: each expert adds at most one partial row tile of BM;
// a multiple of 8, as grouped_tile's shares of the XCDs need it.  0: too many.
template <class CFG>
inline int64_t grouped_blocks(int64_t G, int64_t M, int64_t max_group_rows, int64_t tiles_n) {
  if (G > kGatedMost) return 0;
  int64_t tiles_m = ceil_div(M, CFG::BM) + G;
  if (max_group_rows > 0) tiles_m = std::min(tiles_m, G * ceil_div(std::min(max_group_rows, M), CFG::BM));
  const int64_t blocks = ceil_div(tiles_m * tiles_n, 8) * 8;
  return grid_ok(blocks, CFG::NT) ? blocks : 0;
}

template <class CFG>
inline bool dense_grid(GatedArgs& a) {
  a.tiles_m = ceil_div(a.M, CFG::BM);
  a.tiles_n = ceil_div(a.N, CFG::BN);
  return grid_ok(a.tiles_m * a.tiles_n, CFG::NT);
}

// The partial products of a dense product of few rows, as S slices of M x N.
template <class D, bool GATED>
inline fp8blk_status_t launch_partials(GatedArgs a, int opB, int64_t& S, float* partials, hipStream_t st) {
  const int64_t G = a.K / 128, per = ceil_div(G, S);
  S = ceil_div(G, per);
  if (!dense_grid<typename D::CFG>(a)) return FP8BLK_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_n), (unsigned)S), block(D::CFG::NT);
  if (opB & FP8BLK_OP_T) hipLaunchKernelGGL((k_gated_partial<D, true, GATED>), grid, block, 0, st, a, partials, (int)per);
  else hipLaunchKernelGGL((k_gated_partial<D, false, GATED>), grid, block, 0, st, a, partials, (int)per);
  return launch_status();
}

// The fused kernels on tiles of CFG (BigCfg) or D, dense or grouped, over `blocks` workgroups.
template <bool GROUPED>
inline fp8blk_status_t launch_big(const GatedArgs& a, int opB, int64_t blocks, const GatedOut& o, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(BigCfg::NT);
#define FP8BLK_GATED_LAUNCH(T_, P2_) hipLaunchKernelGGL((k_gated_gemm<BigCfg, GROUPED, T_, P2_>), grid, block, 0, st, a, o)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
}
template <bool GROUPED>
inline fp8blk_status_t launch_big(const GatedArgs& a, int opB, int64_t blocks, const GatedGradOut& o, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(BigCfg::NT);
#define FP8BLK_GATED_LAUNCH(T_, P2_) \
  hipLaunchKernelGGL((k_gated_gemm_backward<BigCfg, GROUPED, T_, P2_>), grid, block, 0, st, a, o)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
}
template <class D, bool GROUPED, bool ONCE = false>
inline fp8blk_status_t launch_deep(const GatedArgs& a, int opB, int64_t blocks, const GatedOut& o, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(D::CFG::NT);
  if (opB & FP8BLK_OP_T) hipLaunchKernelGGL((k_gated_gemm_deep<D, GROUPED, true, ONCE>), grid, block, 0, st, a, o);
  else hipLaunchKernelGGL((k_gated_gemm_deep<D, GROUPED, false, ONCE>), grid, block, 0, st, a, o);
  return launch_status();
}
template <class D, bool GROUPED, bool ONCE = false>
inline fp8blk_status_t launch_deep(const GatedArgs& a, int opB, int64_t blocks, const GatedGradOut& o, hipStream_t st) {
  const dim3 grid((unsigned)blocks), block(D::CFG::NT);
  if (opB & FP8BLK_OP_T) hipLaunchKernelGGL((k_gated_gemm_backward_deep<D, GROUPED, true, ONCE>), grid, block, 0, st, a, o);
  else hipLaunchKernelGGL((k_gated_gemm_backward_deep<D, GROUPED, false, ONCE>), grid, block, 0, st, a, o);
  return launch_status();
}
constexpr int kJoinSlices = 8;  // where there are more than four parts
inline void launch_join(const float* partials, int64_t S, const GatedArgs& a, const GatedOut& o, hipStream_t st) {
  const int64_t groups = a.M * (a.H / 128);
  if (S > 4)
    hipLaunchKernelGGL(k_gated_join<kJoinSlices>, dim3((unsigned)groups), dim3(32 * kJoinSlices), 0, st, partials, (int)S, a.M,
                       a.H, o);
  else
    hipLaunchKernelGGL(k_gated_join<1>, dim3((unsigned)ceil_div(groups, 2)), dim3(64), 0, st, partials, (int)S, a.M, a.H, o);
}
inline void launch_join(const float* partials, int64_t S, const GatedArgs& a, const GatedGradOut& o, hipStream_t st) {
  const int64_t groups = a.M * (a.H / 128);
  if (S > 4)
    hipLaunchKernelGGL(k_gated_join_backward<kJoinSlices>, dim3((unsigned)groups), dim3(32 * kJoinSlices), 0, st, partials,
                       (int)S, a.M, a.H, o);
  else
    hipLaunchKernelGGL(k_gated_join_backward<1>, dim3((unsigned)ceil_div(groups, 2)), dim3(64), 0, st, partials, (int)S, a.M,
                       a.H, o);
}

inline size_t gated_bytes(int64_t M, int64_t H, int64_t K, int64_t N) {
  if (M <= 0 || H <= 0 || K <= 0 || H % 128 != 0 || K % 128 != 0) return 0;
  if (M > kGatedMost || H > kGatedMost || K > kGatedMost) return 0;
  const int64_t S = gated_form(M, N, K, N == H, true).splits;
  return S > 1 ? (size_t)(S * M * N) * sizeof(float) : 0;
}

// A dense product: in parts and joined where that is faster and the workspace is there.
template <bool GATED, class Out>
inline fp8blk_status_t launch_dense(GatedArgs a, int opB, const Out& o, void* workspace, size_t bytes,
                                    hipStream_t st) {
  const size_t need = gated_bytes(a.M, a.H, a.K, a.N);
  const bool split = need > 0 && workspace != nullptr && aligned(workspace, 16) && bytes >= need;
  GatedForm form = gated_form(a.M, a.N, a.K, !GATED, split);
  if (form.splits > 1) {
    float* partials = static_cast<float*>(workspace);
    const fp8blk_status_t got = form.rows == 32 ? launch_partials<FewDeep, GATED>(a, opB, form.splits, partials, st)
                                                : launch_partials<LowDeep, GATED>(a, opB, form.splits, partials, st);
    if (got != FP8BLK_OK) return got;
    launch_join(partials, form.splits, a, o, st);
    return launch_status();
  }
  const bool fits = form.rows == 256   ? dense_grid<BigCfg>(a)
                    : form.rows == 128 ? dense_grid<MidDeep::CFG>(a)
                                       : dense_grid<LowDeep::CFG>(a);
  if (!fits) return FP8BLK_ERR_UNSUPPORTED;
  const int64_t blocks = a.tiles_m * a.tiles_n;
  if (form.rows == 256) return launch_big<false>(a, opB, blocks, o, st);
  if (form.rows == 128) return launch_deep<MidDeep, false>(a, opB, blocks, o, st);
  return launch_deep<LowDeep, false>(a, opB, blocks, o, st);
}

// A product for every expert.
template <bool GATED, class Out>
inline fp8blk_status_t launch_experts(GatedArgs a, int opB, int64_t max_group_rows, const Out& o, hipStream_t st) {
  a.tiles_n = ceil_div(a.N, 256);
  const int rows = expert_rows(a.G, a.M, !GATED);
  const int64_t blocks = rows == 256   ? grouped_blocks<BigCfg>(a.G, a.M, max_group_rows, a.tiles_n)
                         : rows == 128 ? grouped_blocks<MidDeep::CFG>(a.G, a.M, max_group_rows, a.tiles_n)
                                       : grouped_blocks<LowDeep::CFG>(a.G, a.M, max_group_rows, a.tiles_n);
  if (blocks == 0) return FP8BLK_ERR_UNSUPPORTED;
  if (rows == 256) return launch_big<true>(a, opB, blocks, o, st);
  if (rows == 128) return launch_deep<MidDeep, true>(a, opB, blocks, o, st);
  if (read_once(a)) return launch_deep<LowDeep, true, true>(a, opB, blocks, o, st);
  return launch_deep<LowDeep, true>(a, opB, blocks, o, st);
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_gated_gemm_workspace_bytes(int64_t M, int64_t H, int64_t K) { return gated_bytes(M, H, K, 2 * H); }
extern "C" size_t fp8blk_gated_gemm_backward_workspace_bytes(int64_t M, int64_t H, int64_t K) {
  return gated_bytes(M, H, K, H);
}

extern "C" fp8blk_status_t fp8blk_gated_gemm_fp8_blockscaled(
    int64_t M, int64_t H, int64_t K, const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb,
    int opB, const float* sB, int act, uint16_t* u, int64_t ldu, uint16_t* h, int64_t ldh, uint8_t* q, int64_t ldq,
    float* s, uint32_t qflags, void* workspace, size_t workspace_bytes, void* stream) {
  const fp8blk_status_t ok = gated_check(M, H, K, 2 * H, A, lda, sA, B, ldb, opB, sB, act, qflags);
  if (ok != FP8BLK_OK || M == 0 || H == 0) return ok;
  const GatedOut o{u, ldu, h, ldh, q, ldq, s, M, act == FP8BLK_ACT_GELU, (qflags & FP8BLK_SCALE_POW2) != 0};
  if (!forward_ok(M, H, o)) return FP8BLK_ERR_INVALID_ARG;
  const GatedArgs a = gated_args(M, H, K, 2 * H, A, lda, sA, B, ldb, opB, sB);
  return launch_dense<true>(a, opB, o, workspace, workspace_bytes, as_stream(stream));
}

extern "C" fp8blk_status_t fp8blk_grouped_gated_gemm_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t H, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, int act, uint16_t* u, int64_t ldu, uint16_t* h, int64_t ldh, uint8_t* q,
    int64_t ldq, float* s, uint32_t qflags, void* stream) {
  if (G < 0 || max_group_rows < 0) return FP8BLK_ERR_INVALID_ARG;
  const fp8blk_status_t ok = gated_check(G == 0 ? 0 : M_total, H, K, 2 * H, A, lda, sA, B, ldb, opB, sB, act, qflags);
  if (ok != FP8BLK_OK || G == 0 || M_total == 0 || H == 0) return ok;
  if (group_offsets == nullptr || !aligned(group_offsets, 4)) return FP8BLK_ERR_INVALID_ARG;
  const int64_t brows = (opB & FP8BLK_OP_T) ? 2 * H : K;
  if (strideB / ldb < brows || strideB % 16 != 0 || stride_sB < K / 128 * (2 * H / 128)) return FP8BLK_ERR_INVALID_ARG;
  const GatedOut o{u, ldu, h, ldh, q, ldq, s, M_total, act == FP8BLK_ACT_GELU, (qflags & FP8BLK_SCALE_POW2) != 0};
  if (!forward_ok(M_total, H, o)) return FP8BLK_ERR_INVALID_ARG;
  GatedArgs a = gated_args(M_total, H, K, 2 * H, A, lda, sA, B, ldb, opB, sB);
  a.G = G;
  a.offsets = group_offsets;
  a.strideB = strideB;
  a.stride_sB = stride_sB;
  return launch_experts<true>(a, opB, max_group_rows, o, as_stream(stream));
}

extern "C" fp8blk_status_t fp8blk_gated_gemm_backward_fp8_blockscaled(
    int64_t M, int64_t H, int64_t K, const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb,
    int opB, const float* sB, int act, const uint16_t* u, int64_t ldu, uint16_t* du, int64_t lddu, uint16_t* h,
    int64_t ldh, uint8_t* q, int64_t ldq, float* s, uint32_t qflags, void* workspace, size_t workspace_bytes,
    void* stream) {
  const fp8blk_status_t ok = gated_check(M, H, K, H, A, lda, sA, B, ldb, opB, sB, act, qflags);
  if (ok != FP8BLK_OK || M == 0 || H == 0) return ok;
  const GatedGradOut o{u, ldu, du, lddu, h, ldh, q, ldq, s, M, act == FP8BLK_ACT_GELU, (qflags & FP8BLK_SCALE_POW2) != 0};
  if (!backward_ok(M, H, o)) return FP8BLK_ERR_INVALID_ARG;
  const GatedArgs a = gated_args(M, H, K, H, A, lda, sA, B, ldb, opB, sB);
  return launch_dense<false>(a, opB, o, workspace, workspace_bytes, as_stream(stream));
}

extern "C" fp8blk_status_t fp8blk_grouped_gated_gemm_backward_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t H, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, int act, const uint16_t* u, int64_t ldu, uint16_t* du, int64_t lddu,
    uint16_t* h, int64_t ldh, uint8_t* q, int64_t ldq, float* s, uint32_t qflags, void* stream) {
  if (G < 0 || max_group_rows < 0) return FP8BLK_ERR_INVALID_ARG;
  const fp8blk_status_t ok = gated_check(G == 0 ? 0 : M_total, H, K, H, A, lda, sA, B, ldb, opB, sB, act, qflags);
  if (ok != FP8BLK_OK || G == 0 || M_total == 0 || H == 0) return ok;
  if (group_offsets == nullptr || !aligned(group_offsets, 4)) return FP8BLK_ERR_INVALID_ARG;
  const int64_t brows = (opB & FP8BLK_OP_T) ? H : K;
  if (strideB / ldb < brows || strideB % 16 != 0 || stride_sB < K / 128 * (H / 128)) return FP8BLK_ERR_INVALID_ARG;
  const GatedGradOut o{u,   ldu, du, lddu,    h, ldh, q, ldq, s, M_total, act == FP8BLK_ACT_GELU,
                       (qflags & FP8BLK_SCALE_POW2) != 0};
  if (!backward_ok(M_total, H, o)) return FP8BLK_ERR_INVALID_ARG;
  GatedArgs a = gated_args(M_total, H, K, H, A, lda, sA, B, ldb, opB, sB);
  a.G = G;
  a.offsets = group_offsets;
  a.strideB = strideB;
  a.stride_sB = stride_sB;
  return launch_experts<false>(a, opB, max_group_rows, o, as_stream(stream));
}
