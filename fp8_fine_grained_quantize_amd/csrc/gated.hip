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
#include <algorithm>

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
// each: with the products before them within (4 + 2 |z|) 2^-24 of itself (BF16
// has 2^-8), and 0 where e^-z passes FP32's range, z < -88.
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

// --- few rows: the product split over K, joined with the activation ----------

// FP32 partial products [split][M][N] of K groups [split * per, ...).
template <class CFG, bool OPB_T, bool P2>
__global__ __launch_bounds__(CFG::NT) void k_gated_partial(GatedArgs a, float* __restrict__ partials, int per) {
  FP8BLK_DECLARE_STAGES(CFG);
  TileArgs t;
  gated_tile<CFG, false, false>(a, t);
  t.g0 = blockIdx.y * per;
  t.g1 = min(t.g0 + per, (int)(a.K / 128));
  t.C = partials + ((int64_t)blockIdx.y * a.M + t.m0) * a.N;
  t.ldc = a.N;
  gemm_tile<CFG, OPB_T, false, P2, OUT_F32>(t, s_ops0, s_ops1, s_sc0, s_sc1);
}

// Eight columns of a row: their sum over the S partial products, in order.
__device__ __forceinline__ void join8(const float* __restrict__ p, int S, int64_t step, float (&x)[8]) {
  float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  for (int s = 1; s < S; ++s) {
    const float4 c = reinterpret_cast<const float4*>(p + s * step)[0], d = reinterpret_cast<const float4*>(p + s * step)[1];
    a.x += c.x; a.y += c.y; a.z += c.z; a.w += c.w;
    b.x += d.x; b.y += d.y; b.z += d.z; b.w += d.w;
  }
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16_pack(x[0], x[1]), bf16_pack(x[2], x[3]), bf16_pack(x[4], x[5]), bf16_pack(x[6], x[7]));
}
// The codes of eight values of a tile that 16 lanes hold, and its scale.
__device__ __forceinline__ void put_codes(const uint4& w, bool pow2, uint8_t* q, float* s) {
  const uint32_t m = row16_max(abs_max_bits(abs_max_bits(abs_max_bits(abs_max_bits(0, w.x), w.y), w.z), w.w));
  const uint32_t p[4] = {w.x, w.y, w.z, w.w};
  uint32_t c[2];
  float scale;
  if (pow2) encode_bf16<true>(p, m, c, scale);
  else encode_bf16<false>(p, m, c, scale);
  *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[1]);
  if ((threadIdx.x & 15) == 0) *s = scale;
}

// A lane has eight columns of h, 16 lanes a scale group; M * H / 8 lanes, a
// multiple of 16, in workgroups of 256.
__global__ __launch_bounds__(256) void k_gated_join(const float* __restrict__ partials, int S, int64_t M, int64_t H,
                                                     GatedOut o) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = at / (H / 8), c = at % (H / 8) * 8;
  if (m >= M) return;
  float g[8], v[8], x[8];
  const float* p = partials + m * 2 * H + c;
  join8(p, S, M * 2 * H, g);
  join8(p + H, S, M * 2 * H, v);
  if (o.u != nullptr) {
    *reinterpret_cast<uint4*>(o.u + m * o.ldu + c) = pack8(g);
    *reinterpret_cast<uint4*>(o.u + m * o.ldu + H + c) = pack8(v);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = o.gelu ? gated<true>(g[j], v[j]) : gated<false>(g[j], v[j]);
  const uint4 w = pack8(x);
  if (o.h != nullptr) *reinterpret_cast<uint4*>(o.h + m * o.ldh + c) = w;
  if (o.q != nullptr) put_codes(w, o.pow2, o.q + m * o.ldq + c, o.s + (c >> 7) * o.s_ld + m);
}

__global__ __launch_bounds__(256) void k_gated_join_backward(const float* __restrict__ partials, int S, int64_t M,
                                                              int64_t H, GatedGradOut o) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = at / (H / 8), c = at % (H / 8) * 8;
  if (m >= M) return;
  const uint4 ug = *reinterpret_cast<const uint4*>(o.u + m * o.ldu + c);
  const uint4 uv = *reinterpret_cast<const uint4*>(o.u + m * o.ldu + H + c);
  float dh[8], dg[8], dv[8], h[8];
  join8(partials + m * H + c, S, M * H, dh);
  const uint32_t g[4] = {ug.x, ug.y, ug.z, ug.w}, v[4] = {uv.x, uv.y, uv.z, uv.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = j & 1 ? bf16_hi(g[j >> 1]) : bf16_lo(g[j >> 1]), vj = j & 1 ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
    if (o.gelu) gated_grad<true>(dh[j], gj, vj, dg[j], dv[j], h[j]);
    else gated_grad<false>(dh[j], gj, vj, dg[j], dv[j], h[j]);
  }
  const uint4 wg = pack8(dg), wv = pack8(dv);
  if (o.du != nullptr) {
    *reinterpret_cast<uint4*>(o.du + m * o.lddu + c) = wg;
    *reinterpret_cast<uint4*>(o.du + m * o.lddu + H + c) = wv;
  }
  if (o.h != nullptr) *reinterpret_cast<uint4*>(o.h + m * o.ldh + c) = pack8(h);
  if (o.q != nullptr) {
    put_codes(wg, o.pow2, o.q + m * o.ldq + c, o.s + (c >> 7) * o.s_ld + m);
    put_codes(wv, o.pow2, o.q + m * o.ldq + H + c, o.s + ((H + c) >> 7) * o.s_ld + m);
  }
}

// Splits of K for a dense product of M rows and N columns of B, 0 where the
// fused tiles of 256 x 256 are at least half as many as the compute units and
// it is not split at all.
inline int64_t gated_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t big_m = (M - 1) / BigCfg::BM + 1, big_n = (N - 1) / BigCfg::BN + 1;
  if (big_m >= 128 || big_n >= 128 || big_m * big_n >= 128) return 0;
  const int64_t G = K / 128, tiles = ceil_div(M, SmallCfg::BM) * ceil_div(N, SmallCfg::BN);
  int64_t S = ceil_div(2 * (int64_t)device_cus(), tiles);  // two 128 x 128 workgroups fit per CU
  if (S > G / 4) S = G / 4;
  if (S > 16) S = 16;
  return S < 1 ? 1 : S;
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

// Grid of the grouped kernels: each expert adds at most one partial row tile;
// a multiple of 8, as grouped_tile's shares of the XCDs need it.  0: too many.
inline int64_t grouped_blocks(int64_t G, int64_t M, int64_t max_group_rows, int64_t tiles_n) {
  if (G > kGatedMost) return 0;
  int64_t tiles_m = ceil_div(M, BigCfg::BM) + G;
  if (max_group_rows > 0) tiles_m = std::min(tiles_m, G * ceil_div(std::min(max_group_rows, M), BigCfg::BM));
  const int64_t blocks = ceil_div(tiles_m * tiles_n, 8) * 8;
  return grid_ok(blocks, BigCfg::NT) ? blocks : 0;
}

// The partial products of a dense product of few rows, as S slices of M x N.
inline fp8blk_status_t launch_partials(GatedArgs a, int opB, int64_t& S, float* partials, hipStream_t st) {
  using CFG = SmallCfg;
  a.tiles_m = ceil_div(a.M, CFG::BM);
  a.tiles_n = ceil_div(a.N, CFG::BN);
  const int64_t G = a.K / 128, per = ceil_div(G, S);
  S = ceil_div(G, per);
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_n), (unsigned)S), block(CFG::NT);
#define FP8BLK_GATED_LAUNCH(T_, P2_) \
  hipLaunchKernelGGL((k_gated_partial<CFG, T_, P2_>), grid, block, 0, st, a, partials, (int)per)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_gated_gemm_workspace_bytes(int64_t M, int64_t H, int64_t K) {
  if (M <= 0 || H <= 0 || K <= 0 || H % 128 != 0 || K % 128 != 0) return 0;
  return (size_t)(gated_splits(M, 2 * H, K) * M * 2 * H) * sizeof(float);
}
extern "C" size_t fp8blk_gated_gemm_backward_workspace_bytes(int64_t M, int64_t H, int64_t K) {
  if (M <= 0 || H <= 0 || K <= 0 || H % 128 != 0 || K % 128 != 0) return 0;
  return (size_t)(gated_splits(M, H, K) * M * H) * sizeof(float);
}

extern "C" fp8blk_status_t fp8blk_gated_gemm_fp8_blockscaled(
    int64_t M, int64_t H, int64_t K, const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb,
    int opB, const float* sB, int act, uint16_t* u, int64_t ldu, uint16_t* h, int64_t ldh, uint8_t* q, int64_t ldq,
    float* s, uint32_t qflags, void* workspace, size_t workspace_bytes, void* stream) {
  const fp8blk_status_t ok = gated_check(M, H, K, 2 * H, A, lda, sA, B, ldb, opB, sB, act, qflags);
  if (ok != FP8BLK_OK || M == 0 || H == 0) return ok;
  const GatedOut o{u, ldu, h, ldh, q, ldq, s, M, act == FP8BLK_ACT_GELU, (qflags & FP8BLK_SCALE_POW2) != 0};
  if (!forward_ok(M, H, o)) return FP8BLK_ERR_INVALID_ARG;
  GatedArgs a = gated_args(M, H, K, 2 * H, A, lda, sA, B, ldb, opB, sB);
  hipStream_t st = as_stream(stream);
  int64_t S = gated_splits(M, 2 * H, K);
  if (S > 0 && workspace != nullptr && aligned(workspace, 16) &&
      workspace_bytes >= fp8blk_gated_gemm_workspace_bytes(M, H, K)) {
    float* partials = static_cast<float*>(workspace);
    const fp8blk_status_t got = launch_partials(a, opB, S, partials, st);
    if (got != FP8BLK_OK) return got;
    hipLaunchKernelGGL(k_gated_join, dim3((unsigned)ceil_div(M * (H / 8), 256)), dim3(256), 0, st, partials, (int)S, M,
                       H, o);
    return launch_status();
  }
  using CFG = BigCfg;
  a.tiles_m = ceil_div(M, CFG::BM);
  a.tiles_n = H / (CFG::BN / 2);
  if (!grid_ok(a.tiles_m * a.tiles_n, CFG::NT)) return FP8BLK_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(CFG::NT);
#define FP8BLK_GATED_LAUNCH(T_, P2_) hipLaunchKernelGGL((k_gated_gemm<CFG, false, T_, P2_>), grid, block, 0, st, a, o)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_grouped_gated_gemm_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t H, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, int act, uint16_t* u, int64_t ldu, uint16_t* h, int64_t ldh, uint8_t* q,
    int64_t ldq, float* s, uint32_t qflags, void* stream) {
  using CFG = BigCfg;
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
  a.tiles_n = H / (CFG::BN / 2);
  const int64_t blocks = grouped_blocks(G, M_total, max_group_rows, a.tiles_n);
  if (blocks == 0) return FP8BLK_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(CFG::NT);
  hipStream_t st = as_stream(stream);
#define FP8BLK_GATED_LAUNCH(T_, P2_) hipLaunchKernelGGL((k_gated_gemm<CFG, true, T_, P2_>), grid, block, 0, st, a, o)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
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
  GatedArgs a = gated_args(M, H, K, H, A, lda, sA, B, ldb, opB, sB);
  hipStream_t st = as_stream(stream);
  int64_t S = gated_splits(M, H, K);
  if (S > 0 && workspace != nullptr && aligned(workspace, 16) &&
      workspace_bytes >= fp8blk_gated_gemm_backward_workspace_bytes(M, H, K)) {
    float* partials = static_cast<float*>(workspace);
    const fp8blk_status_t got = launch_partials(a, opB, S, partials, st);
    if (got != FP8BLK_OK) return got;
    hipLaunchKernelGGL(k_gated_join_backward, dim3((unsigned)ceil_div(M * (H / 8), 256)), dim3(256), 0, st, partials,
                       (int)S, M, H, o);
    return launch_status();
  }
  using CFG = BigCfg;
  a.tiles_m = ceil_div(M, CFG::BM);
  a.tiles_n = ceil_div(H, CFG::BN);
  if (!grid_ok(a.tiles_m * a.tiles_n, CFG::NT)) return FP8BLK_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(CFG::NT);
#define FP8BLK_GATED_LAUNCH(T_, P2_) \
  hipLaunchKernelGGL((k_gated_gemm_backward<CFG, false, T_, P2_>), grid, block, 0, st, a, o)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_grouped_gated_gemm_backward_fp8_blockscaled(
    int64_t G, const int32_t* group_offsets, int64_t M_total, int64_t max_group_rows, int64_t H, int64_t K,
    const uint8_t* A, int64_t lda, const float* sA, const uint8_t* B, int64_t ldb, int64_t strideB, int opB,
    const float* sB, int64_t stride_sB, int act, const uint16_t* u, int64_t ldu, uint16_t* du, int64_t lddu,
    uint16_t* h, int64_t ldh, uint8_t* q, int64_t ldq, float* s, uint32_t qflags, void* stream) {
  using CFG = BigCfg;
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
  a.tiles_n = ceil_div(H, CFG::BN);
  const int64_t blocks = grouped_blocks(G, M_total, max_group_rows, a.tiles_n);
  if (blocks == 0) return FP8BLK_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(CFG::NT);
  hipStream_t st = as_stream(stream);
#define FP8BLK_GATED_LAUNCH(T_, P2_) \
  hipLaunchKernelGGL((k_gated_gemm_backward<CFG, true, T_, P2_>), grid, block, 0, st, a, o)
  FP8BLK_GATED_BY_B(FP8BLK_GATED_LAUNCH)
#undef FP8BLK_GATED_LAUNCH
  return launch_status();
}
