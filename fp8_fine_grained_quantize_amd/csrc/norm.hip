// The norm after a block with its gate and residual scale, the residual sum
// and the norm before the next block, and their gradients (gfx950).
//
//   u = f r_post w_post,  x' = x + alpha gate u,  n = x' r_pre w_pre,
//   r = (mean_c z^2 + eps)^(-1/2) of the respective input z,
// in one pass: f and x are read once, x' and n written once, and where the
// next GEMM takes E4M3, n is quantized to 1x128 tiles on the way out
// [p1¶3, p2¶4: the inputs of the projections are quantized online].
// Citations [pN¶k]: N-th page of the source collection, k-th paragraph
// (p1 = xn--9g3bo1gtkw0l8ubf92bgle.kr wr_id 85187, p2 = inprokorea.com
// wr_id 735329).
//
// For n_j = z_j r w_j, dr/dz_i = -r^3 z_i / C, so with v = dn w and h = z r
//   dz = r (v - h mean_c(v h)),   dw = sum_m dn h.
#include "../../include/libfp8blk_layer.h"
#include "host_common.h"
#include "layer_device.h"
#include "layer_host.h"

namespace fp8blk {

constexpr int64_t kNormMaxC = 16384;

struct NormFwd {
  const void* x;
  const uint16_t* f;
  const void* w_post;
  const void* gate;
  const void* w_pre;
  void* x_out;
  uint16_t* n;
  uint8_t* q;
  float* s;
  float* rstd_post;
  float* rstd_pre;
  int64_t M, C, ldx, ldf, ldg, ldxo, ldn, ldq;
  float alpha, eps;
  uint32_t flags;
};

// Eight parameters of either type from an element-aligned vector.
template <bool EXACT>
__device__ __forceinline__ void load_param8(const void* p, bool f32, int64_t col, int64_t C, float (&v)[8]) {
  if (f32)
    unpack_end<float, 8, EXACT>(load_end<8, EXACT, false>(reinterpret_cast<const float*>(p), col, C), col, C, v);
  else
    unpack_end<uint16_t, 8, EXACT>(load_end<8, EXACT, false>(reinterpret_cast<const uint16_t*>(p), col, C), col, C, v);
}

// The 1x128 tile of n that a row of 16 lanes holds, eight values each, scaled
// and rounded as the BF16 quantizers do it (fp8_device.h): n / s by Markstein's
// correction with the rounded reciprocal, for FP32 n within one unit in the
// last place of the quotient, or by the exact reciprocal of a power of two.
template <bool POW2>
__device__ __forceinline__ uint2 quantize_tile(const float (&n)[8], float& s) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(n[i]) & 0x7FFFFFFFu);
  const TileScale ts = make_scale<POW2, true>(row16_max(a));
  s = ts.s;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = quotient_fast<POW2, true>(n[i], ts);
  if (__builtin_expect(ts.slow, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = quotient_slow(n[i], ts.s);
  }
  uint2 c;
  c.x = pack4_e4m3(y[0], y[1], y[2], y[3]);
  c.y = pack4_e4m3(y[4], y[5], y[6], y[7]);
  return c;
}

template <bool EXACT, bool NT>
__device__ __forceinline__ void store_codes8(uint8_t* p, int64_t avail, uint2 c) {
  if (EXACT ? avail > 0 : avail >= 8) {
    store_words<NT, 2>((Global<void>*)p, Words<2>::type{c.x, c.y});
    return;
  }
  if (EXACT) return;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < avail) p[j] = (uint8_t)((j < 4 ? c.x : c.y) >> ((j & 3) * 8));
}

// The statistic of a row: (sum / C + eps)^(-1/2).
__device__ __forceinline__ float rstd_of(float sum, float inv_c, float eps) { return 1.0f / sqrtf(sum * inv_c + eps); }

// What a lane reads of one row, before it is unpacked.
template <typename TX, int NCH, bool GATE_ROW, bool EXACT>
struct NormRow {
  RawV<TX, 8> x[NCH];
  RawV<uint16_t, 8> f[NCH], gate[GATE_ROW ? NCH : 1];
};

template <bool NT, typename TX, int NCH, bool GATE_ROW, bool EXACT>
__device__ __forceinline__ void load_row(NormRow<TX, NCH, GATE_ROW, EXACT>& r, const NormFwd& a, int64_t row) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * blockDim.x) * 8;
    r.x[c] = load_end<8, EXACT, NT, (NCH > 1)>(reinterpret_cast<const TX*>(a.x) + row * a.ldx, col, a.C);
    if (a.f != nullptr) r.f[c] = load_end<8, EXACT, NT, (NCH > 1)>(a.f + row * a.ldf, col, a.C);
    if (GATE_ROW) r.gate[c] = load_end<8, EXACT, NT, (NCH > 1)>(reinterpret_cast<const uint16_t*>(a.gate) + row * a.ldg, col, a.C);
  }
}

// A workgroup takes the rows blockIdx.x, blockIdx.x + gridDim.x, ...; lane t
// holds the chunks of eight channels t, t + NT, ... (NCH of them), so that a
// 1x128 tile is one row of 16 lanes, and the parameters of its channels.  The
// next row is loaded before the present one is worked on: the reductions and
// stores of one row cover the other's way from HBM, which bounds it.  8192 x 7168
// (BF16, n and E4M3 out) takes 96 us, 530 MB at 5.5 TB/s; without the next row
// in flight and with the parameters read again for every row it took 162.  A
// decode step of 16 rows takes 5.5 us: launch, one load, two reductions.
template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT>
__global__ __launch_bounds__(1024) void k_residual_norm(const NormFwd a) {
  __shared__ float red[2][2][16];
  const int nt = blockDim.x, nw = nt >> 6;
  const float inv_c = 1.0f / (float)a.C;
  const bool pf32 = (a.flags & FP8BLK_NORM_PARAM_F32) != 0;
  float pc[NCH][8], wn[NCH][8];  // alpha * w_post * (gate per channel); w_pre
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) pc[c][i] = a.alpha;
    float w[8];
    if (a.w_post != nullptr) {
      load_param8<EXACT>(a.w_post, pf32, col, a.C, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) pc[c][i] *= w[i];
    }
    if (a.gate != nullptr && !GATE_ROW) {
      load_param8<EXACT>(a.gate, pf32, col, a.C, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) pc[c][i] *= w[i];
    }
    if (a.w_pre != nullptr) load_param8<EXACT>(a.w_pre, pf32, col, a.C, wn[c]);
  }
  NormRow<TX, NCH, GATE_ROW, EXACT> next;
  load_row<NT>(next, a, blockIdx.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    const NormRow<TX, NCH, GATE_ROW, EXACT> cur = next;
    if (row + gridDim.x < a.M) load_row<NT>(next, a, row + gridDim.x);
    float z[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      unpack_end<TX, 8, EXACT, (NCH > 1)>(cur.x[c], ((int64_t)threadIdx.x + (int64_t)c * nt) * 8, a.C, z[c]);
    if (a.f != nullptr) {
      float r = 1.0f;
      if (a.w_post != nullptr) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          float f[8];
          unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.f[c], ((int64_t)threadIdx.x + (int64_t)c * nt) * 8, a.C, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(f[i], f[i], sum[0]);
        }
        block_sum<1>(sum, red[turn][0], nw);
        r = rstd_of(sum[0], inv_c, a.eps);
        if (a.rstd_post != nullptr && threadIdx.x == 0) a.rstd_post[row] = r;
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
        float f[8];
        unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.f[c], col, a.C, f);
        if (GATE_ROW) {
          float g[8];
          unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.gate[c], col, a.C, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) z[c][i] = __builtin_fmaf(f[i] * r, pc[c][i], z[c][i]);
        store_end<8, EXACT, NT>(reinterpret_cast<TX*>(a.x_out) + row * a.ldxo, col, a.C, z[c]);
      }
    }
    if (a.w_pre == nullptr) continue;
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(z[c][i], z[c][i], sum[0]);
    block_sum<1>(sum, red[turn][1], nw);
    const float r = rstd_of(sum[0], inv_c, a.eps);
    if (a.rstd_pre != nullptr && threadIdx.x == 0) a.rstd_pre[row] = r;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t chunk = (int64_t)threadIdx.x + (int64_t)c * nt, col = chunk * 8, avail = a.C - col;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] = z[c][i] * r * wn[c][i];
      if (a.n != nullptr) store_end<8, EXACT, NT>(a.n + row * a.ldn, col, a.C, z[c]);
      if (a.q != nullptr) {
        float s;
        const uint2 codes = a.flags & FP8BLK_SCALE_POW2 ? quantize_tile<true>(z[c], s) : quantize_tile<false>(z[c], s);
        if (avail > 0) {
          store_codes8<EXACT, NT>(a.q + row * a.ldq + col, avail, codes);
          if ((threadIdx.x & 15) == 0) a.s[(chunk >> 4) * a.M + row] = s;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient.  With h = x' r_pre, v = dn w_pre, m = mean_c(v h) the gradient of
// x' is g = dx_out + r_pre (v - h m), and with h' = f r_post and v' = p g,
// p = alpha gate w_post, df = r_post (v' - h' m'), where
//   m' = mean_c(v' h') = (sum_c p h' (dx_out + r_pre v) - r_pre m sum_c p h' h) / C,
// so that all three sums of a row come from one pass and one barrier.  The
// sums over rows need only two accumulators per channel, of dn h and of
// g h' (times the gate where it is one per token): the channel's own factors
// follow at the end,
//   dw_post = alpha gate sum_m g h',   dgate = alpha w_post sum_m g h'.
// A workgroup takes the rows blockIdx.x, blockIdx.x + gridDim.x, ... with the
// next row's loads in flight, keeps the accumulators in registers and writes
// them as one row of partials, which k_norm_sums adds up in order.  HBM bounds
// it: 8192 x 7168 takes 120 us, 705 MB at 5.9 TB/s, and the sums 5; with two
// reductions a row, three accumulators per channel and no row ahead it was 222
// + 16.
// ---------------------------------------------------------------------------
struct NormBwd {
  const void* x;
  const void* dxo;
  const uint16_t* dn;
  const float* rstd_pre;
  const void* w_pre;
  const uint16_t* f;
  const float* rstd_post;
  const void* w_post;
  const void* gate;
  void* dx;
  uint16_t* df;
  uint16_t* dgate_row;
  float* part_pre;   // [gridDim.x][C] each, or NULL
  float* part_post;
  int64_t M, C, ldx, lddxo, lddn, ldf, ldg, lddx, lddf, lddg;
  float alpha;
  uint32_t flags;
};

// What a lane reads of one chunk of one row, before it is unpacked.
template <typename TX, bool GATE_ROW>
struct NormBwdChunk {
  RawV<TX, 8> x, dxo;
  RawV<uint16_t, 8> dn, f, gate;
};

template <bool EXACT, bool NT, bool LONG, typename TX, bool GATE_ROW>
__device__ __forceinline__ void load_chunk(NormBwdChunk<TX, GATE_ROW>& r, const NormBwd& a, int64_t row, int64_t col) {
  r = {};
  if (a.w_pre != nullptr) {
    r.x = load_end<8, EXACT, NT, LONG>(reinterpret_cast<const TX*>(a.x) + row * a.ldx, col, a.C);
    r.dn = load_end<8, EXACT, NT, LONG>(a.dn + row * a.lddn, col, a.C);
  }
  if (a.dxo != nullptr) r.dxo = load_end<8, EXACT, NT, LONG>(reinterpret_cast<const TX*>(a.dxo) + row * a.lddxo, col, a.C);
  if (a.f != nullptr) r.f = load_end<8, EXACT, NT, LONG>(a.f + row * a.ldf, col, a.C);
  if (GATE_ROW) r.gate = load_end<8, EXACT, NT, LONG>(reinterpret_cast<const uint16_t*>(a.gate) + row * a.ldg, col, a.C);
}

// The parameters of a chunk: alpha * w_post * (gate per channel), and w_pre.
template <bool GATE_ROW, bool EXACT>
__device__ __forceinline__ void load_factors(const NormBwd& a, int64_t col, float (&pc)[8], float (&wn)[8]) {
  const bool pf32 = (a.flags & FP8BLK_NORM_PARAM_F32) != 0;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    pc[i] = a.alpha;
    wn[i] = 0.0f;
  }
  if (a.w_post != nullptr) {
    load_param8<EXACT>(a.w_post, pf32, col, a.C, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) pc[i] *= w[i];
  }
  if (a.gate != nullptr && !GATE_ROW) {
    load_param8<EXACT>(a.gate, pf32, col, a.C, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) pc[i] *= w[i];
  }
  if (a.w_pre != nullptr) load_param8<EXACT>(a.w_pre, pf32, col, a.C, wn);
}

// HOLD: the factors and the next row are held in registers, up to 256 of 512
// lanes.  Where they would not fit beside the accumulators (C above 8192; FP32
// x with a gate per token above 4096) 1024 lanes read factors and rows chunk
// by chunk, and once more (from L2) after the reduction, with the accumulators
// in LDS.
template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT, bool HOLD>
__global__ __launch_bounds__(HOLD ? 512 : 1024) void k_residual_norm_backward(const NormBwd a) {
  constexpr int NH = HOLD ? NCH : 1, UNROLL = NH;  // without HOLD one chunk after the other
  __shared__ float red[2][3 * 16];
  const int nt = blockDim.x, nw = nt >> 6;
  const float inv_c = 1.0f / (float)a.C;
  __shared__ float acc[HOLD ? 1 : 2 * NCH * 8 * 1024];
  float s_pre[NH][8], s_post[NH][8], pc_[NH][8], wn_[NH][8];
  // this lane's accumulator `vec` (0: dn h, 1: g h') of channel i of chunk c in LDS
  auto slot = [&](int vec, int c, int i) -> float& { return acc[((vec * NCH + c) * 8 + i) * 1024 + threadIdx.x]; };
  NormBwdChunk<TX, GATE_ROW> next[NH], cur_[NH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (HOLD) s_pre[c][i] = s_post[c][i] = 0.0f;
      else slot(0, c, i) = slot(1, c, i) = 0.0f;
    }
    if (HOLD) {
      load_factors<GATE_ROW, EXACT>(a, col, pc_[c], wn_[c]);
      load_chunk<EXACT, NT, (NCH > 1)>(next[c], a, blockIdx.x, col);
    }
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1) {
    const float r_pre = a.w_pre != nullptr ? a.rstd_pre[row] : 0.0f;
    const float r_post = a.w_post != nullptr ? a.rstd_post[row] : 1.0f;
    if (HOLD) {
#pragma unroll
      for (int c = 0; c < NH; ++c) {
        cur_[c] = next[c];
        if (row + gridDim.x < a.M)
          load_chunk<EXACT, NT, (NCH > 1)>(next[c], a, row + gridDim.x, ((int64_t)threadIdx.x + (int64_t)c * nt) * 8);
      }
    }
    float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll UNROLL
    for (int c = 0; c < NCH; ++c) {
      float(&pc)[8] = pc_[HOLD ? c : 0];
      float(&wn)[8] = wn_[HOLD ? c : 0];
      NormBwdChunk<TX, GATE_ROW>& cur = cur_[HOLD ? c : 0];
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
      if (!HOLD) {
        load_factors<GATE_ROW, EXACT>(a, col, pc, wn);
        load_chunk<EXACT, NT && HOLD, (NCH > 1)>(cur, a, row, col);
      }
      float h[8], v[8], g[8], hf[8], gt[8];
      unpack_end<TX, 8, EXACT, (NCH > 1)>(cur.x, col, a.C, h);
      unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.dn, col, a.C, v);
      unpack_end<TX, 8, EXACT, (NCH > 1)>(cur.dxo, col, a.C, g);
      unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.f, col, a.C, hf);
      if (GATE_ROW) unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.gate, col, a.C, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] *= r_pre;
        float& sp = HOLD ? s_pre[HOLD ? c : 0][i] : slot(0, c, i);
        sp = __builtin_fmaf(v[i], h[i], sp);
        v[i] *= wn[i];
        sum[0] = __builtin_fmaf(v[i], h[i], sum[0]);
        float p = pc[i] * (hf[i] * r_post);
        if (GATE_ROW) p *= gt[i];
        sum[1] = __builtin_fmaf(p, __builtin_fmaf(r_pre, v[i], g[i]), sum[1]);
        sum[2] = __builtin_fmaf(p, h[i], sum[2]);
      }
    }
    block_sum<3>(sum, red[turn], nw);
    const float m = sum[0] * inv_c;
    const float m_post = a.w_post != nullptr ? (sum[1] - r_pre * m * sum[2]) * inv_c : 0.0f;
#pragma unroll UNROLL
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
      float(&pc)[8] = pc_[HOLD ? c : 0];
      float(&wn)[8] = wn_[HOLD ? c : 0];
      NormBwdChunk<TX, GATE_ROW>& cur = cur_[HOLD ? c : 0];
      if (!HOLD) {
        load_factors<GATE_ROW, EXACT>(a, col, pc, wn);
        load_chunk<EXACT, NT && HOLD, (NCH > 1)>(cur, a, row, col);
      }
      float h[8], v[8], g[8];
      unpack_end<TX, 8, EXACT, (NCH > 1)>(cur.x, col, a.C, h);
      unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.dn, col, a.C, v);
      unpack_end<TX, 8, EXACT, (NCH > 1)>(cur.dxo, col, a.C, g);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        g[i] = __builtin_fmaf(r_pre, __builtin_fmaf(-(h[i] * r_pre), m, v[i] * wn[i]), g[i]);
      if (a.dx != nullptr) store_end<8, EXACT, NT>(reinterpret_cast<TX*>(a.dx) + row * a.lddx, col, a.C, g);
      if (a.f == nullptr) continue;
      unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.f, col, a.C, h);
      float gt[8];
      if (GATE_ROW) unpack_end<uint16_t, 8, EXACT, (NCH > 1)>(cur.gate, col, a.C, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] *= r_post;
        v[i] = g[i] * h[i];  // times its factors: the terms of dw_post and dgate
        float d = pc[i] * g[i];
        if (GATE_ROW) d *= gt[i];
        float& sp = HOLD ? s_post[HOLD ? c : 0][i] : slot(1, c, i);
        sp += GATE_ROW ? v[i] * gt[i] : v[i];
        g[i] = r_post * __builtin_fmaf(-h[i], m_post, d);
      }
      if (GATE_ROW) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= pc[i];
        store_end<8, EXACT, NT>(a.dgate_row + row * a.lddg, col, a.C, v);
      }
      store_end<8, EXACT, NT>(a.df + row * a.lddf, col, a.C, g);
    }
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
    if (!HOLD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_pre[0][i] = slot(0, c, i);
        s_post[0][i] = slot(1, c, i);
      }
    }
    if (a.part_pre != nullptr) store_end<8, EXACT, false>(a.part_pre + (int64_t)blockIdx.x * a.C, col, a.C, s_pre[HOLD ? c : 0]);
    if (a.part_post != nullptr) store_end<8, EXACT, false>(a.part_post + (int64_t)blockIdx.x * a.C, col, a.C, s_post[HOLD ? c : 0]);
  }
}

// Sums over the nb rows of partials in a fixed order: 64 columns per
// workgroup, sixteen row classes, then the sixteen sums in order; blockIdx.y
// picks the vector.  Of the second, both dw_post and dgate are made.
struct NormSums {
  const float* part[2];
  float* dw_pre;
  float* dw_post;
  float* dgate;
  const void* w_post;
  const void* gate;  // per channel
  float alpha;
  bool pf32;
};
__device__ __forceinline__ float param_at(const void* p, bool f32, int64_t i) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
__global__ __launch_bounds__(1024) void k_norm_sums(const NormSums a, int first, int64_t nb, int64_t C) {
  __shared__ float acc[16][64];
  const int vec = first + blockIdx.y;
  const float* part = a.part[vec];
  const int lane = threadIdx.x & 63, cls = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (col < C) {
    for (int64_t b = cls; b < nb; b += 16 * 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = b + 16 * i < nb ? part[(b + 16 * i) * C + col] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
  }
  acc[cls][lane] = sum;
  __syncthreads();
  if (cls == 0 && col < C) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += acc[i][lane];
    if (vec == 0) {
      a.dw_pre[col] = t;
    } else {
      t *= a.alpha;
      if (a.dw_post != nullptr) a.dw_post[col] = a.gate != nullptr ? t * param_at(a.gate, a.pf32, col) : t;
      if (a.dgate != nullptr) a.dgate[col] = a.w_post != nullptr ? t * param_at(a.w_post, a.pf32, col) : t;
    }
  }
}

// Chunks of eight channels per lane, and lanes of a row's workgroup (a multiple
// of 64).  Forward: one chunk up to 1024 lanes, then two (8192 x 7168 took 97 us
// with 896 lanes of one chunk, 99 with 448 of two).  Gradient: at most 512
// lanes where they hold a row ahead, so that each may have 256 registers (123
// us with 448 lanes of two chunks, 128 with 896 of one).
inline int forward_chunks(int64_t C) { return C > 8192 ? 2 : 1; }
inline bool backward_holds(int64_t C, uint32_t flags) {
  return C <= 4096 || (C <= 8192 && (flags & (FP8BLK_NORM_RES_F32 | FP8BLK_NORM_GATE_ROW)) !=
                                        (FP8BLK_NORM_RES_F32 | FP8BLK_NORM_GATE_ROW));
}
inline int backward_chunks(int64_t C) { return C > 4096 ? 2 : 1; }
inline int norm_lanes(int64_t C, int chunks) {
  return (int)(ceil_div(ceil_div(C, (int64_t)8 * chunks), (int64_t)64) * 64);
}

// Workgroups of either kernel: `per_cu` lanes on a compute unit, as many as the
// registers allow at a time (half or twice as many were 1-2 % slower in the
// forward, twice as many 7 % in the gradient, 8192 x 7168).
inline int64_t norm_blocks(int64_t M, int lanes, int64_t per_cu) {
  int64_t n = per_cu / lanes;
  n = (n < 1 ? 1 : n) * device_cus();
  return M < n ? M : n;
}
inline int64_t norm_backward_blocks(int64_t M, int64_t C) {
  return norm_blocks(M, norm_lanes(C, backward_chunks(C)), 512);
}

template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT>
void launch(const NormFwd& a, hipStream_t stream) {
  const int lanes = norm_lanes(a.C, NCH);
  hipLaunchKernelGGL((k_residual_norm<TX, NCH, GATE_ROW, EXACT, NT>), dim3((unsigned)norm_blocks(a.M, lanes, 2048)),
                     dim3((unsigned)lanes), 0, stream, a);
}
template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT, bool HOLD>
void launch(const NormBwd& a, hipStream_t stream) {
  hipLaunchKernelGGL((k_residual_norm_backward<TX, NCH, GATE_ROW, EXACT, NT, HOLD>),
                     dim3((unsigned)norm_backward_blocks(a.M, a.C)), dim3((unsigned)norm_lanes(a.C, NCH)), 0, stream,
                     a);
}

// The kernel for the arguments' types and sizes.
template <typename TX, bool GATE_ROW, bool EXACT, bool NT>
void launch_chunks(const NormFwd& a, hipStream_t stream) {
  if (forward_chunks(a.C) == 1) launch<TX, 1, GATE_ROW, EXACT, NT>(a, stream);
  else launch<TX, 2, GATE_ROW, EXACT, NT>(a, stream);
}
template <typename TX, bool GATE_ROW, bool EXACT, bool NT>
void launch_chunks(const NormBwd& a, hipStream_t stream) {
  if (!backward_holds(a.C, a.flags)) launch<TX, 2, GATE_ROW, EXACT, NT, false>(a, stream);
  else if (backward_chunks(a.C) == 1) launch<TX, 1, GATE_ROW, EXACT, NT, true>(a, stream);
  else launch<TX, 2, GATE_ROW, EXACT, NT, true>(a, stream);
}
template <typename TX, bool GATE_ROW, typename A>
void launch_exact(const A& a, bool nt, hipStream_t stream) {
  if (a.C % 8 != 0) return launch_chunks<TX, GATE_ROW, false, false>(a, stream);  // streamed 5 % slower: rows share lines
  return nt ? launch_chunks<TX, GATE_ROW, true, true>(a, stream) : launch_chunks<TX, GATE_ROW, true, false>(a, stream);
}
// moved: bytes that the call reads and writes.
template <typename A>
void launch_norm(const A& a, int64_t moved, hipStream_t stream) {
  const bool nt = moved >= kStreamBytes, gate_row = (a.flags & FP8BLK_NORM_GATE_ROW) != 0;
  if (a.flags & FP8BLK_NORM_RES_F32)
    gate_row ? launch_exact<float, true>(a, nt, stream) : launch_exact<float, false>(a, nt, stream);
  else
    gate_row ? launch_exact<uint16_t, true>(a, nt, stream) : launch_exact<uint16_t, false>(a, nt, stream);
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" fp8blk_status_t fp8blk_residual_norm(int64_t M, int64_t C, const void* x, int64_t ldx, const uint16_t* f,
                                                int64_t ldf, const void* w_post, const void* gate, int64_t ldg,
                                                float alpha, const void* w_pre, float eps, void* x_out, int64_t ldxo,
                                                uint16_t* n, int64_t ldn, uint8_t* q, int64_t ldq, float* s,
                                                float* rstd_post, float* rstd_pre, uint32_t flags, void* stream) {
  if (flags & ~(FP8BLK_SCALE_POW2 | FP8BLK_NORM_RES_F32 | FP8BLK_NORM_PARAM_F32 | FP8BLK_NORM_GATE_ROW))
    return FP8BLK_ERR_INVALID_ARG;
  if (M < 0 || C < 0 || !(eps >= 0.0f)) return FP8BLK_ERR_INVALID_ARG;
  const bool xf = (flags & FP8BLK_NORM_RES_F32) != 0, gr = (flags & FP8BLK_NORM_GATE_ROW) != 0;
  const uintptr_t pa = flags & FP8BLK_NORM_PARAM_F32 ? 4 : 2;
  if ((w_post != nullptr || gate != nullptr || rstd_post != nullptr) && f == nullptr && M > 0 && C > 0)
    return FP8BLK_ERR_INVALID_ARG;
  if (M == 0 || C == 0) return FP8BLK_OK;
  if (C > kNormMaxC) return FP8BLK_ERR_UNSUPPORTED;
  if (f == nullptr && w_pre == nullptr) return FP8BLK_ERR_INVALID_ARG;
  if (!matrix_ok(x, M, C, ldx, xf ? 4 : 2)) return FP8BLK_ERR_INVALID_ARG;
  if (f != nullptr && (!matrix_ok(f, M, C, ldf, 2) || !matrix_ok(x_out, M, C, ldxo, xf ? 4 : 2)))
    return FP8BLK_ERR_INVALID_ARG;
  if (f == nullptr && x_out != nullptr) return FP8BLK_ERR_INVALID_ARG;
  if (x_out == x && f != nullptr && ldxo != ldx) return FP8BLK_ERR_INVALID_ARG;
  if (!aligned(w_post, pa) || !aligned(w_pre, pa) || (gate == nullptr && gr)) return FP8BLK_ERR_INVALID_ARG;
  if (gate != nullptr && (gr ? !matrix_ok(gate, M, C, ldg, 2) : !aligned(gate, pa))) return FP8BLK_ERR_INVALID_ARG;
  if ((q == nullptr) != (s == nullptr)) return FP8BLK_ERR_INVALID_ARG;
  if (w_pre == nullptr ? (n != nullptr || q != nullptr || rstd_pre != nullptr) : (n == nullptr && q == nullptr))
    return FP8BLK_ERR_INVALID_ARG;
  if (n != nullptr && !matrix_ok(n, M, C, ldn, 2)) return FP8BLK_ERR_INVALID_ARG;
  if (q != nullptr && (!matrix_ok(q, M, C, ldq, 1) || !aligned(s, 4))) return FP8BLK_ERR_INVALID_ARG;
  if ((rstd_post != nullptr && w_post == nullptr) || !aligned(rstd_post, 4) || !aligned(rstd_pre, 4))
    return FP8BLK_ERR_INVALID_ARG;
  if ((flags & FP8BLK_SCALE_POW2) && q == nullptr) return FP8BLK_ERR_INVALID_ARG;
  const NormFwd a{x, f, w_post, gate, w_pre, x_out, n, q, s, rstd_post, rstd_pre,
                  M, C, ldx, ldf, ldg, ldxo, ldn, ldq, alpha, eps, flags};
  const int64_t xe = xf ? 4 : 2;
  launch_norm(a, M * C * (xe + (f != nullptr ? 2 + xe : 0) + (gr ? 2 : 0) + (n != nullptr ? 2 : 0) + (q != nullptr ? 1 : 0)),
              as_stream(stream));
  return launch_status();
}

extern "C" size_t fp8blk_residual_norm_backward_workspace_bytes(int64_t M, int64_t C) {
  if (M <= 0 || C <= 0 || C > kNormMaxC) return 0;
  return (size_t)(norm_backward_blocks(M, C) * C) * 2 * sizeof(float);
}

extern "C" fp8blk_status_t fp8blk_residual_norm_backward(
    int64_t M, int64_t C, const void* x_out, int64_t ldx, const void* dx_out, int64_t lddxo, const uint16_t* dn,
    int64_t lddn, const float* rstd_pre, const void* w_pre, const uint16_t* f, int64_t ldf, const float* rstd_post,
    const void* w_post, const void* gate, int64_t ldg, float alpha, void* dx, int64_t lddx, uint16_t* df, int64_t lddf,
    float* dw_pre, float* dw_post, void* dgate, int64_t lddg, void* workspace, size_t workspace_bytes, uint32_t flags,
    void* stream) {
  if (flags & ~(FP8BLK_NORM_RES_F32 | FP8BLK_NORM_PARAM_F32 | FP8BLK_NORM_GATE_ROW)) return FP8BLK_ERR_INVALID_ARG;
  if (M < 0 || C < 0) return FP8BLK_ERR_INVALID_ARG;
  if (C == 0) return FP8BLK_OK;
  if (C > kNormMaxC) return FP8BLK_ERR_UNSUPPORTED;
  const bool xf = (flags & FP8BLK_NORM_RES_F32) != 0, gr = (flags & FP8BLK_NORM_GATE_ROW) != 0;
  const uintptr_t pa = flags & FP8BLK_NORM_PARAM_F32 ? 4 : 2;
  const int64_t xe = xf ? 4 : 2;
  // which parts there are: by the parameters and gradients that no M empties
  const bool pre = dw_pre != nullptr, postw = dw_post != nullptr, gated = dgate != nullptr;
  if (!aligned(dw_pre, 4) || !aligned(dw_post, 4)) return FP8BLK_ERR_INVALID_ARG;
  if ((w_pre != nullptr) != pre || (w_post != nullptr) != postw) return FP8BLK_ERR_INVALID_ARG;
  if (!aligned(w_pre, pa) || !aligned(w_post, pa)) return FP8BLK_ERR_INVALID_ARG;
  if (gr) {
    if (M > 0 && (gate == nullptr || !gated)) return FP8BLK_ERR_INVALID_ARG;
    if (!matrix_ok(gate, M, C, ldg, 2) || !matrix_ok(dgate, M, C, lddg, 2)) return FP8BLK_ERR_INVALID_ARG;
  } else if ((gate != nullptr) != gated || !aligned(gate, pa) || !aligned(dgate, 4)) {
    return FP8BLK_ERR_INVALID_ARG;
  }
  if (M > 0) {
    if ((dn != nullptr) != pre || (rstd_pre != nullptr) != pre || (rstd_post != nullptr) != postw)
      return FP8BLK_ERR_INVALID_ARG;
    if ((f != nullptr) != (df != nullptr) || (f == nullptr && (postw || gated))) return FP8BLK_ERR_INVALID_ARG;
    if (dx_out == nullptr && dn == nullptr) return FP8BLK_ERR_INVALID_ARG;
    if (pre && (!matrix_ok(x_out, M, C, ldx, xe) || !matrix_ok(dn, M, C, lddn, 2) || !aligned(rstd_pre, 4)))
      return FP8BLK_ERR_INVALID_ARG;
    if (dx_out != nullptr && !matrix_ok(dx_out, M, C, lddxo, xe)) return FP8BLK_ERR_INVALID_ARG;
    if (dx != nullptr && !matrix_ok(dx, M, C, lddx, xe)) return FP8BLK_ERR_INVALID_ARG;
    if (f != nullptr && (!matrix_ok(f, M, C, ldf, 2) || !matrix_ok(df, M, C, lddf, 2) || !aligned(rstd_post, 4)))
      return FP8BLK_ERR_INVALID_ARG;
  }
  const bool sums = pre || postw || (gated && !gr);
  const int64_t nb = M > 0 ? norm_backward_blocks(M, C) : 0;
  if (sums && nb > 0 &&
      (workspace == nullptr || !aligned(workspace, 16) ||
       workspace_bytes < fp8blk_residual_norm_backward_workspace_bytes(M, C)))
    return FP8BLK_ERR_INVALID_ARG;
  float* part_pre = pre && nb > 0 ? reinterpret_cast<float*>(workspace) : nullptr;
  float* part_post =
      (postw || (gated && !gr)) && nb > 0 ? reinterpret_cast<float*>(workspace) + nb * C : nullptr;
  if (nb > 0) {
    const NormBwd a{x_out, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post, gate, dx, df,
                    gr ? reinterpret_cast<uint16_t*>(dgate) : nullptr, part_pre, part_post,
                    M, C, ldx, lddxo, lddn, ldf, ldg, lddx, lddf, lddg, alpha, flags};
    launch_norm(a, M * C * ((pre ? xe + 2 : 0) + (dx_out != nullptr ? xe : 0) + (dx != nullptr ? xe : 0) +
                            (f != nullptr ? 4 : 0) + (gr ? 4 : 0)), as_stream(stream));
    const fp8blk_status_t st = launch_status();
    if (st != FP8BLK_OK) return st;
  }
  if (sums) {
    const int first = pre ? 0 : 1, last = postw || (gated && !gr) ? 1 : 0;
    const NormSums a{{part_pre, part_post}, dw_pre, dw_post, gr ? nullptr : reinterpret_cast<float*>(dgate), w_post,
                     gr ? nullptr : gate, alpha, (flags & FP8BLK_NORM_PARAM_F32) != 0};
    hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)ceil_div(C, (int64_t)64), (unsigned)(last - first + 1)), dim3(1024),
                       0, as_stream(stream), a, first, nb, C);
    return launch_status();
  }
  return FP8BLK_OK;
}
