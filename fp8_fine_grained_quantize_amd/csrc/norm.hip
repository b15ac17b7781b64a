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
constexpr int64_t kPackMaxC = 512;  // rows up to here: several to a workgroup, each held by one wave or part of it
constexpr int kPackLanes = 512;     // most lanes of such a workgroup

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
  int group;  // lanes of a row where a workgroup takes several
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

// Which rows a lane works on.  A workgroup has one row at a time, or (PACK,
// rows of at most 512 channels) one for each group of 16, 32 or 64 lanes.
template <bool PACK>
struct Rows {
  int lane, lanes;      // of the row's
  int64_t first, step;  // the lane's rows
  __device__ __forceinline__ explicit Rows(int group) {
    lanes = PACK ? group : (int)blockDim.x;
    lane = PACK ? (int)threadIdx.x & (group - 1) : (int)threadIdx.x;
    const int per = PACK ? (int)blockDim.x / group : 1;
    first = PACK ? (int64_t)blockIdx.x * per + threadIdx.x / group : blockIdx.x;
    step = (int64_t)gridDim.x * per;
  }
  __device__ __forceinline__ int64_t col(int c) const { return ((int64_t)lane + (int64_t)c * lanes) * 8; }
  // Sums over the row's lanes (block_sum's LDS array where it is a workgroup's).
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N], float* red) const {
    if (PACK) group_sum<N>(v, lanes);
    else block_sum<N>(v, red, lanes >> 6);
  }
};

// What a lane reads of one row, before it is unpacked.
template <typename TX, int NCH, bool GATE_ROW, bool EXACT>
struct NormRow {
  RawV<TX, 8> x[NCH];
  RawV<uint16_t, 8> f[NCH], gate[GATE_ROW ? NCH : 1];
};

template <bool NT, typename TX, int NCH, bool GATE_ROW, bool EXACT, bool PACK>
__device__ __forceinline__ void load_row(NormRow<TX, NCH, GATE_ROW, EXACT>& r, const NormFwd& a, const Rows<PACK>& rows,
                                         int64_t row) {
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = rows.col(c);
    r.x[c] = load_end<8, EXACT, NT, !PACK>(reinterpret_cast<const TX*>(a.x) + row * a.ldx, col, a.C);
    if (a.f != nullptr) r.f[c] = load_end<8, EXACT, NT, !PACK>(a.f + row * a.ldf, col, a.C);
    if (GATE_ROW)
      r.gate[c] = load_end<8, EXACT, NT, !PACK>(reinterpret_cast<const uint16_t*>(a.gate) + row * a.ldg, col, a.C);
  }
}

// A workgroup takes the rows blockIdx.x, blockIdx.x + gridDim.x, ...; lane t
// holds the chunks of eight channels t, t + NT, ... (NCH of them), so that a
// 1x128 tile is one row of 16 lanes, and the parameters of its channels.  Rows
// of at most 512 channels lie several to a workgroup and need no barrier (PACK;
// 1048576 x 128, norm only: 100 us, 211 with a workgroup each).  The next row is
// loaded before the present one is worked on: the reductions and stores of one
// row cover the other's way from HBM, which bounds it.  8192 x 7168 (BF16, n and
// E4M3 out) takes 96 us, 530 MB at 5.5 TB/s; without the next row in flight and
// with the parameters read again for every row it took 162.  A decode step of 16
// rows takes 5.5 us: launch, four loads one after the other (w_post, gate and
// w_pre, each behind a branch on its type, then the row) and two reductions.
// Above 8192 channels two chunks a lane and 1024 lanes leave 128 registers: FP32 x
// with a gate per token or ragged rows, and BF16 x with both, keep 16 to 88 bytes
// a lane in scratch.
template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT, bool PACK>
__global__ __launch_bounds__(PACK ? kPackLanes : 1024) void k_residual_norm(const NormFwd a) {
  __shared__ float red[2][2][16];
  const Rows<PACK> rows(a.group);
  const float inv_c = 1.0f / (float)a.C;
  const bool pf32 = (a.flags & FP8BLK_NORM_PARAM_F32) != 0;
  float pc[NCH][8], wn[NCH][8];  // alpha * w_post * (gate per channel); w_pre
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = rows.col(c);
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
  if (!PACK || rows.first < a.M) load_row<NT>(next, a, rows, rows.first);
  int turn = 0;
  for (int64_t row = rows.first; row < a.M; row += rows.step, turn ^= 1) {
    const NormRow<TX, NCH, GATE_ROW, EXACT> cur = next;
    if (row + rows.step < a.M) load_row<NT>(next, a, rows, row + rows.step);
    float z[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      unpack_end<TX, 8, EXACT, !PACK>(cur.x[c], rows.col(c), a.C, z[c]);
    if (a.f != nullptr) {
      float r = 1.0f;
      if (a.w_post != nullptr) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          float f[8];
          unpack_end<uint16_t, 8, EXACT, !PACK>(cur.f[c], rows.col(c), a.C, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(f[i], f[i], sum[0]);
        }
        rows.sum(sum, red[turn][0]);
        r = rstd_of(sum[0], inv_c, a.eps);
        if (a.rstd_post != nullptr && rows.lane == 0) a.rstd_post[row] = r;
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int64_t col = rows.col(c);
        float f[8];
        unpack_end<uint16_t, 8, EXACT, !PACK>(cur.f[c], col, a.C, f);
        if (GATE_ROW) {
          float g[8];
          unpack_end<uint16_t, 8, EXACT, !PACK>(cur.gate[c], col, a.C, g);
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
    rows.sum(sum, red[turn][1]);
    const float r = rstd_of(sum[0], inv_c, a.eps);
    if (a.rstd_pre != nullptr && rows.lane == 0) a.rstd_pre[row] = r;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = rows.col(c), avail = a.C - col;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] = z[c][i] * r * wn[c][i];
      if (a.n != nullptr) store_end<8, EXACT, NT>(a.n + row * a.ldn, col, a.C, z[c]);
      if (a.q != nullptr) {
        float s;
        const uint2 codes = a.flags & FP8BLK_SCALE_POW2 ? quantize_tile<true>(z[c], s) : quantize_tile<false>(z[c], s);
        if (avail > 0) {
          store_codes8<EXACT, NT>(a.q + row * a.ldq + col, avail, codes);
          if ((rows.lane & 15) == 0) a.s[(col >> 7) * a.M + row] = s;
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
// + 16.  The norm's gradient alone (POST: there is an f) keeps half the
// registers, so twice the lanes are at work: 32768 x 2880 takes 127 us, 149 by
// the other kernel with no f, 65536 x 1025 113 / 236, 16384 x 7168 151 / 152; but
// 131072 x 1024 194 / 185, 32768 x 4096 185 / 177 and FP32 16384 x 7168 297 / 276.
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
  int group;  // lanes of a row where a workgroup takes several
};

// What a lane reads of one chunk of one row, before it is unpacked.
template <typename TX, bool GATE_ROW>
struct NormBwdChunk {
  RawV<TX, 8> x, dxo;
  RawV<uint16_t, 8> dn, f, gate;
};

template <bool EXACT, bool NT, bool LONG, bool POST, typename TX, bool GATE_ROW>
__device__ __forceinline__ void load_chunk(NormBwdChunk<TX, GATE_ROW>& r, const NormBwd& a, int64_t row, int64_t col) {
  r = {};
  if (a.w_pre != nullptr) {
    r.x = load_end<8, EXACT, NT, LONG>(reinterpret_cast<const TX*>(a.x) + row * a.ldx, col, a.C);
    r.dn = load_end<8, EXACT, NT, LONG>(a.dn + row * a.lddn, col, a.C);
  }
  if (a.dxo != nullptr)
    r.dxo = load_end<8, EXACT, NT, LONG>(reinterpret_cast<const TX*>(a.dxo) + row * a.lddxo, col, a.C);
  if (POST) r.f = load_end<8, EXACT, NT, LONG>(a.f + row * a.ldf, col, a.C);
  if (GATE_ROW)
    r.gate = load_end<8, EXACT, NT, LONG>(reinterpret_cast<const uint16_t*>(a.gate) + row * a.ldg, col, a.C);
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
// lanes (ragged rows of 4097 to 8192 channels with FP32 x or a gate per token keep
// 16 and 32 bytes a lane in scratch).  Where they would not fit beside the
// accumulators (C above 8192; FP32 x with a gate per token above 4096) 1024 lanes
// read factors and rows chunk by chunk, and once more (from L2) after the
// reduction, with the accumulators in LDS and no row ahead: 4096 x 16384 takes 231
// us, 805 MB at 3.5 TB/s.
template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT, bool HOLD, bool PACK, bool POST>
__global__ __launch_bounds__(PACK || (HOLD && POST) ? 512 : 1024) void k_residual_norm_backward(const NormBwd a) {
  constexpr int NH = HOLD ? NCH : 1, UNROLL = NH;  // without HOLD one chunk after the other
  // Rows that end inside a chunk: the last lane takes the row's last eight
  // channels, of which the lane before holds some too.  Both compute and store
  // the same for them; sums over the row leave out the last lane's share.  No
  // values are moved and no pieces stored while the row's other waves wait
  // (65536 x 2051: 327 us, 608 with the end's values moved to their places).
  constexpr int SUMS = POST ? 3 : 1;
  constexpr bool OVER = HOLD && !EXACT && !PACK, FULL = EXACT || OVER;
  __shared__ float red[2][3 * 16];
  const Rows<PACK> rows(a.group);
  const float inv_c = 1.0f / (float)a.C;
  auto col_of = [&](int c) { return OVER && rows.col(c) > a.C - 8 ? a.C - 8 : rows.col(c); };
  auto twice = [&](int c) { return (int)(rows.col(c) - col_of(c)); };  // channels of the chunk that a lane before holds
  auto store_col = [&](int c) { return OVER && twice(c) >= 8 ? a.C : col_of(c); };
  __shared__ float acc[HOLD ? PACK ? 8 * kPackLanes : 1 : 2 * NCH * 8 * 1024];
  float s_pre[NH][8], s_post[NH][8], pc_[NH][8], wn_[NH][8];
  // this lane's accumulator `vec` (0: dn h, 1: g h') of channel i of chunk c in LDS
  auto slot = [&](int vec, int c, int i) -> float& { return acc[((vec * NCH + c) * 8 + i) * 1024 + threadIdx.x]; };
  NormBwdChunk<TX, GATE_ROW> next[NH], cur_[NH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = col_of(c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (HOLD) s_pre[c][i] = s_post[c][i] = 0.0f;
      else slot(0, c, i) = slot(1, c, i) = 0.0f;
    }
    if (HOLD) {
      load_factors<GATE_ROW, FULL>(a, col, pc_[c], wn_[c]);
      if (!PACK || rows.first < a.M) load_chunk<FULL, NT, !PACK, POST>(next[c], a, rows.first, col);
    }
  }
  const bool pre = a.w_pre != nullptr, post = POST && a.w_post != nullptr;
  float next_pre = 0.0f, next_post = 1.0f;  // the statistics of the next row
  if (HOLD && rows.first < a.M) {
    if (pre) next_pre = a.rstd_pre[rows.first];
    if (post) next_post = a.rstd_post[rows.first];
  }
  int turn = 0;
  for (int64_t row = rows.first; row < a.M; row += rows.step, turn ^= 1) {
    float r_pre = next_pre, r_post = next_post;
    if (!HOLD) {
      if (pre) r_pre = a.rstd_pre[row];
      if (post) r_post = a.rstd_post[row];
    } else {
      if (OVER) wait_vmem();
      if (row + rows.step < a.M) {
        if (pre) next_pre = a.rstd_pre[row + rows.step];
        if (post) next_post = a.rstd_post[row + rows.step];
      }
#pragma unroll
      for (int c = 0; c < NH; ++c) {
        cur_[c] = next[c];
        if (row + rows.step < a.M)
          load_chunk<FULL, NT, !PACK, POST>(next[c], a, row + rows.step, col_of(c));
      }
    }
    float sum[SUMS] = {}, before[SUMS];  // before the present chunk
#pragma unroll UNROLL
    for (int c = 0; c < NCH; ++c) {
      float(&pc)[8] = pc_[HOLD ? c : 0];
      float(&wn)[8] = wn_[HOLD ? c : 0];
      NormBwdChunk<TX, GATE_ROW>& cur = cur_[HOLD ? c : 0];
      const int64_t col = col_of(c);
      if (!HOLD) {
        load_factors<GATE_ROW, FULL>(a, col, pc, wn);
        load_chunk<FULL, NT && HOLD, !PACK, POST>(cur, a, row, col);
      }
      if (OVER) {
#pragma unroll
        for (int i = 0; i < SUMS; ++i) before[i] = sum[i];
      }
      float h[8], v[8], g[8], hf[8], gt[8];
      unpack_end<TX, 8, FULL, !PACK>(cur.x, col, a.C, h);
      unpack_end<uint16_t, 8, FULL, !PACK>(cur.dn, col, a.C, v);
      unpack_end<TX, 8, FULL, !PACK>(cur.dxo, col, a.C, g);
      if (POST) unpack_end<uint16_t, 8, FULL, !PACK>(cur.f, col, a.C, hf);
      if (GATE_ROW) unpack_end<uint16_t, 8, FULL, !PACK>(cur.gate, col, a.C, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] *= r_pre;
        float& sp = HOLD ? s_pre[HOLD ? c : 0][i] : slot(0, c, i);
        sp = __builtin_fmaf(v[i], h[i], sp);
        v[i] *= wn[i];
        sum[0] = __builtin_fmaf(v[i], h[i], sum[0]);
        if (!POST) continue;
        float p = pc[i] * (hf[i] * r_post);
        if (GATE_ROW) p *= gt[i];
        sum[POST ? 1 : 0] = __builtin_fmaf(p, __builtin_fmaf(r_pre, v[i], g[i]), sum[POST ? 1 : 0]);
        sum[POST ? 2 : 0] = __builtin_fmaf(p, h[i], sum[POST ? 2 : 0]);
      }
      if (OVER && __ballot(twice(c) > 0) != 0) {  // the row's last wave: once more, without them
        asm volatile("");
#pragma unroll
        for (int i = 0; i < SUMS; ++i) sum[i] = twice(c) > 0 ? before[i] : sum[i];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          if (twice(c) == 0 || i < twice(c)) continue;
          sum[0] = __builtin_fmaf(v[i], h[i], sum[0]);
          if (!POST) continue;
          float p = pc[i] * (hf[i] * r_post);
          if (GATE_ROW) p *= gt[i];
          sum[POST ? 1 : 0] = __builtin_fmaf(p, __builtin_fmaf(r_pre, v[i], g[i]), sum[POST ? 1 : 0]);
          sum[POST ? 2 : 0] = __builtin_fmaf(p, h[i], sum[POST ? 2 : 0]);
        }
      }
    }
    rows.sum(sum, red[turn]);
    const float m = sum[0] * inv_c;
    const float m_post = post ? (sum[POST ? 1 : 0] - r_pre * m * sum[POST ? 2 : 0]) * inv_c : 0.0f;
#pragma unroll UNROLL
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = col_of(c);
      float(&pc)[8] = pc_[HOLD ? c : 0];
      float(&wn)[8] = wn_[HOLD ? c : 0];
      NormBwdChunk<TX, GATE_ROW>& cur = cur_[HOLD ? c : 0];
      if (!HOLD) {
        load_factors<GATE_ROW, FULL>(a, col, pc, wn);
        load_chunk<FULL, NT && HOLD, !PACK, POST>(cur, a, row, col);
      }
      float h[8], v[8], g[8];
      unpack_end<TX, 8, FULL, !PACK>(cur.x, col, a.C, h);
      unpack_end<uint16_t, 8, FULL, !PACK>(cur.dn, col, a.C, v);
      unpack_end<TX, 8, FULL, !PACK>(cur.dxo, col, a.C, g);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        g[i] = __builtin_fmaf(r_pre, __builtin_fmaf(-(h[i] * r_pre), m, v[i] * wn[i]), g[i]);
      if (a.dx != nullptr) store_end<8, FULL, NT>(reinterpret_cast<TX*>(a.dx) + row * a.lddx, store_col(c), a.C, g);
      if (!POST) continue;
      unpack_end<uint16_t, 8, FULL, !PACK>(cur.f, col, a.C, h);
      float gt[8];
      if (GATE_ROW) unpack_end<uint16_t, 8, FULL, !PACK>(cur.gate, col, a.C, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] *= r_post;
        v[i] = g[i] * h[i];  // times its factors: the terms of dw_post and dgate
        float d = pc[i] * g[i];
        if (GATE_ROW) d *= gt[i];
        float& sp = HOLD ? s_post[HOLD ? c : 0][i] : slot(1, c, i);
        sp += GATE_ROW ? v[i] * gt[i] : v[i];
        // df = d without a norm, whatever f holds: 0 times an infinite f would be NaN
        g[i] = post ? r_post * __builtin_fmaf(-h[i], m_post, d) : d;
      }
      if (GATE_ROW) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= pc[i];
        store_end<8, FULL, NT>(a.dgate_row + row * a.lddg, store_col(c), a.C, v);
      }
      store_end<8, FULL, NT>(a.df + row * a.lddf, store_col(c), a.C, g);
    }
  }
  if (PACK) {  // the groups' accumulators are added in order: one row of partials
#pragma unroll
    for (int vec = 0; vec < 2; ++vec) {
      float* part = vec == 0 ? a.part_pre : a.part_post;
      if (part == nullptr) continue;
      if (vec == 1) __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[threadIdx.x * 8 + i] = vec == 0 ? s_pre[0][i] : s_post[0][i];
      __syncthreads();
      for (int col = threadIdx.x; col < a.C; col += blockDim.x) {
        float t = 0.0f;
        for (int g = 0; g < (int)blockDim.x; g += rows.lanes) t += acc[g * 8 + col];
        part[(int64_t)blockIdx.x * a.C + col] = t;
      }
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if (!HOLD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_pre[0][i] = slot(0, c, i);
        s_post[0][i] = slot(1, c, i);
      }
    }
    const int64_t part = (int64_t)blockIdx.x * a.C, at = store_col(c);
    if (a.part_pre != nullptr) store_end<8, FULL, false>(a.part_pre + part, at, a.C, s_pre[HOLD ? c : 0]);
    if (a.part_post != nullptr) store_end<8, FULL, false>(a.part_post + part, at, a.C, s_post[HOLD ? c : 0]);
  }
}

// Sums over the nb rows of partials in a fixed order: kSumCols columns per
// workgroup, 1024 / kSumCols row classes, then their sums in order; blockIdx.y
// picks the vector.  Of the second, both dw_post and dgate are made.  Dependent
// loads bound it (8192 x 1024, gradient and sums: 30 us, 32 with 64 columns).
constexpr int kSumCols = 32;
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
  constexpr int CLASSES = 1024 / kSumCols;
  __shared__ float acc[CLASSES][kSumCols];
  const int vec = first + blockIdx.y;
  const float* part = a.part[vec];
  const int lane = threadIdx.x % kSumCols, cls = threadIdx.x / kSumCols;
  const int64_t col = (int64_t)blockIdx.x * kSumCols + lane;
  float sum = 0.0f;
  if (col < C) {
    for (int64_t b = cls; b < nb; b += CLASSES * 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = b + CLASSES * i < nb ? part[(b + CLASSES * i) * C + col] : 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
  }
  acc[cls][lane] = sum;
  __syncthreads();
  if (cls == 0 && col < C) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < CLASSES; ++i) t += acc[i][lane];
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
// with 896 lanes of one chunk, 99 with 448 of two).  Gradient with an f: at most
// 512 lanes where they hold a row ahead, so that each may have 256 registers
// (125 us with 448 lanes of two chunks, 127 with 896 of one); without one, as
// the forward.
inline int forward_chunks(int64_t C) { return C > 8192 ? 2 : 1; }
inline bool backward_holds(int64_t C, uint32_t flags) {
  constexpr uint32_t wide = FP8BLK_NORM_RES_F32 | FP8BLK_NORM_GATE_ROW;
  return C <= 4096 || (C <= 8192 && (flags & wide) != wide);
}
inline int backward_chunks(int64_t C, bool post) { return C > (post ? 4096 : 8192) ? 2 : 1; }
inline int norm_lanes(int64_t C, int chunks) {
  return (int)(ceil_div(ceil_div(C, (int64_t)8 * chunks), (int64_t)64) * 64);
}

// Workgroups of either kernel: `per_cu` lanes on a compute unit, as many as the
// registers allow at a time (half or twice as many were 1-2 % slower in the
// forward to E4M3, half 2 % faster without the codes, twice as many 8 % slower in
// the gradient, 8192 x 7168; 768 lanes instead of 512 in the gradient, 65536 x
// 2048: 298 us, 272).  The gradient of the norm alone has 1024: with 512, 32768 x
// 2880 takes 140 us, not 127, and 65536 x 1025 140, not 113, but 131072 x 1024
// 173, not 193.
inline int64_t norm_blocks(int64_t M, int lanes, int64_t per_cu) {
  int64_t n = per_cu / lanes;
  n = (n < 1 ? 1 : n) * device_cus();
  return M < n ? M : n;
}
// Rows of at most kPackMaxC channels: lanes of a row, and of a workgroup, the
// fewest that reach every compute unit once (gradient of 512 x 128: 7.6 us in
// workgroups of 64 lanes, 9.5 in 512; 1048576 x 128, norm only: 105 in 64, 99 in
// 512, gradient 204 / 189).
inline int norm_group(int64_t C) { return C <= 128 ? 16 : C <= 256 ? 32 : 64; }
inline int packed_lanes(int64_t M, int64_t C) {
  int lanes = 64;
  while (lanes < kPackLanes && M > (int64_t)(lanes / norm_group(C)) * device_cus()) lanes *= 2;
  return lanes;
}
inline int64_t packed_blocks(int64_t M, int64_t C, int64_t per_cu) {
  const int lanes = packed_lanes(M, C);
  return norm_blocks(ceil_div(M, (int64_t)(lanes / norm_group(C))), lanes, per_cu);
}
inline int64_t norm_backward_blocks(int64_t M, int64_t C, bool post) {
  const int64_t per_cu = post ? 512 : 1024;
  return C <= kPackMaxC ? packed_blocks(M, C, per_cu) : norm_blocks(M, norm_lanes(C, backward_chunks(C, post)), per_cu);
}

template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT, bool PACK>
void launch(const NormFwd& a, hipStream_t stream) {
  const int lanes = PACK ? packed_lanes(a.M, a.C) : norm_lanes(a.C, NCH);
  const int64_t blocks = PACK ? packed_blocks(a.M, a.C, 2048) : norm_blocks(a.M, lanes, 2048);
  hipLaunchKernelGGL((k_residual_norm<TX, NCH, GATE_ROW, EXACT, NT, PACK>), dim3((unsigned)blocks),
                     dim3((unsigned)lanes), 0, stream, a);
}
template <typename TX, int NCH, bool GATE_ROW, bool EXACT, bool NT, bool HOLD, bool PACK, bool POST>
void launch(const NormBwd& a, hipStream_t stream) {
  hipLaunchKernelGGL((k_residual_norm_backward<TX, NCH, GATE_ROW, EXACT, NT, HOLD, PACK, POST>),
                     dim3((unsigned)norm_backward_blocks(a.M, a.C, POST)),
                     dim3((unsigned)(PACK ? packed_lanes(a.M, a.C) : norm_lanes(a.C, NCH))), 0, stream, a);
}

// The kernel for the arguments' types and sizes.
template <typename TX, bool GATE_ROW, bool EXACT, bool NT>
void launch_chunks(const NormFwd& a, hipStream_t stream) {
  if (a.C <= kPackMaxC) launch<TX, 1, GATE_ROW, EXACT, NT, true>(a, stream);
  else if (forward_chunks(a.C) == 1) launch<TX, 1, GATE_ROW, EXACT, NT, false>(a, stream);
  else launch<TX, 2, GATE_ROW, EXACT, NT, false>(a, stream);
}
template <typename TX, bool GATE_ROW, bool EXACT, bool NT, bool POST>
void launch_held(const NormBwd& a, hipStream_t stream) {
  if (a.C <= kPackMaxC) return launch<TX, 1, GATE_ROW, EXACT, NT, true, true, POST>(a, stream);
  if (a.C > 8192) return launch<TX, 2, GATE_ROW, EXACT, NT, false, false, POST>(a, stream);
  if constexpr (POST) {
    if (!backward_holds(a.C, a.flags)) return launch<TX, 1, GATE_ROW, EXACT, NT, false, false, true>(a, stream);
    if constexpr (!(GATE_ROW && sizeof(TX) == 4))
      if (a.C > 4096) return launch<TX, 2, GATE_ROW, EXACT, NT, true, false, true>(a, stream);
  }
  launch<TX, 1, GATE_ROW, EXACT, NT, true, false, POST>(a, stream);
}
template <typename TX, bool GATE_ROW, bool EXACT, bool NT>
void launch_chunks(const NormBwd& a, hipStream_t stream) {
  if (GATE_ROW || a.f != nullptr) launch_held<TX, GATE_ROW, EXACT, NT, true>(a, stream);
  else launch_held<TX, false, EXACT, NT, false>(a, stream);
}
template <typename TX, bool GATE_ROW, typename A>
void launch_exact(const A& a, bool nt, hipStream_t stream) {
  if (a.C % 8 != 0)  // streamed 5 % slower: rows share lines
    return launch_chunks<TX, GATE_ROW, false, false>(a, stream);
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
                  M, C, ldx, ldf, ldg, ldxo, ldn, ldq, alpha, eps, flags, norm_group(C)};
  const int64_t xe = xf ? 4 : 2;
  const int64_t each = xe + (f != nullptr ? 2 + xe : 0) + (gr ? 2 : 0) + (n != nullptr ? 2 : 0) + (q != nullptr ? 1 : 0);
  launch_norm(a, M * C * each, as_stream(stream));
  return launch_status();
}

extern "C" size_t fp8blk_residual_norm_backward_workspace_bytes(int64_t M, int64_t C) {
  if (M <= 0 || C <= 0 || C > kNormMaxC) return 0;
  const int64_t both = 2 * norm_backward_blocks(M, C, true), one = norm_backward_blocks(M, C, false);
  return (size_t)((both > one ? both : one) * C) * sizeof(float);
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
  const int64_t nb = M > 0 ? norm_backward_blocks(M, C, f != nullptr) : 0;
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
                    M, C, ldx, lddxo, lddn, ldf, ldg, lddx, lddf, lddg, alpha, flags, norm_group(C)};
    launch_norm(a, M * C * ((pre ? xe + 2 : 0) + (dx_out != nullptr ? xe : 0) + (dx != nullptr ? xe : 0) +
                            (f != nullptr ? 4 : 0) + (gr ? 4 : 0)), as_stream(stream));
    const fp8blk_status_t st = launch_status();
    if (st != FP8BLK_OK) return st;
  }
  if (sums) {
    const int first = pre ? 0 : 1, last = postw || (gated && !gr) ? 1 : 0;
    const NormSums a{{part_pre, part_post}, dw_pre, dw_post, gr ? nullptr : reinterpret_cast<float*>(dgate), w_post,
                     gr ? nullptr : gate, alpha, (flags & FP8BLK_NORM_PARAM_F32) != 0};
    const unsigned vecs = (unsigned)(last - first + 1);
    hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)ceil_div(C, (int64_t)kSumCols), vecs), dim3(1024), 0,
                       as_stream(stream), a, first, nb, C);
    return launch_status();
  }
  return FP8BLK_OK;
}
