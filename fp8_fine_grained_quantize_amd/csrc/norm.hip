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
__device__ __forceinline__ void load_param8(const void* p, bool f32, int64_t col, int64_t avail, float (&v)[8]) {
  if (f32) {
    Raw8<float> r;
    load8(r, reinterpret_cast<const float*>(p) + col, avail);
    unpack8(r, v);
  } else {
    Raw8<uint16_t> r;
    load8(r, reinterpret_cast<const uint16_t*>(p) + col, avail);
    unpack8(r, v);
  }
}

// The 1x128 tile of n that a row of 16 lanes holds, eight values each.  The
// default quotient is fl32(n * fl64(1/s)), the correctly rounded n / s for all
// FP32 n and s (see k_requant_128x1); power-of-two scales multiply by the
// exact reciprocal.
template <bool POW2>
__device__ __forceinline__ uint2 quantize_tile(const float (&n)[8], float& s) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(n[i]) & 0x7FFFFFFFu);
  const TileScale ts = make_scale<POW2, false>(row16_max(a));
  s = ts.s;
  float y[8];
  if (POW2 && !ts.slow) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = n[i] * ts.r;
  } else {
    const double r = 1.0 / (double)ts.s;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf((float)((double)n[i] * r), -kE4M3Max), kE4M3Max);
  }
  uint2 c;
  c.x = pack4_e4m3(y[0], y[1], y[2], y[3]);
  c.y = pack4_e4m3(y[4], y[5], y[6], y[7]);
  return c;
}

__device__ __forceinline__ void store_codes8(uint8_t* p, int64_t avail, uint2 c) {
  if (avail >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < avail) p[j] = (uint8_t)((j < 4 ? c.x : c.y) >> ((j & 3) * 8));
}

// One workgroup per row; lane t holds the chunks of eight channels t, t + NT,
// ... (NCH of them), so that a 1x128 tile is one row of 16 lanes.
template <typename TX, int NCH>
__global__ __launch_bounds__(1024) void k_residual_norm(const NormFwd a) {
  __shared__ float red[2][16];
  const int nt = blockDim.x, nw = nt >> 6;
  const int64_t row = blockIdx.x;
  const float inv_c = 1.0f / (float)a.C;
  const bool pf32 = (a.flags & FP8BLK_NORM_PARAM_F32) != 0;
  float z[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
    Raw8<TX> r;
    load8(r, reinterpret_cast<const TX*>(a.x) + row * a.ldx + col, a.C - col);
    unpack8(r, z[c]);
  }
  if (a.f != nullptr) {
    float f[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
      Raw8<uint16_t> r;
      load8(r, a.f + row * a.ldf + col, a.C - col);
      unpack8(r, f[c]);
    }
    if (a.w_post != nullptr) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(f[c][i], f[c][i], sum[0]);
      block_sum<1>(sum, red[0], nw);
      const float r = 1.0f / sqrtf(sum[0] * inv_c + a.eps);
      if (a.rstd_post != nullptr && threadIdx.x == 0) a.rstd_post[row] = r;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
        float w[8];
        load_param8(a.w_post, pf32, col, a.C - col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[c][i] = f[c][i] * r * w[i];
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
      if (a.gate != nullptr) {
        float g[8];
        if (a.flags & FP8BLK_NORM_GATE_ROW)
          load_param8(reinterpret_cast<const uint16_t*>(a.gate) + row * a.ldg, false, col, a.C - col, g);
        else
          load_param8(a.gate, pf32, col, a.C - col, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[c][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] = __builtin_fmaf(a.alpha, f[c][i], z[c][i]);
      store8(reinterpret_cast<TX*>(a.x_out) + row * a.ldxo + col, a.C - col, z[c]);
    }
  }
  if (a.w_pre == nullptr) return;
  float sum[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(z[c][i], z[c][i], sum[0]);
  block_sum<1>(sum, red[1], nw);
  const float r = 1.0f / sqrtf(sum[0] * inv_c + a.eps);
  if (a.rstd_pre != nullptr && threadIdx.x == 0) a.rstd_pre[row] = r;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t chunk = (int64_t)threadIdx.x + (int64_t)c * nt, col = chunk * 8, avail = a.C - col;
    float w[8];
    load_param8(a.w_pre, pf32, col, avail, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[c][i] = z[c][i] * r * w[i];
    if (a.n != nullptr) store8(a.n + row * a.ldn + col, avail, z[c]);
    if (a.q != nullptr) {
      float s;
      const uint2 codes = a.flags & FP8BLK_SCALE_POW2 ? quantize_tile<true>(z[c], s) : quantize_tile<false>(z[c], s);
      if (avail > 0) {
        store_codes8(a.q + row * a.ldq + col, avail, codes);
        if ((threadIdx.x & 15) == 0) a.s[(chunk >> 4) * a.M + row] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient.  A workgroup takes the rows blockIdx.x, blockIdx.x + gridDim.x, ...
// and keeps its share of the sums over rows (dw_pre, dw_post, dgate) in
// registers; at the end it writes them as one row of partials, which
// k_norm_sums adds up in order.
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
  float* part_gate;
  int64_t M, C, ldx, lddxo, lddn, ldf, ldg, lddx, lddf, lddg;
  float alpha;
  uint32_t flags;
};

template <typename TX, int NCH>
__global__ __launch_bounds__(1024) void k_residual_norm_backward(const NormBwd a) {
  __shared__ float red[2][16];
  const int nt = blockDim.x, nw = nt >> 6;
  const float inv_c = 1.0f / (float)a.C;
  const bool pf32 = (a.flags & FP8BLK_NORM_PARAM_F32) != 0;
  const bool gate_row = (a.flags & FP8BLK_NORM_GATE_ROW) != 0;
  float s_pre[NCH][8], s_post[NCH][8], s_gate[NCH][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[c][i] = s_post[c][i] = s_gate[c][i] = 0.0f;

  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    float g[NCH][8];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[c][i] = 0.0f;
      if (a.dxo != nullptr) {
        Raw8<TX> r;
        load8(r, reinterpret_cast<const TX*>(a.dxo) + row * a.lddxo + col, a.C - col);
        unpack8(r, g[c]);
      }
    }
    if (a.w_pre != nullptr) {
      float h[NCH][8], v[NCH][8];
      float sum[1] = {0.0f};
      const float r = a.rstd_pre[row];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8, avail = a.C - col;
        Raw8<TX> rx;
        Raw8<uint16_t> rd;
        float w[8];
        load8(rx, reinterpret_cast<const TX*>(a.x) + row * a.ldx + col, avail);
        load8(rd, a.dn + row * a.lddn + col, avail);
        load_param8(a.w_pre, pf32, col, avail, w);
        unpack8(rx, h[c]);
        unpack8(rd, v[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[c][i] *= r;
          s_pre[c][i] = __builtin_fmaf(v[c][i], h[c][i], s_pre[c][i]);
          v[c][i] *= w[i];
          sum[0] = __builtin_fmaf(v[c][i], h[c][i], sum[0]);
        }
      }
      block_sum<1>(sum, red[0], nw);
      const float mean = sum[0] * inv_c;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] += r * __builtin_fmaf(-h[c][i], mean, v[c][i]);
    }
    if (a.dx != nullptr) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
        store8(reinterpret_cast<TX*>(a.dx) + row * a.lddx + col, a.C - col, g[c]);
      }
    }
    if (a.f == nullptr) {
      __syncthreads();  // red[0] is read by all before the next row writes it
      continue;
    }
    float h[NCH][8];
    float sum[1] = {0.0f};
    const float r = a.w_post != nullptr ? a.rstd_post[row] : 1.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8, avail = a.C - col;
      Raw8<uint16_t> rf;
      float w[8], gt[8], dg[8];
      load8(rf, a.f + row * a.ldf + col, avail);
      unpack8(rf, h[c]);
      if (a.w_post != nullptr) load_param8(a.w_post, pf32, col, avail, w);
      if (a.gate != nullptr) {
        if (gate_row)
          load_param8(reinterpret_cast<const uint16_t*>(a.gate) + row * a.ldg, false, col, avail, gt);
        else
          load_param8(a.gate, pf32, col, avail, gt);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float d = a.alpha * g[c][i];
        h[c][i] *= r;
        dg[i] = d * (a.w_post != nullptr ? h[c][i] * w[i] : h[c][i]);
        if (a.gate != nullptr) d *= gt[i];
        if (a.w_post != nullptr) {
          s_post[c][i] = __builtin_fmaf(d, h[c][i], s_post[c][i]);
          d *= w[i];
          sum[0] = __builtin_fmaf(d, h[c][i], sum[0]);
        }
        s_gate[c][i] += dg[i];
        g[c][i] = d;
      }
      if (a.dgate_row != nullptr) store8(a.dgate_row + row * a.lddg + col, avail, dg);
    }
    if (a.w_post != nullptr) {
      block_sum<1>(sum, red[1], nw);
      const float mean = sum[0] * inv_c;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] = r * __builtin_fmaf(-h[c][i], mean, g[c][i]);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8;
      store8(a.df + row * a.lddf + col, a.C - col, g[c]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int64_t col = ((int64_t)threadIdx.x + (int64_t)c * nt) * 8, avail = a.C - col;
    if (a.part_pre != nullptr) store8(a.part_pre + (int64_t)blockIdx.x * a.C + col, avail, s_pre[c]);
    if (a.part_post != nullptr) store8(a.part_post + (int64_t)blockIdx.x * a.C + col, avail, s_post[c]);
    if (a.part_gate != nullptr) store8(a.part_gate + (int64_t)blockIdx.x * a.C + col, avail, s_gate[c]);
  }
}

// out[c] = sum over the nb rows of part, in a fixed order: 64 columns per
// workgroup, sixteen row classes, then the sixteen sums in order.
struct NormSums {
  const float* part[3];
  float* out[3];
};
__global__ __launch_bounds__(1024) void k_norm_sums(const NormSums a, int64_t nb, int64_t C) {
  __shared__ float acc[16][64];
  const float* part = a.part[blockIdx.y];
  const int lane = threadIdx.x & 63, cls = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (col < C)
    for (int64_t b = cls; b < nb; b += 16) sum += part[b * C + col];
  acc[cls][lane] = sum;
  __syncthreads();
  if (cls == 0 && col < C) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += acc[i][lane];
    a.out[blockIdx.y][col] = t;
  }
}

// Lanes of a row's workgroup, and chunks per lane (1 or 2).
inline int norm_lanes(int64_t C) {
  const int64_t chunks = ceil_div(C, (int64_t)8);
  const int64_t per = chunks > 1024 ? ceil_div(chunks, (int64_t)2) : chunks;
  return (int)(ceil_div(per, (int64_t)64) * 64);
}

// Workgroups of the gradient kernel.
inline int64_t norm_backward_blocks(int64_t M, int64_t C) {
  int64_t per_cu = 2048 / norm_lanes(C);
  if (per_cu > 4) per_cu = 4;
  const int64_t cap = per_cu * device_cus();
  return M < cap ? M : cap;
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
  if (C > kNormMaxC || M > 0x3FFFFF) return FP8BLK_ERR_UNSUPPORTED;
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
  const dim3 grid((unsigned)M), block((unsigned)norm_lanes(C));
  const bool two = C > 8192;
  if (xf) {
    if (two) hipLaunchKernelGGL((k_residual_norm<float, 2>), grid, block, 0, as_stream(stream), a);
    else hipLaunchKernelGGL((k_residual_norm<float, 1>), grid, block, 0, as_stream(stream), a);
  } else {
    if (two) hipLaunchKernelGGL((k_residual_norm<uint16_t, 2>), grid, block, 0, as_stream(stream), a);
    else hipLaunchKernelGGL((k_residual_norm<uint16_t, 1>), grid, block, 0, as_stream(stream), a);
  }
  return launch_status();
}

extern "C" size_t fp8blk_residual_norm_backward_workspace_bytes(int64_t M, int64_t C) {
  if (M <= 0 || C <= 0 || C > kNormMaxC) return 0;
  return (size_t)(norm_backward_blocks(M, C) * C) * 3 * sizeof(float);
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
  float* ws = reinterpret_cast<float*>(workspace);
  NormSums ns{};
  int nv = 0;
  auto part = [&](void* out) -> float* {
    if (out == nullptr) return nullptr;
    float* p = ws + (int64_t)nv * nb * C;
    ns.part[nv] = p;
    ns.out[nv++] = reinterpret_cast<float*>(out);
    return nb > 0 ? p : nullptr;
  };
  float* part_pre = part(dw_pre);
  float* part_post = part(dw_post);
  float* part_gate = part(gr ? nullptr : dgate);
  if (nb > 0) {
    const NormBwd a{x_out, dx_out, dn, rstd_pre, w_pre, f, rstd_post, w_post, gate, dx, df,
                    gr ? reinterpret_cast<uint16_t*>(dgate) : nullptr, part_pre, part_post, part_gate,
                    M, C, ldx, lddxo, lddn, ldf, ldg, lddx, lddf, lddg, alpha, flags};
    const dim3 grid((unsigned)nb), block((unsigned)norm_lanes(C));
    const bool two = C > 8192;
    if (xf) {
      if (two) hipLaunchKernelGGL((k_residual_norm_backward<float, 2>), grid, block, 0, as_stream(stream), a);
      else hipLaunchKernelGGL((k_residual_norm_backward<float, 1>), grid, block, 0, as_stream(stream), a);
    } else {
      if (two) hipLaunchKernelGGL((k_residual_norm_backward<uint16_t, 2>), grid, block, 0, as_stream(stream), a);
      else hipLaunchKernelGGL((k_residual_norm_backward<uint16_t, 1>), grid, block, 0, as_stream(stream), a);
    }
    const fp8blk_status_t st = launch_status();
    if (st != FP8BLK_OK) return st;
  }
  if (nv > 0) {
    hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)ceil_div(C, (int64_t)64), (unsigned)nv), dim3(1024), 0,
                       as_stream(stream), ns, nb, C);
    return launch_status();
  }
  return FP8BLK_OK;
}
