// Device-side building blocks of the operators around the GEMMs (gfx950):
// chunks of eight values in FP32 registers, loaded from and stored to BF16 or
// FP32 rows, and sums over a wave and a workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_device.h"

namespace fp8blk {

typedef float f32x2_l __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_l __attribute__((ext_vector_type(2)));

// Two FP32 values to BF16 (nearest even, NaN kept), `lo` in bits 15:0.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_l{lo, hi}, bf16x2_l));
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu); }

// 16 bytes at an address aligned only to the element: one dwordx4 access (the
// hardware takes unaligned global accesses).
struct __attribute__((packed, aligned(2))) U128 {
  uint32_t w[4];
};
__device__ __forceinline__ uint4 load_u128(const void* p) {
  const U128 u = *reinterpret_cast<const U128*>(p);
  return make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]);
}
__device__ __forceinline__ void store_u128(void* p, const uint4& v) {
  U128 u;
  u.w[0] = v.x; u.w[1] = v.y; u.w[2] = v.z; u.w[3] = v.w;
  *reinterpret_cast<U128*>(p) = u;
}

// Eight raw elements of a row: one 16-byte word for BF16, two for FP32.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 a;
};
template <>
struct Raw8<float> {
  uint4 a, b;
};

__device__ __forceinline__ void zero8(Raw8<uint16_t>& r) { r.a = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void zero8(Raw8<float>& r) { r.a = r.b = make_uint4(0u, 0u, 0u, 0u); }

// `avail` elements are left in the row; those past its end read as zero and
// are not touched in memory.
__device__ __forceinline__ void load8(Raw8<uint16_t>& r, const uint16_t* p, int64_t avail) {
  zero8(r);
  if (avail >= 8) {
    r.a = load_u128(p);
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < avail) w[j >> 1] |= (uint32_t)p[j] << ((j & 1) * 16);
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p, int64_t avail) {
  zero8(r);
  if (avail >= 8) {
    r.a = load_u128(p);
    r.b = load_u128(p + 4);
  } else {
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < avail) w[j] = __float_as_uint(p[j]);
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

__device__ __forceinline__ void unpack8(const Raw8<uint16_t>& r, float (&v)[8]) {
  v[0] = bf16_lo(r.a.x); v[1] = bf16_hi(r.a.x);
  v[2] = bf16_lo(r.a.y); v[3] = bf16_hi(r.a.y);
  v[4] = bf16_lo(r.a.z); v[5] = bf16_hi(r.a.z);
  v[6] = bf16_lo(r.a.w); v[7] = bf16_hi(r.a.w);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
  v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
  v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
  v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
  v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t avail, const float (&v)[8]) {
  const uint4 w = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  if (avail >= 8) {
    store_u128(p, w);
  } else {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < avail) p[j] = (uint16_t)(a[j >> 1] >> ((j & 1) * 16));
  }
}
__device__ __forceinline__ void store8(float* p, int64_t avail, const float (&v)[8]) {
  if (avail >= 8) {
    store_u128(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    store_u128(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < avail) p[j] = v[j];
  }
}

// Sum over the wave's 64 lanes, the same bits in every lane.  FP32: four DPP
// steps inside each row of 16 lanes, then the rows and the halves exchanged by
// register swaps; no LDS traffic, where a lane exchange by __shfl costs an LDS
// round trip per step.
template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_f32<0xB1>(v);   // quad_perm 1,0,3,2
  v += dpp_f32<0x4E>(v);   // quad_perm 2,3,0,1
  v += dpp_f32<0x141>(v);  // row_half_mirror
  v += dpp_f32<0x140>(v);  // row_mirror
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A barrier that orders LDS accesses only: global loads and stores in flight
// stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Sums of N values over the workgroup's `nw` (at most 16) waves, the same bits
// in every lane.  `red` holds N * 16 floats of LDS; there is one barrier, so
// consecutive calls take turns over two LDS arrays (a slower wave may still
// read the last one's).
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red, int nw) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (nw == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 16 + (threadIdx.x >> 6)] = v[i];
  }
  lds_barrier();
  const int w = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = row16_sum(w < nw ? red[i * 16 + w] : 0.0f);
}

}  // namespace fp8blk
