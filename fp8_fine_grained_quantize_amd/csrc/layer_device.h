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

// Pointers to global memory, told to the compiler where it cannot see it.
template <typename T>
using Global = __attribute__((address_space(1))) T;
template <typename T>
__device__ __forceinline__ Global<T>* global(T* p) { return (Global<T>*)p; }

// V elements of either type at an address aligned only to the element (the
// hardware takes unaligned global accesses), as FP32.  NT: streamed past the
// caches (see kStreamBytes in layer_host.h).
template <int N>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(N)));
  typedef type unaligned __attribute__((aligned(2)));
};
template <typename T, int V>
using RawV = typename Words<V * (int)sizeof(T) / 4>::type;
template <int V, bool NT, typename T>
__device__ __forceinline__ RawV<T, V> load_raw(const Global<const T>* p) {
  auto* q = (const Global<const typename Words<V * (int)sizeof(T) / 4>::unaligned>*)p;
  return NT ? __builtin_nontemporal_load(q) : *q;
}
template <typename T, int V>
__device__ __forceinline__ void unpack_v(const RawV<T, V>& r, float (&v)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = __uint_as_float(r[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      v[2 * j] = bf16_lo(r[j]);
      v[2 * j + 1] = bf16_hi(r[j]);
    }
  }
}
template <bool NT, int N>
__device__ __forceinline__ void store_words(Global<void>* p, const typename Words<N>::type& r) {
  auto* q = (Global<typename Words<N>::unaligned>*)p;
  if (NT) __builtin_nontemporal_store(r, q);
  else *q = r;
}
template <int V, bool NT>
__device__ __forceinline__ void store_v(Global<float>* p, const float (&v)[V]) {
  typename Words<V>::type r;
#pragma unroll
  for (int j = 0; j < V; ++j) r[j] = __float_as_uint(v[j]);
  store_words<NT, V>(p, r);
}
template <int V, bool NT>
__device__ __forceinline__ void store_v(Global<uint16_t>* p, const float (&v)[V]) {
  typename Words<V / 2>::type r;
#pragma unroll
  for (int j = 0; j < V / 2; ++j) r[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
  store_words<NT, V / 2>(p, r);
}
// Streaming pays where a lane's piece is one access: eight FP32 values are two,
// 32 bytes apart from lane to lane, and a line that is streamed can be gone
// before the second.  Norm of FP32 rows, every tensor separate: 65536 x 2048 330
// us streamed and 306 not, its gradient 461 / 451; gradient of 1048576 x 128 377 /
// 350; of 32768 x 7168 forward 520 / 517, but its gradient 746 / 761.
template <int V, typename T>
constexpr bool one_access() { return V * sizeof(T) <= 16; }

// V elements of a row of C from column col on, where the row may end inside
// them or before: values past its end are zero and memory past it is not
// touched.  EXACT: C is a multiple of V.  Otherwise the last V elements of the
// row are loaded and unpack_end moves them to their places, so that a row's
// end costs no branch and no wait where it is loaded (rows shorter than V come
// element by element; LONG: there are none).
template <int V, bool EXACT, bool NT, bool LONG = false, typename T>
__device__ __forceinline__ RawV<T, V> load_end(const T* row, int64_t col, int64_t C) {
  if (EXACT) {
    RawV<T, V> r{};
    if (col < C) r = load_raw<V, NT && one_access<V, T>()>(global(row + col));
    return r;
  }
  if (LONG || C >= V) return load_raw<V, NT && one_access<V, T>()>(global(row + (col < C - V ? col : C - V)));
  RawV<T, V> r{};
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (col + j >= C) continue;
    if constexpr (sizeof(T) == 4) r[j] = __float_as_uint(row[col + j]);
    else r[j >> 1] |= (uint32_t)row[col + j] << ((j & 1) * 16);
  }
  return r;
}
template <typename T, int V, bool EXACT, bool LONG = false>
__device__ __forceinline__ void unpack_end(const RawV<T, V>& r, int64_t col, int64_t C, float (&v)[V]) {
  unpack_v<T, V>(r, v);
  if (EXACT || (!LONG && C < V)) return;
  const int64_t d = col + V - C;  // elements that precede column col in r
  if (__ballot(d > 0) == 0) return;  // every wave but the row's last one
  asm volatile("");                  // keeps the branch: the moves are as much work as all else
#pragma unroll
  for (int k = 1; k < V; k *= 2) {
    const bool move = d > 0 && (d & k) != 0;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = move ? (j + k < V ? v[j + k] : 0.0f) : v[j];
  }
  if (d >= V) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.0f;
  }
}
// The elements inside the row are stored, an end in pieces of four, two and one.
template <int V, bool EXACT, bool NT, typename T>
__device__ __forceinline__ void store_end(T* row, int64_t col, int64_t C, const float (&v)[V]) {
  const int64_t avail = C - col;
  if (EXACT ? avail > 0 : avail >= V) {
    store_v<V, NT && one_access<V, T>()>(global(row + col), v);
    return;
  }
  if (EXACT || avail <= 0) return;
  T* p = row + col;
  int at = 0;  // elements stored so far: a multiple of the piece's size
#pragma unroll
  for (int n = V / 2; n >= 1; n /= 2) {
    if (!(avail & n)) continue;
#pragma unroll
    for (int s = 0; s < V; s += n) {
      if (s != at) continue;
#pragma unroll
      for (int j = 0; j < n; ++j) p[s + j] = from_f32<T>(v[s + j]);
    }
    at += n;
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
__device__ __forceinline__ float add_row16(float v) {  // of a pair of rows
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_row32(float v) {  // of the wave's halves
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
__device__ __forceinline__ float wave_sum(float v) { return add_row32(add_row16(row16_sum(v))); }
// The same over groups of 16, 32 or 64 lanes (`lanes`, uniform): groups that
// have left the loop around it are not read.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int lanes) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = row16_sum(v[i]);
    if (lanes > 16) v[i] = add_row16(v[i]);
    if (lanes > 32) v[i] = add_row32(v[i]);
  }
}
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Waits for this wave's loads, and its stores: one counter counts both.  Before
// a row's successor is loaded in a loop: where the loads that follow may be
// skipped, the compiler can wait for a value only by waiting for every load,
// the successor's too, so the present row's values have to be there first.
// Gradient of the norm, every tensor separate: rows that end inside a chunk
// 65536 x 2051 325 us, 399 without, 65536 x 1025 192 / 239; rows of whole chunks
// gain nothing by it (32768 x 4096 with a gate per token 365 / 365) and lose
// what the stores take to leave (8192 x 7168 126 / 125, FP32 32768 x 7168 776 /
// 760), so they do not wait.
__device__ __forceinline__ void wait_vmem() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

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
