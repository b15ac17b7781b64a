// Tables of many tensors, cut into chunks of kChunk elements, and the walk of a
// workgroup over a contiguous run of them (gradient clipping, optimizer step).
// A table entry has n elements in rows of cols and its first chunk chunk0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8blk {

constexpr int64_t kChunk = 1024;

// The tensor that owns chunk c, found by the wave: 64 candidates at a time.
// Every entry has at least one chunk, so chunk0 ascends strictly.
template <class Entry>
__device__ __forceinline__ int64_t find_entry(const Entry* __restrict__ tab, int64_t n, int64_t c) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, len = n;  // the owner is in [lo, lo + len), tab[lo].chunk0 <= c
  while (len > 1) {
    const int64_t step = (len + 63) / 64;
    const int64_t i = lo + lane * step;
    const uint64_t le = __ballot(lane * step < len && tab[i].chunk0 <= c);
    const int64_t last = 63 - __builtin_clzll(le);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

// Element offset of a flat index: rows lie ld elements apart.
__device__ __forceinline__ int64_t at(int64_t i, int64_t cols, int64_t ld) { return i / cols * ld + i % cols; }

// The tensors of a workgroup's chunks [c, c1), one range of elements each.
template <class Entry>
struct Walk {
  const Entry* tab;
  int64_t n, t, c, c1;
  Entry e;
  int64_t lo, hi;
  __device__ __forceinline__ Walk(const Entry* tab_, int64_t n_, int64_t chunks)
      : tab(tab_), n(n_), t(0), c(chunks * blockIdx.x / gridDim.x), c1(chunks * (blockIdx.x + 1) / gridDim.x) {
    if (c < c1) t = find_entry(tab, n, c);
  }
  __device__ __forceinline__ bool step() {
    if (c >= c1) return false;
    e = tab[t];
    const int64_t end = t + 1 < n ? min(tab[t + 1].chunk0, c1) : c1;
    lo = (c - e.chunk0) * kChunk;
    hi = min((end - e.chunk0) * kChunk, e.n);
    c = end;
    ++t;
    return true;
  }
};

}  // namespace fp8blk
