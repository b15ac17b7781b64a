// Global gradient norm over many tensors, and clipping by it (gfx950).
//
//   N = (sum over all elements g^2)^(1/2),   out = g min(1, max_norm / (N + eps)).
//
// Two passes over the gradients, both bound by HBM: no element can be scaled
// before the last one is read.  All tensors are cut into chunks of kChunk
// elements; a workgroup takes a contiguous run of chunks, finds the first
// one's tensor in the table once and walks on from there, one loop per tensor.
// A lane loads 16 contiguous bytes at a time (FP32 in pairs of 16 bytes, 32
// apart from lane to lane, made the combine 10 % slower).  Squares are summed
// in FP64 (one conversion and one FMA per element, hidden behind the loads):
// an FP32 sum of squares would overflow from gradients of 2^64 on and lose
// those below 2^-63.  The partial sums are added in a fixed order, by every
// workgroup of the second pass for itself, which saves a launch between.
// 3.76 GB of FP32 gradients: 535 us for the squares (7.0 TB/s read) and 1467 for
// the scaling (5.1 TB/s read and written); 200 small tensors of 1.2 M elements
// in all: 4.9 and 6.7 us, launch, search of the table and partial sums.  Rows that
// do not follow each other are taken element by element, one load in flight and a
// 64-bit division each, which bound them: 131072 rows of 7165 FP32 values at a
// pitch of 7168, squares 2.1 ms where dense values take 0.54.
#include "../../include/libfp8blk_layer.h"
#include "host_common.h"
#include "layer_device.h"

namespace fp8blk {

constexpr int64_t kChunk = 1024;
constexpr int kGradBlocks = 1024;  // most workgroups, one partial sum each (2048: 1 % slower over 3.8 GB)
static_assert(kGradBlocks * sizeof(double) <= FP8BLK_GRAD_WORKSPACE_BYTES, "partial sums fit the workspace");

// One entry of the table; its chunks are [chunk0, the next entry's chunk0).
struct GradEntry {
  const void* src;
  void* dst;
  int64_t n, cols, ld, ldo;  // n = rows * cols elements
  int64_t chunk0;
  uint32_t flags;
  uint32_t pitched;
};
static_assert(sizeof(GradEntry) == 64, "table entry");

// The tensor that owns chunk c, found by the wave: 64 candidates at a time.
// Every entry has at least one chunk, so chunk0 ascends strictly.
__device__ __forceinline__ int64_t find_entry(const GradEntry* __restrict__ tab, int64_t n, int64_t c) {
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

// Calls body(v, k) for groups of V contiguous elements of [lo, hi), v from
// element k on in FP32: kUnroll groups per lane in flight while whole ones are
// left, then one by one; tail(x, k) gets the last elements of the range that
// fill no group.  Eight in flight gain 0.5 % over 3.8 GB but cost 20 % over 200
// small tensors.
constexpr int kUnroll = 4;
template <int V, bool NT, typename TS, typename B, typename E>
__device__ __forceinline__ void each_group(const Global<const TS>* src, int64_t lo, int64_t hi, B body, E tail) {
  int64_t i = lo;
  for (; i + 256 * V * kUnroll <= hi; i += 256 * V * kUnroll) {
    RawV<TS, V> raw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) raw[u] = load_raw<V, NT>(src + i + (u * 256 + (int)threadIdx.x) * V);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float v[V];
      unpack_v<TS, V>(raw[u], v);
      body(v, i + (u * 256 + (int)threadIdx.x) * V);
    }
  }
  for (i += threadIdx.x * V; i + V <= hi; i += 256 * V) {
    float v[V];
    unpack_v<TS, V>(load_raw<V, NT>(src + i), v);
    body(v, i);
  }
  if (i < hi)
    for (int64_t k = i; k < hi; ++k) tail(to_f32(src[k]), k);
}

// The workgroup's elements [lo, hi) of one gradient: adds their squares.
template <typename TS, bool NT>
__device__ __forceinline__ void add_squares(const GradEntry& e, int64_t lo, int64_t hi, double& sum) {
  constexpr int V = 16 / sizeof(TS);
  const Global<const TS>* src = global(reinterpret_cast<const TS*>(e.src));  // not known of a pointer read from memory
  auto one = [&](float x, int64_t) { sum = __builtin_fma((double)x, (double)x, sum); };
  if (e.pitched) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += 256) one(to_f32(src[at(i, e.cols, e.ld)]), i);
    return;
  }
  each_group<V, NT, TS>(src, lo, hi, [&](const float (&v)[V], int64_t k) {
#pragma unroll
    for (int j = 0; j < V; ++j) one(v[j], k);
  }, one);
}

// ... and scales them into the output.
template <typename TS, typename TD, bool NT>
__device__ __forceinline__ void scale_range(const GradEntry& e, int64_t lo, int64_t hi, float c) {
  constexpr int V = sizeof(TS) == 2 && sizeof(TD) == 2 ? 8 : 4;
  const Global<const TS>* src = global(reinterpret_cast<const TS*>(e.src));  // not known of a pointer read from memory
  Global<TD>* dst = global(reinterpret_cast<TD*>(e.dst));
  if (e.pitched) {
    for (int64_t i = lo + threadIdx.x; i < hi; i += 256)
      dst[at(i, e.cols, e.ldo)] = from_f32<TD>(to_f32(src[at(i, e.cols, e.ld)]) * c);
    return;
  }
  each_group<V, NT, TS>(src, lo, hi, [&](const float (&v)[V], int64_t k) {
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = v[j] * c;
    store_v<V, NT>(dst + k, o);
  }, [&](float x, int64_t k) { dst[k] = from_f32<TD>(x * c); });
}

// The gradients of a workgroup's chunks [c, c1), one range of elements each.
struct Walk {
  const GradEntry* tab;
  int64_t n, t, c, c1;
  GradEntry e;
  int64_t lo, hi;
  __device__ __forceinline__ Walk(const GradEntry* tab_, int64_t n_, int64_t chunks)
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

template <bool NT>
__global__ __launch_bounds__(256) void k_grad_squares(const GradEntry* __restrict__ tab, int64_t n, int64_t chunks,
                                                       double* __restrict__ partial) {
  __shared__ double red[4];
  double sum = 0.0;
  Walk w(tab, n, chunks);
  while (w.step()) {
    if (w.e.flags & FP8BLK_GRAD_F32) add_squares<float, NT>(w.e, w.lo, w.hi, sum);
    else add_squares<uint16_t, NT>(w.e, w.lo, w.hi, sum);
  }
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) partial[blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// The norm from the partial sums, the same bits in every workgroup of 256.
__device__ __forceinline__ float norm_of(const double* __restrict__ partial, int np, double* red) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < np; i += 256) sum += partial[i];
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  return (float)sqrt(red[0] + red[1] + red[2] + red[3]);
}

__global__ __launch_bounds__(256) void k_grad_norm(const double* __restrict__ partial, int np,
                                                    float* __restrict__ norm) {
  __shared__ double red[4];
  const float v = norm_of(partial, np, red);
  if (threadIdx.x == 0) *norm = v;
}

// given != NULL: the norm to clip by; otherwise it comes from the partial
// sums and workgroup 0 writes it to *norm.
template <bool NT>
__global__ __launch_bounds__(256) void k_grad_scale(const GradEntry* __restrict__ tab, int64_t n, int64_t chunks,
                                                     const float* given, const double* __restrict__ partial, int np,
                                                     float max_norm, float eps, float* norm) {
  __shared__ double red[4];
  Walk w(tab, n, chunks);  // the search of the table overlaps the partial sums' way from memory
  float total;
  if (given != nullptr) {
    total = *given;
  } else {
    total = norm_of(partial, np, red);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  }
  float coef = max_norm / (total + eps);
  coef = coef >= 1.0f ? 1.0f : coef;  // a NaN stays
  while (w.step()) {
    if (coef == 1.0f && w.e.dst == w.e.src) continue;
    if (w.e.flags & FP8BLK_GRAD_F32) {
      if (w.e.flags & FP8BLK_GRAD_OUT_F32) scale_range<float, float, NT>(w.e, w.lo, w.hi, coef);
      else scale_range<float, uint16_t, NT>(w.e, w.lo, w.hi, coef);
    } else {
      if (w.e.flags & FP8BLK_GRAD_OUT_F32) scale_range<uint16_t, float, NT>(w.e, w.lo, w.hi, coef);
      else scale_range<uint16_t, uint16_t, NT>(w.e, w.lo, w.hi, coef);
    }
  }
}

inline unsigned grad_blocks(int64_t chunks) { return (unsigned)(chunks < kGradBlocks ? chunks : kGradBlocks); }

// Streamed loads and stores (see kStreamBytes) from 2^24 elements on, already
// below the Infinity Cache's size: both passes over FP32 gradients into other
// FP32 tensors took 37 us streamed and 41 cached at 64 MiB, 70 / 80 at 128,
// 142 / 160 at 256, 544 / 594 at 1024, but 17 / 15 at 16 MiB.
inline bool grad_stream(int64_t chunks) { return chunks >= ((int64_t)1 << 24) / kChunk; }

inline bool table_ok(const void* table, int64_t n, int64_t chunks) {
  if (n < 0 || chunks < n) return false;
  return n == 0 ? chunks == 0 : table != nullptr && aligned(table, 8);
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" size_t fp8blk_grad_table_bytes(int64_t n) { return n > 0 ? (size_t)n * sizeof(GradEntry) : 0; }

extern "C" fp8blk_status_t fp8blk_grad_table_build(const fp8blk_grad_t* list, int64_t n, void* table,
                                                   size_t table_bytes, int64_t* chunks) {
  if (n < 0 || chunks == nullptr) return FP8BLK_ERR_INVALID_ARG;
  if (n > 0 && (list == nullptr || table == nullptr || !aligned(table, 8) || table_bytes < fp8blk_grad_table_bytes(n)))
    return FP8BLK_ERR_INVALID_ARG;
  int64_t next = 0;
  for (int64_t i = 0; i < n; ++i) {
    const fp8blk_grad_t& g = list[i];
    const uintptr_t se = g.flags & FP8BLK_GRAD_F32 ? 4 : 2, de = g.flags & FP8BLK_GRAD_OUT_F32 ? 4 : 2;
    if ((g.flags & ~(FP8BLK_GRAD_F32 | FP8BLK_GRAD_OUT_F32)) || g.reserved != 0) return FP8BLK_ERR_INVALID_ARG;
    if (g.rows <= 0 || g.cols <= 0 || g.ld < g.cols || g.ldo < g.cols || g.rows > INT64_MAX / 16 / g.ld ||
        g.rows > INT64_MAX / 16 / g.ldo)
      return FP8BLK_ERR_INVALID_ARG;  // empty gradients have no place in the table
    if (g.grad == nullptr || g.out == nullptr || !aligned(g.grad, se) || !aligned(g.out, de))
      return FP8BLK_ERR_INVALID_ARG;
    if (g.grad == g.out && (se != de || g.ld != g.ldo)) return FP8BLK_ERR_INVALID_ARG;
    GradEntry e{};
    e.src = g.grad;
    e.dst = g.out;
    e.n = g.rows * g.cols;
    e.cols = g.cols;
    e.ld = g.ld;
    e.ldo = g.ldo;
    e.chunk0 = next;
    e.flags = g.flags;
    e.pitched = g.rows > 1 && (g.ld != g.cols || g.ldo != g.cols);
    next += ceil_div(e.n, kChunk);
    reinterpret_cast<GradEntry*>(table)[i] = e;
  }
  *chunks = next;
  return FP8BLK_OK;
}

extern "C" fp8blk_status_t fp8blk_grad_norm(const void* table, int64_t n, int64_t chunks, float* norm, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  if (!table_ok(table, n, chunks) || norm == nullptr || !aligned(norm, 4)) return FP8BLK_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 8) || workspace_bytes < FP8BLK_GRAD_WORKSPACE_BYTES)
    return FP8BLK_ERR_INVALID_ARG;
  const unsigned nb = grad_blocks(chunks);
  double* partial = reinterpret_cast<double*>(workspace);
  if (nb > 0)
    hipLaunchKernelGGL((grad_stream(chunks) ? k_grad_squares<true> : k_grad_squares<false>), dim3(nb), dim3(256), 0, as_stream(stream),
                       reinterpret_cast<const GradEntry*>(table), n, chunks, partial);
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(256), 0, as_stream(stream), partial, (int)nb, norm);
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_grad_clip(const void* table, int64_t n, int64_t chunks, const float* norm,
                                            float max_norm, float eps, void* stream) {
  if (!table_ok(table, n, chunks) || norm == nullptr || !aligned(norm, 4) || !(max_norm >= 0.0f) || !(eps >= 0.0f))
    return FP8BLK_ERR_INVALID_ARG;
  if (n == 0) return FP8BLK_OK;
  hipLaunchKernelGGL((grad_stream(chunks) ? k_grad_scale<true> : k_grad_scale<false>), dim3(grad_blocks(chunks)), dim3(256), 0, as_stream(stream),
                     reinterpret_cast<const GradEntry*>(table), n, chunks, norm, nullptr, 0, max_norm, eps, nullptr);
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_grad_clip_norm(const void* table, int64_t n, int64_t chunks, float max_norm,
                                                 float eps, float* norm, void* workspace, size_t workspace_bytes,
                                                 void* stream) {
  if (!table_ok(table, n, chunks) || norm == nullptr || !aligned(norm, 4) || !(max_norm >= 0.0f) || !(eps >= 0.0f))
    return FP8BLK_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 8) || workspace_bytes < FP8BLK_GRAD_WORKSPACE_BYTES)
    return FP8BLK_ERR_INVALID_ARG;
  if (n == 0) return fp8blk_grad_norm(table, n, chunks, norm, workspace, workspace_bytes, stream);
  const unsigned nb = grad_blocks(chunks);
  double* partial = reinterpret_cast<double*>(workspace);
  hipLaunchKernelGGL((grad_stream(chunks) ? k_grad_squares<true> : k_grad_squares<false>), dim3(nb), dim3(256), 0, as_stream(stream),
                     reinterpret_cast<const GradEntry*>(table), n, chunks, partial);
  const fp8blk_status_t st = launch_status();
  if (st != FP8BLK_OK) return st;
  hipLaunchKernelGGL((grad_stream(chunks) ? k_grad_scale<true> : k_grad_scale<false>), dim3(nb), dim3(256), 0, as_stream(stream),
                     reinterpret_cast<const GradEntry*>(table), n, chunks, nullptr, partial, (int)nb, max_norm, eps,
                     norm);
  return launch_status();
}
