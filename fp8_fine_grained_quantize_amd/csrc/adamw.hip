// One AdamW step over many tensors (gfx950).
//
//   g = grad c,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
// c the clipping factor of a norm in device memory, so that clipping costs no
// pass of its own.  The pages keep the moments in low precision [p2¶4]: FP32,
// BF16, or E4M3 codes of m and sqrt(v) with a scale for 128 values (the root
// halves the exponents that the codes have to span).
// Citations [pN¶k]: N-th page of the source collection, k-th paragraph
// (p2 = inprokorea.com wr_id 735329).
//
// Bound by HBM: 28 bytes a value in FP32, 16.125 with E4M3 moments, against some
// 40 operations.  A workgroup takes a contiguous run of chunks (tensor_table.h);
// a lane holds four consecutive values, so that FP32 is one 16-byte access, and
// 32 lanes a group of 128, whose maximum is found by lane exchanges.
// Measured, with BF16 copies: 0.94e9 values in FP32 4.76 ms (5.9 TB/s), with E4M3
// moments rounded at random 3.12 ms (5.5 TB/s); 60e6 values in BF16 throughout,
// without copies, 172 us (4.9 TB/s counting 14 bytes a value); 1.2e6 values in 200
// tensors 9 us, three dependent reads of the table and one of the data.  With E4M3
// moments the vector instructions, 96 a value, take three quarters of the time (121
// of them all of it): a root by root_of, a scale's reciprocal by one Newton step, magnitudes
// without signs, and addresses in scalar registers took 0.27e9 values without
// copies from 829 to 752 us (BF16 parameters, to nearest: 700 to 615).
//
// Every operation is rounded by itself, none fused, in the order in which a
// program of elementary FP32 operations takes them: a value that differs in its
// last bit can fall to another E4M3 code, 6 to 12 % away, so that only equal
// operations give equal codes.
#include <algorithm>
#include <cmath>

#include "../../include/libfp8blk_train.h"
#include "host_common.h"
#include "layer_device.h"
#include "tensor_table.h"

namespace fp8blk {

struct AdamEntry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  int64_t n, cols, ldp, ldg, ldc;
  int64_t chunk0;
  float decay;
  uint32_t flags;
  uint32_t index;
  uint32_t pitched;
};
static_assert(sizeof(AdamEntry) == 120, "table entry");

struct AdamArgs {
  double beta1, beta2;
  double lr;
  int64_t step;
  const float* lr_at;
  const int64_t* step_at;
  const int64_t* seed_at;
  const float* norm;
  float b1, nb1, b2, nb2, eps;  // nb = 1 - b
  float max_norm, clip_eps;
  float step_size, root;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t seed;
};

// The 32-bit finalizer of MurmurHash3 (A. Appleby, public domain) over an
// element's place, its low and its high half, and a key.
__device__ __forceinline__ uint32_t random_bits(uint32_t key, uint32_t place, uint32_t high) {
  uint32_t h = (place * 0x9E3779B1u ^ high) + key;
  h = (h ^ h >> 16) * 0x85EBCA6Bu;
  h = (h ^ h >> 13) * 0xC2B2AE35u;
  return h ^ h >> 16;
}

// BF16 by adding 16 random bits below the kept ones and dropping those (a NaN stays one).
__device__ __forceinline__ float to_bf16_random(float x, uint32_t r16) {
  return x == x ? __uint_as_float((__float_as_uint(x) + r16) & 0xFFFF0000u) : x;
}

// sqrt(x), correctly rounded, of what is zero or at least 2^-100 (NaN and
// infinity stay): Tuckerman's test.  s, the hardware's root, is off by one unit at
// most, and of s and its neighbours the root lies nearest to s unless s (s - ulp)
// >= x or s (s + ulp) < x.  Neither holds for zero.
__device__ __forceinline__ float root_of(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);
  const float down = __uint_as_float(__float_as_uint(s) - 1), up = __uint_as_float(__float_as_uint(s) + 1);
  const float r = __builtin_fmaf(-down, s, x) <= 0.0f ? down : s;
  return __builtin_fmaf(-up, s, x) > 0.0f ? up : r;
}

// The scale of a group with that maximum, and its reciprocal for the quotients
// (by one Newton step, within one unit in the last place; see fp8_device.h).
__device__ __forceinline__ TileScale moment_scale(uint32_t amax_bits) {
  TileScale t{1.0f, 1.0f, false};
  if (amax_bits == 0) return t;
  t.s = __uint_as_float(amax_bits) * (1.0f / kE4M3Max);
  const float r = __builtin_amdgcn_rcpf(t.s);
  t.r = __builtin_fmaf(__builtin_fmaf(-t.s, r, 1.0f), r, r);
  t.slow = !(t.s >= 0x1p-100f && t.s <= 0x1p100f);
  return t;
}

// Codes of four values of a group of 128 that 32 lanes hold.  ROOT: the values
// are not negative and none above zero becomes zero.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], bool random, const uint32_t (&r16)[4], float& scale) {
  constexpr uint32_t magnitude = ROOT ? 0xFFFFFFFFu : 0x7FFFFFFFu;
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) a = max(a, __float_as_uint(x[j]) & magnitude);
  a = row16_max(a);
  const auto o = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  const TileScale ts = moment_scale(max(o[0], o[1]));
  scale = ts.s;
  float y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // quotient_fast, without its sign
    const float q = x[j] * ts.r;
    y[j] = __builtin_fmaf(__builtin_fmaf(-ts.s, q, x[j]), ts.r, q);
  }
  if (__builtin_expect(ts.slow, 0)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = quotient_slow(x[j], ts.s);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // 2^-9, the smallest code, stays what it is below.
    float v = __builtin_amdgcn_fmed3f(__builtin_fabsf(y[j]), ROOT && x[j] > 0.0f ? 0x1p-9f : 0.0f, kE4M3Max);
    if (random) {  // below 2^-6 the codes lie 2^-9 apart, as they do from there to 2^-5
      const float up = v < 0x1p-6f ? 0x1p-6f : 0.0f;
      v = __uint_as_float((__float_as_uint(v + up) + (r16[j] << 4)) & 0xFFF00000u) - up;
    }
    y[j] = ROOT ? v : __builtin_copysignf(v, x[j]);
  }
  return pack4_e4m3(y[0], y[1], y[2], y[3]);
}

__device__ __forceinline__ void decode4(uint32_t c, float s, float (&x)[4]) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
  x[0] = lo[0] * s;
  x[1] = lo[1] * s;
  x[2] = hi[0] * s;
  x[3] = hi[1] * s;
}

// How a lane's four values lie in memory: one after another; in a row of a
// tensor whose rows lie apart; or in two rows of one.
enum Lie { DENSE, ROW, ROWS };

// A lane's place: element `base` of its tensor, the same for the whole
// workgroup and a multiple of kChunk, and `mine` from there on: an address in
// scalar registers and an offset of 32 bits in vector ones.
struct Place {
  int64_t base;
  uint32_t mine;
  int count;  // of the lane's four elements, those that exist
  Lie lie;
  int64_t row, col;  // of the first of them, unless DENSE
  __device__ __forceinline__ int64_t index() const { return base + mine; }
  // Element j's offset, in rows of cols, ld apart.
  __device__ __forceinline__ int64_t at(int j, int64_t cols, int64_t ld) const {
    if (lie == DENSE) return index() + j;
    int64_t r = row, c = col + j;
    while (c >= cols) c -= cols, ++r;  // at most three times
    return r * ld + c;
  }
};

// The elements at a place of a tensor in rows of cols, ld apart (4 at once: one
// access unless they lie in two rows); those that do not exist zero.
template <bool NT, typename T>
__device__ __forceinline__ RawV<T, 4> load4(const T* t, const Place& w, int64_t cols, int64_t ld) {
  if (w.count == 4 && w.lie == DENSE) return load_raw<4, NT>(global(t + w.base) + w.mine);
  if (w.count == 4 && w.lie == ROW) return load_raw<4, NT>(global(t + w.at(0, cols, ld)));
  RawV<T, 4> r{};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= w.count) continue;
    const T x = global(t)[w.at(j, cols, ld)];
    if constexpr (sizeof(T) == 4) r[j] = __float_as_uint(x);
    else r[j >> 1] |= (uint32_t)x << ((j & 1) * 16);
  }
  return r;
}
template <bool NT, typename T>
__device__ __forceinline__ void store4(T* t, const float (&v)[4], const Place& w, int64_t cols, int64_t ld) {
  if (w.count == 4 && w.lie == DENSE) return store_v<4, NT>(global(t + w.base) + w.mine, v);
  if (w.count == 4 && w.lie == ROW) return store_v<4, NT>(global(t + w.at(0, cols, ld)), v);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < w.count) global(t)[w.at(j, cols, ld)] = from_f32<T>(v[j]);
}

// The moments' type as stored, and what a lane loads of them.
template <int ST>
struct Moment {
  typedef uint16_t type;
  typedef RawV<uint16_t, 4> raw;
};
template <>
struct Moment<FP8BLK_ADAMW_F32> {
  typedef float type;
  typedef RawV<float, 4> raw;
};
template <>
struct Moment<FP8BLK_ADAMW_E4M3> {
  typedef uint8_t type;
  typedef uint32_t raw;
};

template <typename TP, typename TG, int ST>
struct Quad {  // what a lane loads of its four values
  RawV<TP, 4> p;
  RawV<TG, 4> g;
  typename Moment<ST>::raw m, v;
  float ms, vs;
};

template <typename TP, typename TG, int ST, bool NT>
struct AdamRange {
  typedef typename Moment<ST>::type TM;
  const AdamEntry& e;
  const AdamArgs& a;
  float clip, keep, step_size, root;  // keep: 1 - lr decay
  uint32_t key;
  bool random;

  __device__ __forceinline__ Quad<TP, TG, ST> load(const Place& w) const {
    // FP32 moments of large tables: a wave reads one tensor after another.  Four
    // reads and four writes at the same place of as many tensors, from every
    // wave at once, is what memory does worst: 0.94e9 values 4.83 ms at once, 4.54
    // in turn.  With E4M3 moments the waits cost more than that: 3.12 / 3.50, and
    // with BF16 ones they win as often as they lose (60e6 values 172 / 187 us).
    constexpr bool TURNS = NT && ST == FP8BLK_ADAMW_F32;
    Quad<TP, TG, ST> q{};
    q.p = load4<NT>((const TP*)e.p, w, e.cols, e.ldp);
    if (TURNS) wait_vmem();
    q.g = load4<NT>((const TG*)e.g, w, e.cols, e.ldg);
    if (TURNS) wait_vmem();
    if constexpr (ST == FP8BLK_ADAMW_E4M3) {
      const Global<const uint8_t>*m = global((const uint8_t*)e.m + w.base) + w.mine,
                   *v = global((const uint8_t*)e.v + w.base) + w.mine;
      if (w.count == 4) {
        q.m = *(const Global<const uint32_t>*)m;
        q.v = *(const Global<const uint32_t>*)v;
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          if (j >= w.count) continue;
          q.m |= (uint32_t)m[j] << (8 * j);
          q.v |= (uint32_t)v[j] << (8 * j);
        }
      }
      if (w.count > 0) {
        q.ms = global(e.ms + (w.base >> 7))[w.mine >> 7];
        q.vs = global(e.vs + (w.base >> 7))[w.mine >> 7];
      }
    } else {
      q.m = load4<NT>((const TM*)e.m, dense(w), 0, 0);
      if (TURNS) wait_vmem();
      q.v = load4<NT>((const TM*)e.v, dense(w), 0, 0);
    }
    return q;
  }

  // Every lane of the wave takes part (count may be 0): E4M3 scales are found across lanes.
  __device__ __forceinline__ void finish(const Quad<TP, TG, ST>& q, const Place& w) const {
    float p[4], g[4], m[4], v[4], r[4];
    unpack_v<TP, 4>(q.p, p);
    unpack_v<TG, 4>(q.g, g);
    if constexpr (ST == FP8BLK_ADAMW_E4M3) {
      decode4(q.m, q.ms, m);
      decode4(q.v, q.vs, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= v[j];
    } else {
      unpack_v<TM, 4>(q.m, m);
      unpack_v<TM, 4>(q.v, v);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] *= clip;
      m[j] = a.b1 * m[j] + a.nb1 * g[j];
      v[j] = a.b2 * v[j] + a.nb2 * g[j] * g[j];
      r[j] = ST != FP8BLK_ADAMW_BF16 ? root_of(v[j]) : sqrtf(v[j]);  // BF16: sqrtf with the loop below is 4 % faster
    }
    uint32_t least = 0xFFFFFFFFu;  // zeros become the largest
#pragma unroll
    for (int j = 0; j < 4; ++j) least = min(least, __float_as_uint(v[j]) - 1);
    if (ST != FP8BLK_ADAMW_BF16 && __builtin_expect(least < 0x0D800000u, 0)) {  // 2^-100
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = sqrtf(v[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = p[j] * keep - step_size * m[j] / (r[j] * root + a.eps);
    const uint32_t place = (uint32_t)w.base + w.mine, high = (uint32_t)((uint64_t)w.base >> 32);
    uint32_t rm[4] = {}, rv[4] = {};
    if (ST != FP8BLK_ADAMW_F32 && random) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t h = random_bits(key, place + j, high);
        rm[j] = h & 0xFFFFu;
        rv[j] = h >> 16;
      }
    }
    if constexpr (ST == FP8BLK_ADAMW_E4M3) {
      float ms, vs;
      const uint32_t mc = encode4<false>(m, random, rm, ms), vc = encode4<true>(r, random, rv, vs);
      Global<uint8_t>*md = global((uint8_t*)e.m + w.base) + w.mine, *vd = global((uint8_t*)e.v + w.base) + w.mine;
      if (w.count == 4) {
        store_words<NT, 1>((Global<void>*)md, Words<1>::type{mc});
        store_words<NT, 1>((Global<void>*)vd, Words<1>::type{vc});
      } else {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          if (j >= w.count) continue;
          md[j] = (uint8_t)(mc >> (8 * j));
          vd[j] = (uint8_t)(vc >> (8 * j));
        }
      }
      if (w.count > 0 && (threadIdx.x & 31) == 0) {
        global(e.ms + (w.base >> 7))[w.mine >> 7] = ms;
        global(e.vs + (w.base >> 7))[w.mine >> 7] = vs;
      }
    } else {
      if (ST == FP8BLK_ADAMW_BF16 && random) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[j] = to_bf16_random(m[j], rm[j]);
          v[j] = to_bf16_random(v[j], rv[j]);
        }
      }
      store4<NT>((TM*)e.m, m, dense(w), 0, 0);
      store4<NT>((TM*)e.v, v, dense(w), 0, 0);
    }
    if (e.copy != nullptr) store4<NT>(e.copy, p, w, e.cols, e.ldc);
    if (sizeof(TP) == 2 && random) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = to_bf16_random(p[j], random_bits(key ^ 0x5BD1E995u, place + j, high) & 0xFFFFu);
    }
    store4<NT>((TP*)e.p, p, w, e.cols, e.ldp);
  }

  // The elements [lo, hi); lo is a multiple of kChunk, hi too unless the tensor
  // ends there.  A chunk's loads go out before the stores of the one before: one
  // counter counts both, so that loads behind stores would wait for them.
  __device__ __forceinline__ void run(int64_t lo, int64_t hi) const {
    const uint32_t mine = threadIdx.x * 4;
    int64_t base = lo;
    if (!e.pitched && base + kChunk <= hi) {
      Quad<TP, TG, ST> q = load({base, mine, 4, DENSE});
      auto two = [&]() {
        const Quad<TP, TG, ST> next = load({base + kChunk, mine, 4, DENSE});
        finish(q, {base, mine, 4, DENSE});
        q = next;
        base += kChunk;
      };
      if constexpr (ST == FP8BLK_ADAMW_BF16) {
        while (base + 2 * kChunk <= hi) two();
      } else {  // by twos, without moving `next` to `q`: E4M3 5 % of its instructions (BF16: 4 % slower)
        for (; base + 3 * kChunk <= hi; base += 2 * kChunk) {
          const Quad<TP, TG, ST> next = load({base + kChunk, mine, 4, DENSE});
          finish(q, {base, mine, 4, DENSE});
          q = load({base + 2 * kChunk, mine, 4, DENSE});
          finish(next, {base + kChunk, mine, 4, DENSE});
        }
        if (base + 2 * kChunk <= hi) two();
      }
      finish(q, {base, mine, 4, DENSE});
      base += kChunk;
    }
    const Lie lie = !e.pitched ? DENSE : (e.cols & 3) == 0 ? ROW : ROWS;
    for (; base < hi; base += kChunk) {
      const int left = (int)max((int64_t)0, min((int64_t)4, hi - base - mine));
      Place w{base, mine, left, lie};
      if (lie != DENSE) {  // one division for every tensor and value
        w.row = w.index() / e.cols;
        w.col = w.index() - w.row * e.cols;
      }
      finish(load(w), w);
    }
  }
  static __device__ __forceinline__ Place dense(const Place& w) { return {w.base, w.mine, w.count, DENSE}; }
};

// With lr or step in device memory every lane takes the powers of beta (FP64)
// before its first load, where few chunks a workgroup follow.  Values from the
// host / from the device: 0.94e9 values in FP32 4.90 / 4.79 ms, with E4M3 moments
// rounded at random 3.14 / 3.18 ms; 0.27e9 BF16 parameters with E4M3 moments 589 /
// 690 us; 60e6 values in BF16 throughout 152 to 174 / 181 us (a replayed graph as
// the device form).
template <int ST, bool NT>
__global__ __launch_bounds__(256) void k_adamw(const AdamEntry* __restrict__ tab, int64_t n, int64_t chunks,
                                                AdamArgs a, bool random) {
  Walk<AdamEntry> w(tab, n, chunks);
  double lr = a.lr;
  float step_size = a.step_size, root = a.root, clip = 1.0f;
  if (a.lr_at != nullptr) lr = *a.lr_at;
  if (a.step_at != nullptr) {
    const double t = (double)*a.step_at;
    root = 1.0f / (float)sqrt(1.0 - pow(a.beta2, t));
    step_size = (float)(lr / (1.0 - pow(a.beta1, t)));
  } else if (a.lr_at != nullptr) {
    step_size = (float)(lr / (1.0 - pow(a.beta1, (double)a.step)));
  }
  const uint32_t seed = a.seed_at != nullptr ? (uint32_t)*a.seed_at : a.seed;
  if (a.norm != nullptr) {
    clip = a.max_norm * (1.0f / (*a.norm + a.clip_eps));
    clip = clip >= 1.0f ? 1.0f : clip;  // a NaN stays
  }
  while (w.step()) {
    const float keep = (float)(1.0 - lr * w.e.decay);
    const uint32_t key = seed + w.e.index * 0x27D4EB2Fu;
    auto run = [&](auto tp, auto tg) {
      AdamRange<decltype(tp), decltype(tg), ST, NT>{w.e, a, clip, keep, step_size, root, key, random}.run(w.lo, w.hi);
    };
    if (w.e.flags & FP8BLK_ADAMW_PARAM_F32) {
      if (w.e.flags & FP8BLK_ADAMW_GRAD_F32) run(float(), float());
      else run(float(), uint16_t());
    } else {
      if (w.e.flags & FP8BLK_ADAMW_GRAD_F32) run(uint16_t(), float());
      else run(uint16_t(), uint16_t());
    }
  }
}

// Streamed loads and stores (see kStreamBytes in layer_host.h) from 2^25 elements
// on: with FP32 throughout 16e6 elements took 72 us streamed and 66 not, 0.94e9
// 4.9 and 5.2 ms; with BF16 throughout 60e6 149 and 158 us.
inline bool adam_stream(int64_t chunks) { return chunks >= ((int64_t)1 << 25) / kChunk; }

// Chunks of a workgroup.  Short runs keep the waves' places in memory close
// together, longer ones cover the search of the table: 0.94e9 values with FP32
// moments 4.76 / 4.67 / 4.90 / 4.95 ms with 1 / 2 / 3 / 4 chunks each (persistent
// workgroups 5.4 and more); with E4M3 moments 3.14 / 3.07 / 3.10 with 2 / 4 / 8, and
// 60e6 values in BF16 190 / 174 / 190 us.
inline int64_t adam_run(int state, int64_t chunks) {
  return std::clamp<int64_t>(chunks / 4096, 1, state == FP8BLK_ADAMW_F32 ? 2 : 4);
}
// LDS that a workgroup of a streamed table asks for and does not use, so that
// five of them share a compute unit (four with BF16 moments), not seven: the fewer
// places memory is worked on at once, the better.  FP32 moments 4.67 ms with five,
// 4.76 with six, 4.78 with four; BF16 throughout 174.4 us with four, 174.9 with
// five, 178 with seven; E4M3 3.07 / 3.09 / 3.15 ms with four / five / seven, but
// without copies and FP32 gradients 730 / 698 / 702 us (0.27e9 values).
inline unsigned adam_room(int state) { return state == FP8BLK_ADAMW_BF16 ? 40000 : 32000; }

inline bool state_ok(int state) {
  return state == FP8BLK_ADAMW_F32 || state == FP8BLK_ADAMW_BF16 || state == FP8BLK_ADAMW_E4M3;
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_train_abi_version(void) { return 1; }

extern "C" size_t fp8blk_adamw_table_bytes(int64_t n) { return n > 0 ? (size_t)n * sizeof(AdamEntry) : 0; }

extern "C" fp8blk_status_t fp8blk_adamw_table_build(const fp8blk_adamw_t* list, int64_t n, int state, void* table,
                                                    size_t table_bytes, int64_t* chunks) {
  if (n < 0 || chunks == nullptr || !state_ok(state)) return FP8BLK_ERR_INVALID_ARG;
  if (n > 0 && (list == nullptr || table == nullptr || !aligned(table, 8) || table_bytes < fp8blk_adamw_table_bytes(n)))
    return FP8BLK_ERR_INVALID_ARG;
  int64_t next = 0;
  for (int64_t i = 0; i < n; ++i) {
    const fp8blk_adamw_t& t = list[i];
    const uintptr_t pe = t.flags & FP8BLK_ADAMW_PARAM_F32 ? 4 : 2, ge = t.flags & FP8BLK_ADAMW_GRAD_F32 ? 4 : 2;
    const uintptr_t me = state == FP8BLK_ADAMW_BF16 ? 2 : 4;  // codes are read four at a time
    if ((t.flags & ~(FP8BLK_ADAMW_PARAM_F32 | FP8BLK_ADAMW_GRAD_F32)) || t.reserved != 0) return FP8BLK_ERR_INVALID_ARG;
    if (t.rows <= 0 || t.cols <= 0) return FP8BLK_ERR_INVALID_ARG;  // empty tensors have no place in the table
    for (const int64_t ld : {t.ldp, t.ldg, t.copy != nullptr ? t.ldc : t.cols})
      if (ld < t.cols || t.rows > INT64_MAX / 16 / ld) return FP8BLK_ERR_INVALID_ARG;
    if (t.param == nullptr || t.grad == nullptr || t.m == nullptr || t.v == nullptr) return FP8BLK_ERR_INVALID_ARG;
    if (!aligned(t.param, pe) || !aligned(t.grad, ge) || !aligned(t.m, me) || !aligned(t.v, me) || !aligned(t.copy, 2))
      return FP8BLK_ERR_INVALID_ARG;
    const bool scaled = state == FP8BLK_ADAMW_E4M3;
    if (scaled != (t.m_scale != nullptr) || scaled != (t.v_scale != nullptr) || !aligned(t.m_scale, 4) ||
        !aligned(t.v_scale, 4))
      return FP8BLK_ERR_INVALID_ARG;
    AdamEntry e{};
    e.p = t.param;
    e.g = t.grad;
    e.m = t.m;
    e.v = t.v;
    e.ms = t.m_scale;
    e.vs = t.v_scale;
    e.copy = t.copy;
    e.n = t.rows * t.cols;
    e.cols = t.cols;
    e.ldp = t.ldp;
    e.ldg = t.ldg;
    e.ldc = t.copy != nullptr ? t.ldc : t.cols;
    e.chunk0 = next;
    e.decay = t.decay;
    e.flags = t.flags;
    e.index = t.index;
    e.pitched = t.rows > 1 && (t.ldp != t.cols || t.ldg != t.cols || e.ldc != t.cols);
    next += ceil_div(e.n, kChunk);
    reinterpret_cast<AdamEntry*>(table)[i] = e;
  }
  *chunks = next;
  return FP8BLK_OK;
}

extern "C" fp8blk_status_t fp8blk_adamw_step(const void* table, int64_t n, int64_t chunks, int state,
                                             const fp8blk_adamw_step_t* s, void* stream) {
  if (n < 0 || chunks < n || !state_ok(state) || s == nullptr) return FP8BLK_ERR_INVALID_ARG;
  if (n == 0 ? chunks != 0 : table == nullptr || !aligned(table, 8)) return FP8BLK_ERR_INVALID_ARG;
  if (!(s->beta1 >= 0.0 && s->beta1 < 1.0) || !(s->beta2 >= 0.0 && s->beta2 < 1.0) || !(s->eps >= 0.0))
    return FP8BLK_ERR_INVALID_ARG;
  if ((s->lr_at == nullptr && !(s->lr - s->lr == 0.0)) || (s->step_at == nullptr && s->step < 1) ||
      (s->flags & ~FP8BLK_ADAMW_RANDOM))
    return FP8BLK_ERR_INVALID_ARG;
  if (!aligned(s->lr_at, 4) || !aligned(s->step_at, 8) || !aligned(s->seed_at, 8) || !aligned(s->norm, 4))
    return FP8BLK_ERR_INVALID_ARG;
  if (s->norm != nullptr && (!(s->max_norm >= 0.0f) || !(s->clip_eps >= 0.0f))) return FP8BLK_ERR_INVALID_ARG;
  if (n == 0) return FP8BLK_OK;
  AdamArgs a{};
  a.beta1 = s->beta1;
  a.beta2 = s->beta2;
  a.lr = s->lr;
  a.step = s->step;
  a.lr_at = s->lr_at;
  a.step_at = s->step_at;
  a.seed_at = s->seed_at;
  a.norm = s->norm;
  a.b1 = (float)s->beta1;
  a.nb1 = (float)(1.0 - s->beta1);
  a.b2 = (float)s->beta2;
  a.nb2 = (float)(1.0 - s->beta2);
  a.eps = (float)s->eps;
  a.max_norm = s->max_norm;
  a.clip_eps = s->clip_eps;
  if (s->step_at == nullptr) {
    a.step_size = (float)(s->lr / (1.0 - pow(s->beta1, (double)s->step)));
    a.root = 1.0f / (float)sqrt(1.0 - pow(s->beta2, (double)s->step));
  }
  a.seed = s->seed;
  // A launch counts its lanes in 32 bits.
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(chunks, adam_run(state, chunks)), 0xFFFFFF)), block(256);
  const AdamEntry* tab = reinterpret_cast<const AdamEntry*>(table);
  const bool random = s->flags & FP8BLK_ADAMW_RANDOM, nt = adam_stream(chunks);
  const unsigned room = nt ? adam_room(state) : 0;
#define FP8BLK_ADAMW_LAUNCH(ST_)                                                                                    \
  hipLaunchKernelGGL((nt ? k_adamw<ST_, true> : k_adamw<ST_, false>), grid, block, room, as_stream(stream), tab, n, chunks, \
                     a, random)
  if (state == FP8BLK_ADAMW_F32) FP8BLK_ADAMW_LAUNCH(FP8BLK_ADAMW_F32);
  else if (state == FP8BLK_ADAMW_BF16) FP8BLK_ADAMW_LAUNCH(FP8BLK_ADAMW_BF16);
  else FP8BLK_ADAMW_LAUNCH(FP8BLK_ADAMW_E4M3);
#undef FP8BLK_ADAMW_LAUNCH
  return launch_status();
}
