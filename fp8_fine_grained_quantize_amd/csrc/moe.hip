// Tokens into expert order and back, and the gradients (gfx950).
//
// The grouped GEMMs take rows ordered by expert with device-resident offsets;
// each token goes to K experts [p5¶3] and MoE activations are quantized before
// they are dispatched [p2¶4].  Citations [pN¶k]: N-th page of the source
// collection, k-th paragraph (p2 = inprokorea.com wr_id 735329, p5 =
// inprokorea.com wr_id 890463).
//
// With the rows of a permutation r(t, k) of the pairs:
//   dispatch  out[r(t, k)] = x[t]
//   combine   y[t] = sum_k w(t, k) rows[r(t, k)]
// and, as the two are each other's transpose, the gradient of dispatch is the
// combine with w = 1, that of the combine the dispatch of w dy, and
// dw(t, k) = <dy[t], rows[r(t, k)]>.  All of them move memory and compute next
// to nothing: HBM bounds them.
#include "../../include/libfp8blk_layer.h"
#include "host_common.h"
#include "layer_device.h"
#include "layer_host.h"

namespace fp8blk {

// ---------------------------------------------------------------------------
// Sort by expert: a stable counting sort.  The rank of a pair is
//   off[e] + (pairs of e before its workgroup) + (before its wave) + (before it
//   in its wave),
// the last from a wave-wide match of equal keys by ballots over the key's
// bits, so the order is the pairs' own and nothing depends on timing.  Up to
// kSortOne pairs one workgroup does it all; up to kSortAll every workgroup
// counts all pairs for itself; above, k_moe_count first counts each workgroup's
// segment and every workgroup of k_moe_sort then sums the counts before it.
// Dropped pairs form the last bucket, key E.  Latency bounds it, launches,
// barriers and dependent loads: 128 pairs take 3.1 us, 65536 pairs of 256 experts
// 2.7 + 7.0 us, of which the sums over the workgroups' counts are 2 and the scan
// with its four barriers 2.5.
// ---------------------------------------------------------------------------
constexpr int kMaxExperts = 960;       // 16 waves' counts, kept within 64 KB of LDS
// Pairs that one workgroup sorts, and that one launch does: 256 experts take 4.1
// us for 1024 pairs in one workgroup, 5.2 for 2048 (5.3 in two), 7.3 for 4096
// (5.5 in four that count all pairs, 7.3 in two launches); 8192 take 5.9 in one
// launch and 7.7 in two, 16384 7.1 and 7.8, but where all pairs have one expert,
// whose count they add to one after the other, 8192 take 11.7 and 8.6, 16384 18.8
// and 8.7.  With more than 512 experts one workgroup sorts twice as many: the
// counts of all pairs beside those of 16 waves are kept within 64 KB of LDS, which
// 960 experts would pass (70 KB).
constexpr int64_t kSortOne = 2048, kSortAll = 8192, kSortOneWide = 4096;
constexpr int64_t kSortBlocks = 256;   // most workgroups of the two-launch sort
constexpr int kSortWaves = 16;

template <typename ID>
__device__ __forceinline__ int sort_key(const ID* __restrict__ ids, int64_t ld, uint32_t K, uint32_t p, int E) {
  const int64_t i = ld == (int64_t)K ? (int64_t)p : (int64_t)(p / K) * ld + p % K;
  const ID v = ids[i];
  return v >= 0 && v < (ID)E ? (int)v : E;
}

template <typename ID>
__global__ __launch_bounds__(1024) void k_moe_count(const ID* __restrict__ ids, int64_t ld, uint32_t K, uint32_t P,
                                                     int E, uint32_t per_block, int32_t* __restrict__ hist) {
  extern __shared__ int32_t lds[];
  for (int e = threadIdx.x; e <= E; e += blockDim.x) lds[e] = 0;
  __syncthreads();
  const uint32_t p0 = blockIdx.x * per_block;
  const uint32_t p1 = min(p0 + per_block, P);
  for (uint32_t p = p0 + threadIdx.x; p < p1; p += blockDim.x) atomicAdd(&lds[sort_key(ids, ld, K, p, E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[(int64_t)blockIdx.x * E + e] = lds[e];
}

// Inclusive sum over the wave's 64 lanes by DPP row shifts and broadcasts: no
// lane exchange through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t dpp_add(int32_t v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int32_t wave_scan(int32_t v) {
  v = dpp_add<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8: inside rows of 16 lanes
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
}

// nb workgroups of nw waves (at most kSortWaves); each wave takes per_wave (a
// multiple of 64) consecutive pairs.  LDS: cnt[nw][E+1], scan[2][nw] and, with
// several workgroups and E at most half of blockDim, 2 * blockDim partial counts.
// blockDim > E: thread e deals with the bucket of expert e, thread E with that
// of the dropped pairs.
template <typename ID>
__global__ __launch_bounds__(1024) void k_moe_sort(const ID* __restrict__ ids, int64_t ld, uint32_t K, uint32_t P,
                                                    int E, int nbits, uint32_t per_wave,
                                                    const int32_t* __restrict__ hist, int32_t* __restrict__ offsets,
                                                    int32_t* __restrict__ row_of, int32_t* __restrict__ slot_of) {
  extern __shared__ int32_t lds[];
  const int nw = blockDim.x >> 6;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int EB = E + 1;
  int32_t* cnt = lds;             // [nw][E+1]
  int32_t* scan = lds + nw * EB;  // [2][nw]
  const uint32_t b0 = blockIdx.x * per_wave * nw;
  const uint32_t w0 = min(b0 + wave * per_wave, P);
  const uint32_t w1 = min(w0 + per_wave, P);
  const int e = threadIdx.x;

  // Expert e's pairs in all workgroups, and in those before this one: groups
  // of EP threads share the workgroups' counts, eight loads in flight.
  const int EP = (E + 63) & ~63, groups = hist != nullptr && EP > 0 ? (int)blockDim.x / EP : 0;
  int32_t total = 0, before = 0;
  if (groups > 0) {
    const int grp = e / EP, ee = e - grp * EP;
    if (grp < groups && ee < E) {
      const uint32_t last = gridDim.x - 1;
      for (uint32_t h0 = grp; h0 <= last; h0 += 8 * groups) {
        int32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = hist[(int64_t)min(h0 + i * groups, last) * E + ee];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          total += h0 + i * groups <= last ? h[i] : 0;
          before += h0 + i * groups < blockIdx.x ? h[i] : 0;
        }
      }
    }
  }
  for (int i = threadIdx.x; i < nw * EB; i += blockDim.x) cnt[i] = 0;
  int32_t* part = scan + 2 * nw;  // [2][blockDim.x]
  const bool all = hist == nullptr && gridDim.x > 1;
  if (all) part[e] = part[blockDim.x + e] = 0;
  __syncthreads();
  for (uint32_t p = w0 + lane; p < w1; p += 64) atomicAdd(&cnt[wave * EB + sort_key(ids, ld, K, p, E)], 1);
  if (all) {  // the other workgroups' pairs too: those before b0 apart
    for (uint32_t p0 = threadIdx.x; p0 < P; p0 += 8 * blockDim.x) {
      int key[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = sort_key(ids, ld, K, min(p0 + i * blockDim.x, P - 1), E);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t p = p0 + i * blockDim.x;
        if (p < P) atomicAdd(&part[(p < b0 ? blockDim.x : 0) + key[i]], 1);
      }
    }
  }
  if (groups > 1) {
    part[e] = total;
    part[blockDim.x + e] = before;
  }
  __syncthreads();

  int32_t c[kSortWaves];  // of bucket e in each wave
  if (e <= E) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = cnt[min(w, nw - 1) * EB + e];
  }
  if (groups > 1) {
    total = before = 0;
    if (e < E)
      for (int i = 0; i < groups; ++i) {
        total += part[i * EP + e];
        before += part[blockDim.x + i * EP + e];
      }
  } else if (all && e < E) {
    before = part[blockDim.x + e];
    total = part[e] + before;
  } else if (groups == 0 && e < E) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) total += w < nw ? c[w] : 0;
  }
  const int32_t incl = wave_scan(total), incl_before = wave_scan(before);
  if (lane == 63) {
    scan[wave] = incl;
    scan[nw + wave] = incl_before;
  }
  __syncthreads();
  int32_t off = incl - total, kept = 0, kept_before = 0;
  for (int w = 0; w < EP >> 6; ++w) {  // the waves that hold experts
    off += w < wave ? scan[w] : 0;
    kept += scan[w];
    kept_before += scan[nw + w];
  }
  if (e <= E) {
    if (blockIdx.x == 0) offsets[e] = e < E ? off : kept;
    // the row at which each wave's pairs of the bucket start
    int32_t run = e < E ? off + before : kept + (int32_t)min(b0, P) - kept_before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      if (w < nw) cnt[w * EB + e] = run;
      run += c[w];
    }
  }
  __syncthreads();

  for (uint32_t p0 = w0; p0 < w1; p0 += 64) {
    const uint32_t p = p0 + lane;
    const bool valid = p < w1;
    const int key = valid ? sort_key(ids, ld, K, p, E) : E;
    uint64_t same = __ballot(valid);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = (key >> b) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    const int lower = __popcll(same & ((1ull << lane) - 1));
    const int32_t row = cnt[wave * EB + key] + lower;
    __builtin_amdgcn_wave_barrier();  // every lane has read before the leaders advance
    if (valid && lower == 0) cnt[wave * EB + key] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (valid) {
      row_of[p] = key < E ? row : -1 - row;
      slot_of[row] = key < E ? (int32_t)p : -1 - (int32_t)p;
    }
  }
}

// ---------------------------------------------------------------------------
// Dispatch: a workgroup takes one token and a segment of its row, reads each
// 16-byte chunk once and writes it to the K rows of the token's experts.  The
// 1x128 scales lie [group][row], so they are gathered instead, by workgroups
// of their own at the end of the grid: 256 consecutive rows x kScaleGroups
// groups, written coalesced (the scales of all tokens stay in L2).  HBM writes
// bound it: 8192 tokens of 7168 codes to 65536 rows take 99 us, 545 MB at 5.5
// TB/s (109 through the caches); counters show each code and scale written once,
// the codes read once and the scales once by each of the eight L2s (76 MB read for
// 61).  A row's last 16 bytes are moved whole, some of them by two lanes (32768
// tokens of 8 rows of 259 codes: 23 us, 41 byte by byte); UNIT, the bytes of an
// element, is the step of rows shorter than that.  Narrow rows leave most lanes
// of their token's workgroup idle, with codes 252 of 256 at 64 channels: 32768
// tokens of 8 rows of 64 take 21 us, of which moving the bytes would be 4.
// ---------------------------------------------------------------------------
constexpr int kScaleGroups = 8;

// Sixteen bytes at any address.
typedef Words<4>::type Bytes16 __attribute__((aligned(1)));

template <int UNIT>
__device__ __forceinline__ uint4 load_part(const uint8_t* p, int64_t avail) {
  if (avail >= 16) {
    const auto v = *(const Global<const Bytes16>*)p;
    return make_uint4(v.x, v.y, v.z, v.w);
  }
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; j += UNIT)
    if (j < avail) {
      const uint32_t v = UNIT == 2 ? *reinterpret_cast<const uint16_t*>(p + j) : p[j];
      w[j >> 2] |= v << ((j & 3) * 8);
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int UNIT, bool NT>
__device__ __forceinline__ void store_part(uint8_t* p, int64_t avail, const uint4& v) {
  if (avail >= 16) {
    auto* q = (Global<Bytes16>*)p;
    if (NT) __builtin_nontemporal_store(Bytes16{v.x, v.y, v.z, v.w}, q);
    else *q = Bytes16{v.x, v.y, v.z, v.w};
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 16; j += UNIT)
    if (j < avail) {
      if (UNIT == 2)
        *reinterpret_cast<uint16_t*>(p + j) = (uint16_t)(w[j >> 2] >> ((j & 3) * 8));
      else
        p[j] = (uint8_t)(w[j >> 2] >> ((j & 3) * 8));
    }
}

template <int UNIT, bool SCALES, bool NT>
__global__ __launch_bounds__(256) void k_moe_dispatch(const uint8_t* __restrict__ x, int64_t ldx, int64_t row_bytes,
                                                       int64_t T, uint32_t K, const int32_t* __restrict__ row_of,
                                                       uint8_t* __restrict__ out, int64_t ldo, uint32_t segs,
                                                       const float* __restrict__ s, int64_t G,
                                                       const int32_t* __restrict__ slot_of, float* __restrict__ sr) {
  const int64_t P = T * K;
  const int64_t copies = T * segs;
  if (!SCALES || (int64_t)blockIdx.x < copies) {
    const int64_t t = blockIdx.x / segs;
    int64_t col = ((int64_t)(blockIdx.x % segs) * blockDim.x + threadIdx.x) * 16;
    if (col >= row_bytes) return;
    if (row_bytes >= 16 && col > row_bytes - 16) col = row_bytes - 16;  // a row's end: some bytes twice
    const int64_t avail = row_bytes - col;
    const uint4 v = load_part<UNIT>(x + t * ldx + col, avail);
    for (uint32_t k = 0; k < K; ++k) {
      const int32_t r = row_of[t * K + k];
      const int64_t row = r < 0 ? -1 - (int64_t)r : (int64_t)r;
      if (row < P) store_part<UNIT, NT>(out + row * ldo + col, avail, r < 0 ? make_uint4(0u, 0u, 0u, 0u) : v);
    }
    return;
  }
  const int64_t b = (int64_t)blockIdx.x - copies;
  const int64_t row_blocks = (P + 255) / 256;
  const int64_t r = (b % row_blocks) * 256 + threadIdx.x;
  const int64_t g0 = b / row_blocks * kScaleGroups;
  if (r >= P) return;
  const int32_t p = slot_of[r];
  const int64_t t = p < 0 ? -1 : (int64_t)((uint32_t)p / K);
#pragma unroll
  for (int i = 0; i < kScaleGroups; ++i) {
    if (g0 + i < G) sr[(g0 + i) * P + r] = t < 0 || t >= T ? 1.0f : s[(g0 + i) * T + t];
  }
}

// ---------------------------------------------------------------------------
// Combine: a workgroup takes one token and a segment of the row; a lane sums V
// channels over the token's rows in FP32, k ascending, loads of eight rows in
// flight.  V fills 16 bytes of the wider type, so that a wave's loads and
// stores are contiguous: FP32 in two accesses 32 bytes apart from lane to lane
// took 387 us instead of 347 for the rows (8192 tokens, 8 rows of 7168 each)
// and 348 instead of 252 for the sums (32768 tokens, one BF16 row of 7168 each).
// The last V channels of a row that ends inside a lane's are summed whole, some
// by two lanes (8192 tokens of one FP32 row of 7169: 77 us, 108 with the end
// moved and stored in pieces).  HBM reads bound it: 8192 tokens of 8 FP32 rows of
// 7168 take 319 us, 2.0 GB at 6.3 TB/s; a decode step of 16 tokens 3.6 us, its
// launch and two dependent loads.
// ---------------------------------------------------------------------------
template <typename TR, typename TY>
constexpr int combine_width() { return sizeof(TR) == 2 && sizeof(TY) == 2 ? 8 : 4; }

template <typename TR, typename TY, bool WEIGHTED, bool EXACT, bool NT>
__global__ __launch_bounds__(256) void k_moe_combine(const TR* __restrict__ rows, int64_t ldr, int64_t C, int64_t T,
                                                      uint32_t K, const int32_t* __restrict__ row_of,
                                                      const float* __restrict__ w, TY* __restrict__ y, int64_t ldy,
                                                      uint32_t segs) {
  constexpr int V = combine_width<TR, TY>();
  const int64_t P = T * K;
  const int64_t t = blockIdx.x / segs;
  int64_t col = ((int64_t)(blockIdx.x % segs) * blockDim.x + threadIdx.x) * V;
  if (col >= C) return;
  if (!EXACT && C >= V && col > C - V) col = C - V;  // a row's end: some channels by two lanes, alike
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  for (uint32_t k0 = 0; k0 < K; k0 += 8) {
    RawV<TR, V> raw[8];
    bool on[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t k = k0 + j;
      const int64_t r = k < K ? row_of[t * K + k] : -1;
      on[j] = r >= 0 && r < P;
      if (on[j]) raw[j] = load_end<V, EXACT, NT>(rows + r * ldr, col, C);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!on[j]) continue;
      const float wk = WEIGHTED ? w[t * K + k0 + j] : 1.0f;
      float v[V];
      unpack_v<TR, V>(raw[j], v);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = WEIGHTED ? __builtin_fmaf(wk, v[i], acc[i]) : acc[i] + v[i];
    }
  }
  store_end<V, EXACT, NT>(y + t * ldy, col, C, acc);
}

// ---------------------------------------------------------------------------
// Gradient of the combine: a workgroup takes one token, reads dy once, and for
// eight experts at a time reads their rows, adds up the eight dot products
// (FP32, lane by lane over the channels, then across lanes) and writes the
// eight scaled copies of dy: rows and their gradients pass once.  HBM bounds
// it, reads and writes of scattered rows in equal parts: 8192 tokens of 8 BF16
// rows of 7168 take 395 us, 2.0 GB at 5.1 TB/s.  The eight rows' addresses do not
// fit the scalar registers: 47 to 98 of them are kept in lanes of vector ones.
// ---------------------------------------------------------------------------
template <typename TY, typename TR, typename TD, bool EXACT, bool NT>
__global__ __launch_bounds__(512) void k_moe_combine_backward(const TY* __restrict__ dy, int64_t lddy,
                                                               const TR* __restrict__ rows, int64_t ldr, int64_t T,
                                                               uint32_t K, int64_t C,
                                                               const int32_t* __restrict__ row_of,
                                                               const float* __restrict__ w, TD* __restrict__ drows,
                                                               int64_t lddr, float* __restrict__ dw) {
  constexpr int V = sizeof(TY) == 2 && sizeof(TR) == 2 && sizeof(TD) == 2 ? 8 : 4;
  __shared__ float red[2][8 * 16];
  const int64_t P = T * K;
  const int64_t t = blockIdx.x;
  const int nw = blockDim.x >> 6;
  int turn = 0;
  for (uint32_t k0 = 0; k0 < K; k0 += 8) {
    int64_t row[8];  // -1: no such pair
    bool on[8];
    float wk[8], dot[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool is = k0 + j < K;
      const int32_t r = is ? row_of[t * K + k0 + j] : 0;
      row[j] = r < 0 ? -1 - (int64_t)r : (int64_t)r;
      on[j] = is && r >= 0 && row[j] < P;
      if (!is || row[j] >= P) row[j] = -1;
      wk[j] = on[j] ? w[t * K + k0 + j] : 0.0f;
      dot[j] = 0.0f;
    }
    for (int64_t c0 = (int64_t)threadIdx.x * V; c0 < C; c0 += (int64_t)blockDim.x * V) {
      // a row's end: `twice` channels by two lanes, alike but for the dot products
      const int64_t col = !EXACT && C >= V && c0 > C - V ? C - V : c0;
      const int twice = (int)(c0 - col);
      const bool ends = !EXACT && __ballot(twice > 0) != 0;
      float d[V];
      const RawV<TY, V> raw_dy = load_end<V, EXACT, false>(dy + t * lddy, col, C);
      RawV<TR, V> raw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (on[j]) raw[j] = load_end<V, EXACT, NT>(rows + row[j] * ldr, col, C);
      unpack_v<TY, V>(raw_dy, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (row[j] < 0) continue;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = on[j] ? wk[j] * d[i] : 0.0f;
        if (on[j]) {
          float v[V];
          unpack_v<TR, V>(raw[j], v);
          if (!ends) {
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = __builtin_fmaf(d[i], v[i], dot[j]);
          } else {
            asm volatile("");  // a branch, not a choice at each channel
#pragma unroll
            for (int i = 0; i < V; ++i) dot[j] = i >= twice ? __builtin_fmaf(d[i], v[i], dot[j]) : dot[j];
          }
        }
        store_end<V, EXACT, NT>(drows + row[j] * lddr, col, C, o);
      }
    }
    block_sum<8>(dot, red[turn], nw);
    turn ^= 1;
    if (threadIdx.x == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k0 + j < K) dw[t * K + k0 + j] = dot[j];
    }
  }
}

// Parts of a row and lanes per part (a multiple of 64, at most `most`) so that
// the row's chunks fill the lanes evenly.
struct RowSplit {
  uint32_t segs, lanes;
};
inline RowSplit split_row(int64_t chunks, int64_t most = 256) {
  RowSplit r;
  if (chunks < 1) chunks = 1;
  r.segs = (uint32_t)ceil_div(chunks, most);
  r.lanes = (uint32_t)(ceil_div(ceil_div(chunks, (int64_t)r.segs), (int64_t)64) * 64);
  return r;
}

constexpr int64_t kMaxPairs = 0x7FFFFFFF - (1 << 20);
// Channels: more than any memory holds, and few enough that neither a row's
// parts (RowSplit) nor the product of sizes overflow.
constexpr int64_t kMaxChannels = (int64_t)1 << 40;

// Sizes of a token matrix with K rows per token: FP8BLK_OK where they can be
// worked on.
inline fp8blk_status_t pairs_ok(int64_t T, int64_t K, int64_t C) {
  if (T < 0 || K < 0 || C < 0) return FP8BLK_ERR_INVALID_ARG;
  if ((K > 0 && T > kMaxPairs / K) || (T > 0 && C > kMaxChannels)) return FP8BLK_ERR_UNSUPPORTED;
  return FP8BLK_OK;
}

// Most pairs of one workgroup, and of one launch.
inline int64_t sort_one(int64_t E) { return E <= 512 ? kSortOne : kSortOneWide; }
inline int64_t sort_launch(int64_t E) { return E <= 512 ? kSortAll : kSortOneWide; }

inline int64_t sort_per_wave(int64_t P) {
  return ceil_div(ceil_div(P, kSortBlocks * kSortWaves), (int64_t)64) * 64;
}

template <typename ID>
fp8blk_status_t launch_sort(const ID* ids, int64_t ld, uint32_t K, int64_t P, int E, int32_t* offsets, int32_t* row_of,
                            int32_t* slot_of, int32_t* hist, hipStream_t stream) {
  int nbits = 0;
  while ((E >> nbits) != 0) ++nbits;
  if (P <= sort_one(E)) {
    int64_t nw = ceil_div(P, (int64_t)64);
    if (nw > kSortWaves) nw = kSortWaves;
    if (nw < ceil_div((int64_t)E + 1, (int64_t)64)) nw = ceil_div((int64_t)E + 1, (int64_t)64);
    const uint32_t per_wave = (uint32_t)(ceil_div(ceil_div(P, nw), (int64_t)64) * 64);
    const size_t lds = (size_t)(nw * (E + 1) + 2 * nw) * 4;
    hipLaunchKernelGGL(k_moe_sort<ID>, dim3(1), dim3((unsigned)nw * 64), lds, stream, ids, ld, K, (uint32_t)P, E, nbits,
                       per_wave, nullptr, offsets, row_of, slot_of);
    return launch_status();
  }
  const uint32_t per_wave = (uint32_t)sort_per_wave(P), per_block = per_wave * kSortWaves;
  const unsigned nb = (unsigned)ceil_div(P, (int64_t)per_block);
  if (P <= sort_launch(E)) {
    hist = nullptr;
  } else {
    hipLaunchKernelGGL(k_moe_count<ID>, dim3(nb), dim3(1024), (size_t)(E + 1) * 4, stream, ids, ld, K, (uint32_t)P, E,
                       per_block, hist);
    const fp8blk_status_t st = launch_status();
    if (st != FP8BLK_OK) return st;
  }
  const size_t lds = (size_t)(kSortWaves * (E + 1) + 2 * kSortWaves + (E <= 512 ? 2 * kSortWaves * 64 : 0)) * 4;
  hipLaunchKernelGGL(k_moe_sort<ID>, dim3(nb), dim3(kSortWaves * 64), lds, stream, ids, ld, K, (uint32_t)P, E, nbits,
                     per_wave, hist, offsets, row_of, slot_of);
  return launch_status();
}

struct CombineArgs {
  const void* rows;
  int64_t ldr, C, T;
  uint32_t K;
  const int32_t* row_of;
  const float* w;
  void* y;
  int64_t ldy;
};
template <typename TR, typename TY, bool WEIGHTED, bool EXACT, bool NT>
void launch_combine(const CombineArgs& a, RowSplit sp, hipStream_t stream) {
  hipLaunchKernelGGL((k_moe_combine<TR, TY, WEIGHTED, EXACT, NT>), dim3((unsigned)(a.T * sp.segs)), dim3(sp.lanes), 0,
                     stream, reinterpret_cast<const TR*>(a.rows), a.ldr, a.C, a.T, a.K, a.row_of, a.w,
                     reinterpret_cast<TY*>(a.y), a.ldy, sp.segs);
}
template <typename TR, typename TY>
void pick_combine(const CombineArgs& a, RowSplit sp, hipStream_t stream) {
  const bool exact = a.C % combine_width<TR, TY>() == 0;
  const bool nt = a.T * a.C * (int64_t)(a.K * sizeof(TR) + sizeof(TY)) >= kStreamBytes;
  if (a.w != nullptr) {
    if (!exact) return launch_combine<TR, TY, true, false, false>(a, sp, stream);
    return nt ? launch_combine<TR, TY, true, true, true>(a, sp, stream)
              : launch_combine<TR, TY, true, true, false>(a, sp, stream);
  }
  if (!exact) return launch_combine<TR, TY, false, false, false>(a, sp, stream);
  return nt ? launch_combine<TR, TY, false, true, true>(a, sp, stream)
            : launch_combine<TR, TY, false, true, false>(a, sp, stream);
}

// Lanes of a token's workgroup, at most.  Few rows a token leave a large
// workgroup waiting on its own start and reduction: 32768 tokens of one row of
// 7168 took 272 us with 256 lanes, 328 with 512 and 682 with 896, 16384 tokens
// of two rows of 4096 107 / 138 / 137; with 8 rows of 7168, 64 tokens took 9.4 /
// 8.2 / 8.6 and 8192 tokens 369 / 369 / 366.
inline int64_t combine_grad_lanes(uint32_t K) { return K < 4 ? 256 : 512; }

struct CombineGradArgs {
  const void* dy;
  int64_t lddy;
  const void* rows;
  int64_t ldr, T;
  uint32_t K;
  int64_t C;
  const int32_t* row_of;
  const float* w;
  void* drows;
  int64_t lddr;
  float* dw;
  uint32_t lanes;  // of a token's workgroup
};
template <typename TY, typename TR, typename TD, bool EXACT, bool NT>
void launch_combine_backward(const CombineGradArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((k_moe_combine_backward<TY, TR, TD, EXACT, NT>), dim3((unsigned)a.T), dim3(a.lanes), 0, stream,
                     reinterpret_cast<const TY*>(a.dy), a.lddy, reinterpret_cast<const TR*>(a.rows), a.ldr, a.T, a.K,
                     a.C, a.row_of, a.w, reinterpret_cast<TD*>(a.drows), a.lddr, a.dw);
}
template <typename TY, typename TR, typename TD>
void pick_combine_backward(const CombineGradArgs& a, hipStream_t stream) {
  if (a.C % 8 != 0) return launch_combine_backward<TY, TR, TD, false, false>(a, stream);
  if (a.T * a.K * a.C * (int64_t)(sizeof(TR) + sizeof(TD)) >= kStreamBytes)
    return launch_combine_backward<TY, TR, TD, true, true>(a, stream);
  return launch_combine_backward<TY, TR, TD, true, false>(a, stream);
}

}  // namespace fp8blk

using namespace fp8blk;

extern "C" int fp8blk_layer_abi_version(void) { return 1; }

extern "C" size_t fp8blk_moe_sort_workspace_bytes(int64_t T, int64_t K, int64_t E) {
  if (pairs_ok(T, K, 0) != FP8BLK_OK || E < 0 || E > kMaxExperts || T * K <= sort_launch(E)) return 0;
  return (size_t)(ceil_div(T * K, sort_per_wave(T * K) * kSortWaves) * E) * 4;
}

extern "C" fp8blk_status_t fp8blk_moe_sort(const void* expert_ids, int64_t T, int64_t K, int64_t ld, int64_t E,
                                           int32_t* offsets, int32_t* row_of, int32_t* slot_of, void* workspace,
                                           size_t workspace_bytes, uint32_t flags, void* stream) {
  if ((flags & ~FP8BLK_MOE_IDS_I64) || E < 0) return FP8BLK_ERR_INVALID_ARG;
  const fp8blk_status_t st = pairs_ok(T, K, 0);
  if (st != FP8BLK_OK) return st;
  if (E > kMaxExperts) return FP8BLK_ERR_UNSUPPORTED;
  const bool i64 = (flags & FP8BLK_MOE_IDS_I64) != 0;
  const int64_t P = T * K;
  if (!vec_ok(offsets, E + 1)) return FP8BLK_ERR_INVALID_ARG;
  if (P > 0 && (ld < K || !vec_ok(expert_ids, P, i64 ? 8 : 4) || !vec_ok(row_of, P) || !vec_ok(slot_of, P)))
    return FP8BLK_ERR_INVALID_ARG;
  const size_t need = fp8blk_moe_sort_workspace_bytes(T, K, E);
  if (need != 0 && (workspace == nullptr || !aligned(workspace, 4) || workspace_bytes < need))
    return FP8BLK_ERR_INVALID_ARG;
  if (i64)
    return launch_sort(reinterpret_cast<const int64_t*>(expert_ids), ld, (uint32_t)K, P, (int)E, offsets, row_of,
                       slot_of, reinterpret_cast<int32_t*>(workspace), as_stream(stream));
  return launch_sort(reinterpret_cast<const int32_t*>(expert_ids), ld, (uint32_t)K, P, (int)E, offsets, row_of, slot_of,
                     reinterpret_cast<int32_t*>(workspace), as_stream(stream));
}

extern "C" fp8blk_status_t fp8blk_moe_dispatch(const uint16_t* x, int64_t T, int64_t C, int64_t ldx, int64_t K,
                                               const int32_t* row_of, uint16_t* out, int64_t ldo, void* stream) {
  const fp8blk_status_t st = pairs_ok(T, K, C);
  if (st != FP8BLK_OK) return st;
  if (T == 0 || K == 0 || C == 0) return FP8BLK_OK;
  if (!matrix_ok(x, T, C, ldx, 2) || !matrix_ok(out, T * K, C, ldo, 2) || !vec_ok(row_of, T * K))
    return FP8BLK_ERR_INVALID_ARG;
  const RowSplit sp = split_row(ceil_div(2 * C, (int64_t)16));
  if (!grid_ok(T * sp.segs, sp.lanes)) return FP8BLK_ERR_UNSUPPORTED;
  const bool nt = 2 * T * (K + 1) * C >= kStreamBytes;
  hipLaunchKernelGGL((nt ? k_moe_dispatch<2, false, true> : k_moe_dispatch<2, false, false>),
                     dim3((unsigned)(T * sp.segs)), dim3(sp.lanes), 0, as_stream(stream),
                     reinterpret_cast<const uint8_t*>(x), 2 * ldx, 2 * C, T, (uint32_t)K, row_of,
                     reinterpret_cast<uint8_t*>(out), 2 * ldo, sp.segs, nullptr, (int64_t)0, nullptr, nullptr);
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_moe_dispatch_fp8(const uint8_t* q, int64_t T, int64_t C, int64_t ldq, const float* s,
                                                   int64_t K, const int32_t* row_of, const int32_t* slot_of,
                                                   uint8_t* qr, int64_t ldqr, float* sr, void* stream) {
  const fp8blk_status_t st = pairs_ok(T, K, C);
  if (st != FP8BLK_OK) return st;
  if (T == 0 || K == 0 || C == 0) return FP8BLK_OK;
  const int64_t G = ceil_div(C, (int64_t)128), P = T * K;
  if (!matrix_ok(q, T, C, ldq, 1) || !matrix_ok(qr, P, C, ldqr, 1) || !vec_ok(s, T) || !vec_ok(sr, P) ||
      !vec_ok(row_of, P) || !vec_ok(slot_of, P))
    return FP8BLK_ERR_INVALID_ARG;
  RowSplit sp = split_row(ceil_div(C, (int64_t)16));
  sp.lanes = 256;  // the scale workgroups take 256 rows each
  const int64_t blocks = T * sp.segs + ceil_div(P, (int64_t)256) * ceil_div(G, (int64_t)kScaleGroups);
  if (!grid_ok(blocks, sp.lanes)) return FP8BLK_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(((P + T) * C >= kStreamBytes ? k_moe_dispatch<1, true, true> : k_moe_dispatch<1, true, false>),
                     dim3((unsigned)blocks), dim3(sp.lanes), 0, as_stream(stream), q, ldq, C, T, (uint32_t)K, row_of, qr,
                     ldqr, sp.segs, s, G, slot_of, sr);
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_moe_combine(const void* rows, int64_t T, int64_t K, int64_t C, int64_t ldr,
                                              const int32_t* row_of, const float* weights, void* y, int64_t ldy,
                                              uint32_t flags, void* stream) {
  if (flags & ~(FP8BLK_MOE_ROWS_F32 | FP8BLK_MOE_TOKENS_F32)) return FP8BLK_ERR_INVALID_ARG;
  const fp8blk_status_t st = pairs_ok(T, K, C);
  if (st != FP8BLK_OK) return st;
  if (T == 0 || C == 0) return FP8BLK_OK;
  const bool rf = (flags & FP8BLK_MOE_ROWS_F32) != 0, yf = (flags & FP8BLK_MOE_TOKENS_F32) != 0;
  if (!matrix_ok(rows, T * K, C, ldr, rf ? 4 : 2) || !matrix_ok(y, T, C, ldy, yf ? 4 : 2) || !vec_ok(row_of, T * K) ||
      (weights != nullptr && !aligned(weights, 4)))
    return FP8BLK_ERR_INVALID_ARG;
  const RowSplit sp = split_row(ceil_div(C, (int64_t)(rf || yf ? 4 : 8)));
  if (!grid_ok(T * sp.segs, sp.lanes)) return FP8BLK_ERR_UNSUPPORTED;
  const CombineArgs a{rows, ldr, C, T, (uint32_t)K, row_of, weights, y, ldy};
  auto* go = rf ? (yf ? pick_combine<float, float> : pick_combine<float, uint16_t>)
                : (yf ? pick_combine<uint16_t, float> : pick_combine<uint16_t, uint16_t>);
  go(a, sp, as_stream(stream));
  return launch_status();
}

extern "C" fp8blk_status_t fp8blk_moe_combine_backward(const void* dy, int64_t lddy, const void* rows, int64_t ldr,
                                                       int64_t T, int64_t K, int64_t C, const int32_t* row_of,
                                                       const float* weights, void* drows, int64_t lddr,
                                                       float* dweights, uint32_t flags, void* stream) {
  if (flags & ~(FP8BLK_MOE_ROWS_F32 | FP8BLK_MOE_TOKENS_F32 | FP8BLK_MOE_DROWS_F32)) return FP8BLK_ERR_INVALID_ARG;
  const fp8blk_status_t st = pairs_ok(T, K, C);
  if (st != FP8BLK_OK) return st;
  if (T == 0 || K == 0) return FP8BLK_OK;
  const bool yf = (flags & FP8BLK_MOE_TOKENS_F32) != 0, rf = (flags & FP8BLK_MOE_ROWS_F32) != 0;
  const bool df = (flags & FP8BLK_MOE_DROWS_F32) != 0;
  if (!matrix_ok(dy, T, C, lddy, yf ? 4 : 2) || !matrix_ok(rows, T * K, C, ldr, rf ? 4 : 2) ||
      !matrix_ok(drows, T * K, C, lddr, df ? 4 : 2) || !vec_ok(row_of, T * K) || !vec_ok(weights, T * K) ||
      !vec_ok(dweights, T * K))
    return FP8BLK_ERR_INVALID_ARG;
  // channels of a lane as in k_moe_combine_backward: 16 bytes of the widest type
  const uint32_t lanes = split_row(ceil_div(C, (int64_t)(yf || rf || df ? 4 : 8)), combine_grad_lanes((uint32_t)K)).lanes;
  if (!grid_ok(T, lanes)) return FP8BLK_ERR_UNSUPPORTED;
  using U = uint16_t;
  using F = float;
  const CombineGradArgs a{dy, lddy, rows, ldr, T, (uint32_t)K, C, row_of, weights, drows, lddr, dweights, lanes};
  auto* go = yf ? (rf ? (df ? pick_combine_backward<F, F, F> : pick_combine_backward<F, F, U>)
                      : (df ? pick_combine_backward<F, U, F> : pick_combine_backward<F, U, U>))
                : (rf ? (df ? pick_combine_backward<U, F, F> : pick_combine_backward<U, F, U>)
                      : (df ? pick_combine_backward<U, U, F> : pick_combine_backward<U, U, U>));
  go(a, as_stream(stream));
  return launch_status();
}
