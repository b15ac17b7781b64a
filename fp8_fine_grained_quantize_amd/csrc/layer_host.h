// Host-side rules shared by the operators around the GEMMs.
#pragma once

#include "host_common.h"

namespace fp8blk {

// A call that moves this many bytes (reads and writes, the size of the
// Infinity Cache) reads its rows and writes its outputs as streams, past the
// caches: little of them would be left there for a next reader.  Measured both
// ways, alone and followed by a reader of the outputs:
//   combine of 8 FP32 rows of 7168 per token, then residual_norm: 4096 tokens
//   (952 MB moved) 203 us streamed, 246 cached; 1024 tokens (238 MB) 53 / 59;
//   512 tokens (119 MB) 28 / 27.
//   dispatch of BF16 rows, then combine: 4096 tokens (504 MB) 210 / 240,
//   2048 (252 MB) 99 / 89, 256 (32 MB) 14 / 13.
//   residual_norm of 8192 x 7168 to BF16 and E4M3 alone 103 / 109, its
//   gradient 125 / 137; clipping of 3.8 GB 2021 / 2122.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// A launch counts its lanes in 32 bits.
inline bool grid_ok(int64_t blocks, int64_t lanes) { return blocks <= 0xFFFFFFFFll / lanes && blocks <= 0x7FFFFFFF; }

}  // namespace fp8blk
