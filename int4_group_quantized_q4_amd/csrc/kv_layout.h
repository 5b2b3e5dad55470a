// The key-value cache's layout in one page, shared by the kernels that write,
// read and attend over it (see w4a16.h).
#pragma once

#include "common.h"
#include "w4a16.h"

namespace w4 {

constexpr int kKvTile = 16;   // tokens per tile

// Sizes of a cache format at NG groups of 32 dimensions per head.
template <int FMT, int NG>
struct KvLayout {
  static constexpr int D = 32 * NG;
  static constexpr int U = FMT == W4_KV_BF16 ? 1 : FMT == W4_KV_E4M3 ? 2 : (NG < 4 ? NG : 4);   // groups per unit
  static constexpr int NU = NG / U;                                                           // units per tile
  static constexpr int kGroupBytes = FMT == W4_KV_BF16 ? 16 : FMT == W4_KV_E4M3 ? 8 : 4;     // of one lane
  static constexpr int kUnitBytes = U * kGroupBytes;      // of one lane: 16 (8 for Q4 at 64 dimensions)
  static constexpr int kTileBytes = NU * 64 * kUnitBytes; // codes of 16 tokens
  static constexpr int kScaleTileBytes = FMT == W4_KV_BF16 ? 0 : FMT == W4_KV_E4M3 ? 64 : 32 * NG;
};

// Bytes of a head's K (or V) rows in a page of `page` tokens.
__host__ __device__ constexpr int64_t kv_block_bytes(int fmt, int64_t page, int64_t dim) {
  return fmt == W4_KV_BF16 ? page * dim * 2 : fmt == W4_KV_E4M3 ? page * (dim + 4) : page * (dim / 2 + dim / 16);
}

}  // namespace w4
