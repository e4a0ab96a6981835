// Layout of the paged K/V cache, shared by the kernels that write, read and attend over it
// (the byte-level description is in include/stem.h).
//
// A page is one selection block of one sequence; its record for one kv head is block/16 tiles of
// 16 tokens, each [K codes | V codes | scales]. Inside a tile the codes lie in the order in which
// a warp's mma.m16n8k16 fragments want them, so a lane reads its operand words as whole 16-byte
// pieces at lane * 16 (no bank conflicts, no transposition):
//   K (A operand of K Q^T; rows are tokens): lane 4g + t holds tokens g and g + 8 and, of each
//     32-channel group, channels 8t .. 8t + 7;
//   V (A operand of V^T P; rows are channels): lane 4g + t holds token pairs (2t, 2t + 1) and
//     (2t + 8, 2t + 9) and, of each group, channels 4g .. 4g + 3; the two tokens of a pair share
//     each 32-bit word (low and high half).
// Codes of 4 and 8 bits are stored with an offset of 8 and 128, so that a masked word is a pair
// of fp16 subnormals code * 2^-24: no conversion instruction stands between memory and the MMA.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "stem.h"

namespace stem {

constexpr int kKvGroup = 32;  // channels that share a scale
constexpr int kKvTile = 16;   // tokens of a tile

template <int FMT, int D>
struct Kv {
  static constexpr int NG = D / kKvGroup;                                  // groups of a row
  static constexpr int WPG = FMT == STEM_KV_BF16 ? 4 : FMT == STEM_KV_Q8 ? 2 : 1;  // words, below
  static constexpr int BITS = FMT == STEM_KV_BF16 ? 16 : FMT == STEM_KV_Q8 ? 8 : 4;
  static constexpr int PIECES = 2 * NG * WPG / 4;  // 16-byte pieces a lane holds of K (or of V)
  static constexpr int CODES = PIECES * 512;       // bytes of a tile's K (or V) codes
  static constexpr int SCROW = FMT == STEM_KV_BF16 ? 0 : 4 * NG;  // scale bytes of a token (K | V)
  static constexpr int TILE_BYTES = 2 * CODES + kKvTile * SCROW;
  static constexpr int QMAX = FMT == STEM_KV_Q8 ? 127 : 7;
  static constexpr int OFFSET = FMT == STEM_KV_Q8 ? 128 : 8;
  static_assert(CODES == kKvTile * D * BITS / 8, "a tile's codes fill their pieces");

  // Byte offset in a tile's K (or V) codes of word w of (row half i, group g) of a lane.
  static __host__ __device__ constexpr int word(int i, int g, int w, int lane) {
    const int n = (i * NG + g) * WPG + w;
    return ((n / 4) * 32 + lane) * 16 + (n % 4) * 4;
  }
};

inline int kv_tile_bytes(int fmt, int D) {
  const int bits = fmt == STEM_KV_BF16 ? 16 : fmt == STEM_KV_Q8 ? 8 : 4;
  return kKvTile * D * 2 * bits / 8 + (fmt == STEM_KV_BF16 ? 0 : kKvTile * 4 * (D / kKvGroup));
}

inline __host__ __device__ int64_t kv_record_bytes(int tile_bytes, int block) {
  return static_cast<int64_t>(tile_bytes) * (block / kKvTile);
}

// What every cache kernel gets of a stem_cache_t (by value).
struct KvCache {
  unsigned char* pages;
  float* kbar;
  float* vnorm;
  const int32_t* table;
  int num_pages, Hkv, block, nseq, max_blocks;
  int64_t record;  // bytes of one (page, kv head)
  bool vmax;

  __host__ __device__ __forceinline__ unsigned char* at(int page, int head) const {
    return pages + (static_cast<int64_t>(page) * Hkv + head) * record;
  }
};

// The page of block j of a sequence, or -1 (with the status word set) when the table's entry is
// not a page of the cache. seq and j are in range.
__host__ __device__ __forceinline__ int kv_page(const KvCache& c, int seq, int j, int32_t* status) {
  const int p = c.table[static_cast<int64_t>(seq) * c.max_blocks + j];
  if (p >= 0 && p < c.num_pages) return p;
  if (status) *status = STEM_ERR_ARG;
  return -1;
}

// The part of tokens pos .. pos + n - 1 that lies in the b-th block they touch: block j, tokens
// [lo, hi) of it, and the row (may be negative) of the block's token 0. False: nothing to do, with
// the status word set where the range is not one of the cache or n is above most.
__host__ __device__ __forceinline__ bool kv_block_rows(const KvCache& c, int64_t pos, int64_t n,
                                                       int most, int b, int32_t* status, int& j,
                                                       int& first, int& lo, int& hi) {
  if (n == 0) return false;
  const int64_t cap = static_cast<int64_t>(c.max_blocks) * c.block;
  if (pos < 0 || n < 0 || n > most || pos + n > cap) {
    if (status) *status = STEM_ERR_ARG;
    return false;
  }
  const int64_t jj = pos / c.block + b, b0 = jj * c.block, end = pos + n;
  if (b0 >= end) return false;
  j = static_cast<int>(jj);
  lo = static_cast<int>(pos > b0 ? pos - b0 : 0);
  hi = static_cast<int>(end - b0 < c.block ? end - b0 : c.block);
  first = static_cast<int>(b0 - pos);
  return true;
}

}  // namespace stem
