// What the decode kernels read of a query row, with its checks.
#pragma once

#include "decode_internal.h"
#include "kv_layout.cuh"

namespace stem {

// Sequence and visible length of row r; a row that names no sequence of the cache, or a length
// outside it, sets the status word and counts as empty.
__host__ __device__ __forceinline__ void decode_row(const KvCache& c, const DecodeRows& r, int row,
                                                    int& seq, int& len) {
  seq = r.rows ? r.rows[row] : row;
  len = r.lens[row];
  const bool ok = seq >= 0 && seq < c.nseq && len >= 0 &&
                  static_cast<int64_t>(len) <= static_cast<int64_t>(c.max_blocks) * c.block;
  if (!ok) {
    if (r.status) *r.status = STEM_ERR_ARG;
    seq = 0;
    len = 0;
  }
}

// Entries of a part where the number of all entries (below 2^31) sets it. As it is not less than an
// at_once-th of them, items with n_i entries have sum ceil(n_i / chunk) <= items + at_once parts.
// Half as much again as an even share: fewer items are cut, and the CTAs that come free take the rest.
// (With 1.25, 1.5 and 2 even shares: 32 ragged rows of per-head lists of up to 16K at 16 bits take 111,
// 101 and 100 us; every block of 4 ragged rows of up to 64K at 8 bits 53, 55 and 64; a selection and
// its attention of 64 rows of up to 32K at 4 bits 90 with each.)
__host__ __device__ __forceinline__ int part_entries(int total, int at_once, int least) {
  const int chunk = static_cast<int>((total / 2 * int64_t{3} + at_once - 1) / at_once);
  return chunk > least ? chunk : least;
}

__device__ __forceinline__ Entry entry_of(const KvCache& c, int seq, int j, uint32_t heads,
                                          int32_t* status) {
  const int page = kv_page(c, seq, j, status);
  return page < 0 ? Entry{0, 0u} : Entry{page, static_cast<uint32_t>(j) | heads << 16};
}

// The list of an item from its blocks' head bits, in block order: mask holds a byte for each of the
// blocks 0 .. last (last < 0: none). Called by a CTA of THREADS threads; scan: THREADS / 32 words.
template <int THREADS>
__device__ __forceinline__ void write_union(const KvCache& c, const DecodeLists& lists,
                                            int64_t item, int seq, int last, int nh,
                                            const uint32_t* mask, uint32_t* scan,
                                            int32_t* status) {
  const int tid = threadIdx.x, words = last < 0 ? 0 : last / 4 + 1;
  const uint32_t none = 0xffu << nh & 0xffu;  // columns without a head go along with any block
  const int run = (words + THREADS - 1) / THREADS;  // thread t owns a run of words
  const int w0 = min(tid * run, words), w1 = min(w0 + run, words);
  uint32_t n = 0;
  for (int w = w0; w < w1; ++w)
    for (int b = 0; b < 4; ++b) n += (mask[w] >> (8 * b) & 0xffu) != 0;
  uint32_t s = n;
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (tid % 32 >= o) s += y;
  }
  __syncthreads();
  if (tid % 32 == 31) scan[tid / 32] = s;
  __syncthreads();
  uint32_t total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < tid / 32) s += scan[w];
    total += scan[w];
  }
  uint32_t at = s - n;
  Entry* out = lists.list + item * lists.most;
  for (int w = w0; w < w1; ++w)
    for (int b = 0; b < 4; ++b) {
      const uint32_t m = mask[w] >> (8 * b) & 0xffu;
      if (m) out[at++] = entry_of(c, seq, 4 * w + b, m | none, status);
    }
  if (tid == 0) lists.count[item] = static_cast<int32_t>(total);
}

}  // namespace stem
