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

}  // namespace stem
