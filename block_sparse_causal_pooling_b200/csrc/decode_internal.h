// Internal declarations of the decode path (cache.cu, decode_select.cu, decode_attn.cu) shared
// with its host API (decode_api.cpp).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "stem_internal.h"

namespace stem {

struct KvCache;

// Writes (write) or reads back rows of K and V: k, v [nseq, Hkv, T, D] with the given strides in
// elements, tokens pos[s] .. pos[s] + count[s] - 1 of sequence s (cache.cu).
cudaError_t launch_cache_rows(bool write, int format, int D, int dtype, const KvCache& c, void* k,
                              void* v, int T, int64_t s_seq, int64_t s_head, int64_t s_tok,
                              const int32_t* pos, const int32_t* count, int32_t* status,
                              cudaStream_t st);

// The query rows of a decode call and the lists of their kept blocks.
struct DecodeRows {
  const void* q;  // bfloat16 [R, Hq, D]
  int R, Hq;
  const int32_t* rows;  // sequence of each row, NULL: row r is sequence r
  const int32_t* lens;  // cached tokens each row sees
  int kcap;             // entries of a list
  int32_t* sel_idx;     // [R, Hq, kcap]
  int32_t* sel_cnt;     // [R, Hq]
  int32_t* status;
};

// An entry of the attention's lists: the block's page, the block | query heads that keep it << 16.
struct Entry {
  int page;
  uint32_t what;
};
constexpr int kDecodeHeads = 8;  // query heads of an item (columns of an MMA)

// One list of blocks for each (row, kv head) where its heads share it, else for each item (row, kv
// head, 8 of its query heads): [lists][most] and [lists].
struct DecodeLists {
  Entry* list = nullptr;
  int32_t* count = nullptr;
  int32_t* arrived = nullptr;  // [items]: parts of the item that are there; whoever writes the lists
                               // sets it to 0
  int most = 0;
  int tiles_h = 0;  // items of a kv head
};

// Block scores and selection (decode_select.cu); writes the attention's lists too where lists.list
// is not NULL.
cudaError_t launch_decode_select(const KvCache& c, int D, const DecodeRows& r,
                                 const int32_t* budget, SelMetric metric, const DecodeLists& lists,
                                 cudaStream_t st);

// Attention over the kept blocks (decode_attn.cu). share: the query heads of a kv head have one
// list (that of the first). ws: decode_attn_bytes() of workspace, 256-byte aligned; planned: its
// lists are there already.
DecodeLists decode_lists(const KvCache& c, int format, int D, const DecodeRows& r, bool share,
                         unsigned char* ws);
cudaError_t launch_decode_attn(const KvCache& c, int format, int D, const DecodeRows& r, bool share,
                               bool planned, void* out, float* lse, unsigned char* ws,
                               cudaStream_t st);
size_t decode_attn_bytes(int format, int D, int block, int Hkv, int max_blocks, int R, int Hq,
                         int kcap, bool share);

}  // namespace stem
