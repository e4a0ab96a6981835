// C ABI of the decode path (declared in include/stem.h): validation, workspace carve-up and the
// launch sequence for the paged cache and the attention of single query tokens.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "decode_internal.h"
#include "kv_layout.cuh"
#include "stem.h"

namespace stem {
namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxGrid = 65535;  // of the second and third grid dimension

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_err(cudaError_t e) {
  if (e == cudaSuccess) return STEM_OK;
  cudaGetLastError();  // clear a sticky launch error in this thread's runtime state
  return STEM_ERR_CUDA;
}

int check_format(int D, int block, int format) {
  if (D != 64 && D != 128) return STEM_ERR_ARG;
  if (block != 64 && block != 128) return STEM_ERR_ARG;
  if (format != STEM_KV_BF16 && format != STEM_KV_Q8 && format != STEM_KV_Q4) return STEM_ERR_ARG;
  return STEM_OK;
}

int check_cache(const stem_cache_t* c) {
  if (c == nullptr) return STEM_ERR_ARG;
  const int rc = check_format(c->D, c->block, c->format);
  if (rc != STEM_OK) return rc;
  if (c->num_pages < 0 || c->Hkv < 1 || c->nseq < 0 || c->max_blocks < 1) return STEM_ERR_ARG;
  if (c->vsum != STEM_VSUM_MEAN && c->vsum != STEM_VSUM_MAX) return STEM_ERR_ARG;
  if (c->max_blocks > STEM_MAX_NB) return STEM_ERR_UNSUPPORTED;
  if (c->Hkv > kMaxGrid || c->nseq > kMaxGrid) return STEM_ERR_UNSUPPORTED;
  return STEM_OK;
}

int check_buffers(const stem_cache_t* c) {
  if (!c->pages || !c->kbar || !c->vnorm || !c->table) return STEM_ERR_ARG;
  if (!aligned(c->pages, 16) || !aligned(c->kbar, 16) || !aligned(c->vnorm, 4) ||
      !aligned(c->table, 4))
    return STEM_ERR_ARG;
  return STEM_OK;
}

KvCache device_cache(const stem_cache_t* c) {
  KvCache d;
  d.pages = static_cast<unsigned char*>(c->pages);
  d.kbar = c->kbar;
  d.vnorm = c->vnorm;
  d.table = c->table;
  d.num_pages = c->num_pages;
  d.Hkv = c->Hkv;
  d.block = c->block;
  d.nseq = c->nseq;
  d.max_blocks = c->max_blocks;
  d.record = kv_record_bytes(kv_tile_bytes(c->format, c->D), c->block);
  d.vmax = c->vsum == STEM_VSUM_MAX;
  return d;
}

int clear_status(int32_t* status, cudaStream_t st) {
  return status ? cuda_err(cudaMemsetAsync(status, 0, sizeof(int32_t), st)) : STEM_OK;
}

// Rows that are written need places of their own: each step, from the smallest on, leaves what the
// smaller ones span behind it.
bool apart(const int64_t* step, const int32_t* extent, int D) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return step[a] < step[b]; });
  int64_t span = D;
  for (const int n : order) {
    if (extent[n] < 2) continue;
    if (step[n] < span) return false;
    if (step[n] > (INT64_MAX - span) / (extent[n] - 1)) return false;  // (past any memory)
    span += step[n] * (extent[n] - 1);
  }
  return true;
}

int cache_rows(bool write, const stem_cache_t* c, void* k, void* v, int dtype, int T,
               const int64_t* strides, const int32_t* pos, const int32_t* count, int32_t* status,
               cudaStream_t st) {
  int rc = check_cache(c);
  if (rc != STEM_OK) return rc;
  if (dtype != STEM_BF16 && dtype != STEM_F32) return STEM_ERR_ARG;
  if (T < 0 || strides == nullptr) return STEM_ERR_ARG;
  if (static_cast<int64_t>(T) > static_cast<int64_t>(c->max_blocks) * c->block) return STEM_ERR_ARG;
  const int64_t elt = dtype == STEM_BF16 ? 2 : 4;
  const int32_t extent[3] = {c->nseq, c->Hkv, T};
  int64_t step[3];  // (along an axis of one row there is none, whatever its stride says)
  for (int n = 0; n < 3; ++n) {
    step[n] = extent[n] > 1 ? strides[n] : 0;
    if (step[n] < 0 || step[n] * elt % 16 != 0) return STEM_ERR_ARG;
  }
  if (c->nseq == 0 || T == 0) return STEM_OK;
  if (!write && !apart(step, extent, c->D)) return STEM_ERR_ARG;
  if ((rc = check_buffers(c)) != STEM_OK) return rc;
  if (!k || !v || !pos || !aligned(k, 16) || !aligned(v, 16) || !aligned(pos, 4) ||
      !aligned(count, 4) || !aligned(status, 4))
    return STEM_ERR_ARG;
  if ((rc = clear_status(status, st)) != STEM_OK) return rc;
  return cuda_err(launch_cache_rows(write, c->format, c->D, dtype, device_cache(c), k, v, T,
                                    step[0], step[1], step[2], pos, count, status, st));
}

// ------------------------------------------------------------------ decode

// The workspace depends on whether heads share lists: the larger of the two, so that one size
// serves every method.
size_t workspace(const stem_cache_t* c, int R, int Hq, int kcap) {
  size_t most = kAlign;
  for (int share = 0; share < 2; ++share) {
    const size_t n = decode_attn_bytes(c->format, c->D, c->block, c->Hkv, c->max_blocks, R, Hq,
                                       kcap, share != 0);
    if (n > most) most = n;
  }
  return align_up(most);
}

int check_shape(const stem_cache_t* c, int R, int Hq, int kcap) {
  const int rc = check_cache(c);
  if (rc != STEM_OK) return rc;
  if (R < 0 || Hq < 1 || Hq % c->Hkv != 0 || kcap < 1 || kcap > c->max_blocks) return STEM_ERR_ARG;
  if (R > kMaxGrid || Hq > kMaxGrid ||
      static_cast<int64_t>(R) * Hq * c->max_blocks > 0x7fffffffLL)
    return STEM_ERR_UNSUPPORTED;
  return STEM_OK;
}

// What the two stages have in common; returns 1 for an empty call.
int check_decode(const stem_decode_args_t* a, bool select, bool attend) {
  if (a == nullptr) return STEM_ERR_ARG;
  int rc = check_shape(a->cache, a->R, a->Hq, a->kcap);
  if (rc != STEM_OK) return rc;
  if (a->dtype != STEM_BF16 && a->dtype != STEM_F32) return STEM_ERR_ARG;
  if (a->dtype != STEM_BF16) return STEM_ERR_UNSUPPORTED;
  const stem_method_t* m = a->method;
  if (m == nullptr) return STEM_ERR_ARG;
  if (m->share != STEM_SHARE_HEAD && m->share != STEM_SHARE_GROUP) return STEM_ERR_ARG;
  if (select) {
    if (m->metric != STEM_METRIC_PRODUCT && m->metric != STEM_METRIC_ADDITIVE) return STEM_ERR_ARG;
    if (m->metric == STEM_METRIC_ADDITIVE &&
        (!(std::isfinite(m->beta) && m->beta >= 0.0f) || (m->clamp != 0 && m->clamp != 1)))
      return STEM_ERR_ARG;
    if (m->score != STEM_SCORE_POOLED && m->score != STEM_SCORE_ANTIDIAG) return STEM_ERR_ARG;
    if (m->score != STEM_SCORE_POOLED) return STEM_ERR_UNSUPPORTED;
  }
  if (a->R == 0) return 1;
  if ((rc = check_buffers(a->cache)) != STEM_OK) return rc;
  if (a->cache->nseq == 0) return STEM_ERR_ARG;
  if (!a->rows && a->R > a->cache->nseq) return STEM_ERR_ARG;
  if (!a->q || !a->lens || !a->sel_idx || !a->sel_cnt) return STEM_ERR_ARG;
  if (!aligned(a->q, 16) || !aligned(a->lens, 4) || !aligned(a->rows, 4) ||
      !aligned(a->sel_idx, 4) || !aligned(a->sel_cnt, 4) || !aligned(a->status, 4))
    return STEM_ERR_ARG;
  if (select && (!a->budget || !aligned(a->budget, 4))) return STEM_ERR_ARG;
  if (attend && (!a->out || !aligned(a->out, 16) || !aligned(a->lse, 4))) return STEM_ERR_ARG;
  if (!attend) return STEM_OK;  // (the selection keeps everything on chip)
  if (a->workspace == nullptr || !aligned(a->workspace, kAlign) ||
      a->workspace_bytes < workspace(a->cache, a->R, a->Hq, a->kcap))
    return STEM_ERR_WORKSPACE;
  return STEM_OK;
}

int run_decode(const stem_decode_args_t* a, bool select, bool attend, cudaStream_t st) {
  int rc = check_decode(a, select, attend);
  if (rc != STEM_OK) return rc == 1 ? STEM_OK : rc;
  auto* ws = static_cast<unsigned char*>(a->workspace);
  const KvCache c = device_cache(a->cache);
  const DecodeRows r{a->q,    a->R,       a->Hq,      a->rows,  a->lens,
                     a->kcap, a->sel_idx, a->sel_cnt, a->status};
  const bool share = a->method->share == STEM_SHARE_GROUP;
  if ((rc = clear_status(a->status, st)) != STEM_OK) return rc;
  if (select) {
    SelMetric m;
    m.additive = a->method->metric == STEM_METRIC_ADDITIVE;
    m.beta = a->method->beta;
    m.clamp = a->method->clamp != 0;
    m.group = share;
    DecodeLists lists;  // with the attention to follow, the selection leaves its lists
    if (attend) lists = decode_lists(c, a->cache->format, a->cache->D, r, share, ws);
    rc = cuda_err(launch_decode_select(c, a->cache->D, r, a->budget, m, lists, st));
    if (rc != STEM_OK) return rc;
  }
  if (!attend) return STEM_OK;
  return cuda_err(launch_decode_attn(c, a->cache->format, a->cache->D, r, share, select, a->out,
                                     a->lse, ws, st));
}

}  // namespace
}  // namespace stem

using namespace stem;

extern "C" {

size_t stem_cache_page_bytes(int D, int block, int format) {
  if (check_format(D, block, format) != STEM_OK) return 0;
  return static_cast<size_t>(kv_record_bytes(kv_tile_bytes(format, D), block));
}

int stem_cache_append(const stem_cache_t* c, const void* k, const void* v, int dtype, int T,
                      const int64_t* strides, const int32_t* pos, const int32_t* count,
                      int32_t* status, void* stream) {
  return cache_rows(true, c, const_cast<void*>(k), const_cast<void*>(v), dtype, T, strides, pos,
                    count, status, static_cast<cudaStream_t>(stream));
}

int stem_cache_read(const stem_cache_t* c, void* k, void* v, int dtype, int T,
                    const int64_t* strides, const int32_t* pos, const int32_t* count,
                    int32_t* status, void* stream) {
  return cache_rows(false, c, k, v, dtype, T, strides, pos, count, status,
                    static_cast<cudaStream_t>(stream));
}

size_t stem_decode_workspace_size(const stem_cache_t* c, int R, int Hq, int kcap) {
  if (check_shape(c, R, Hq, kcap) != STEM_OK || R == 0) return 0;
  return workspace(c, R, Hq, kcap);
}

int stem_decode_select(const stem_decode_args_t* a, void* stream) {
  return run_decode(a, true, false, static_cast<cudaStream_t>(stream));
}

int stem_decode_attn(const stem_decode_args_t* a, void* stream) {
  return run_decode(a, false, true, static_cast<cudaStream_t>(stream));
}

int stem_decode(const stem_decode_args_t* a, void* stream) {
  return run_decode(a, true, true, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
