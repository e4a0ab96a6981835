// Block selection for single query tokens (stem_decode_select): the token's scores against the
// cached blocks' summaries, the metric, and the k(i) blocks it keeps.
//
//   s_hj = q_h . kbar_j / sqrt(D) over the blocks j < i before the diagonal block i (all full),
//   ranked by s + ln n or s + beta e, per head or summed over a kv head's query heads.
//
// Everything that decides between two blocks is held in double precision: a row's k-th and
// (k+1)-th blocks among a thousand can be closer than a float32 dot product is accurate, and the
// choice is meant to be the definition's. The device has one double FMA for two float32 ones, so
// this costs less than reading kbar: 2 G D flops a block and kv head against 4 D bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "decode_rows.cuh"

namespace stem {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kScoreWarps = 8;
constexpr int kScoreBlocks = 32;  // blocks a CTA scores
constexpr int kPickThreads = 256;
constexpr int kHeads = 4;  // query heads a warp scores at once

// ------------------------------------------------------------------ scores

// One warp per cached block: lane l holds channels (D/32) l .. of kbar and of kHeads queries; the
// heads' partial sums are folded so that five shuffle steps reduce all of them.
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(KvCache c, DecodeRows r,
                                                                 double* scores) {
  constexpr int CH = D / 32;
  const int row = blockIdx.z, kv = blockIdx.y, G = r.Hq / c.Hkv;
  int seq, len;
  decode_row(c, r, row, seq, len);
  const int last = (len + c.block - 1) / c.block - 1;
  const int j0 = blockIdx.x * kScoreBlocks, j1 = min(j0 + kScoreBlocks, last);
  if (j0 >= j1) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const double scale = 1.0 / sqrt(static_cast<double>(D));
  for (int h0 = 0; h0 < G; h0 += kHeads) {
    double q[kHeads][CH];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      const bool on = h0 + h < G;
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(r.q) +
                               (static_cast<int64_t>(row) * r.Hq + kv * G + (on ? h0 + h : 0)) * D +
                               lane * CH;
#pragma unroll
      for (int e = 0; e < CH; ++e) q[h][e] = on ? static_cast<double>(__bfloat162float(p[e])) : 0.0;
    }
    for (int j = j0 + warp; j < j1; j += kScoreWarps) {
      const int page = kv_page(c, seq, j, r.status);
      double s[kHeads];
      float k[CH];
      if (page >= 0) {
        const float* kb = c.kbar + (static_cast<int64_t>(page) * c.Hkv + kv) * D + lane * CH;
        if constexpr (CH == 4) {
          const float4 x = *reinterpret_cast<const float4*>(kb);
          k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(kb);
          k[0] = x.x, k[1] = x.y;
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          s[h] = 0.0;
#pragma unroll
          for (int e = 0; e < CH; ++e) s[h] = fma(q[h][e], static_cast<double>(k[e]), s[h]);
        }
      } else {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) s[h] = -INFINITY;
      }
      // fold: after the first two steps lane l holds head (l & 1) * 2 + (l >> 1 & 1)
      const bool up1 = lane & 1, up2 = lane & 2;
      double a0 = up1 ? s[2] : s[0], a1 = up1 ? s[3] : s[1];
      a0 += __shfl_xor_sync(kFull, up1 ? s[0] : s[2], 1);
      a1 += __shfl_xor_sync(kFull, up1 ? s[1] : s[3], 1);
      double t = up2 ? a1 : a0;
      t += __shfl_xor_sync(kFull, up2 ? a0 : a1, 2);
#pragma unroll
      for (int o = 4; o < 32; o *= 2) t += __shfl_xor_sync(kFull, t, o);
      const int h = (lane & 1) * 2 + (lane >> 1 & 1);
      if (lane < kHeads && h0 + h < G)
        scores[(static_cast<int64_t>(row) * r.Hq + kv * G + h0 + h) * c.max_blocks + j] = t * scale;
    }
  }
}

// ------------------------------------------------------------------ selection

// Order-preserving map of a double to an unsigned integer; NaN ranks with -infinity, -0 with +0.
__device__ __forceinline__ uint64_t rank_of(double x) {
  x = isnan(x) ? -INFINITY : x + 0.0;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
  return b >> 63 ? ~b : b | 1ull << 63;
}

// What a block's V magnitude adds to its key.
__device__ __forceinline__ double magnitude(const SelMetric& m, float n) {
  if (!m.additive) return log(static_cast<double>(n));
  if (m.beta == 0.f) return 0.0;
  const double e = 2.0 * log(static_cast<double>(n));
  return static_cast<double>(m.beta) * (m.clamp && e < 0.0 ? 0.0 : e);
}

__device__ __forceinline__ double block_max(double x, double* buf) {
  for (int o = 16; o; o /= 2) x = fmax(x, __shfl_xor_sync(kFull, x, o));
  __syncthreads();
  if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = x;
  __syncthreads();
  x = buf[0];
  for (int n = 1; n < kPickThreads / 32; ++n) x = fmax(x, buf[n]);
  return x;
}
__device__ __forceinline__ double block_sum(double x, double* buf) {
  for (int o = 16; o; o /= 2) x += __shfl_xor_sync(kFull, x, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = x;
  __syncthreads();
  x = buf[0];
  for (int n = 1; n < kPickThreads / 32; ++n) x += buf[n];
  return x;
}
// Exclusive prefix sum over the CTA's threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* buf) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t s = x;
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t y = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = s;
  __syncthreads();
  uint32_t before = 0;
  for (int n = 0; n < warp; ++n) before += buf[n];
  return before + s - x;
}

// One CTA per (row, list): keys of the candidates 1 .. i - 1 in shared memory, the k - 2 best by a
// radix select from the first digit in which the keys differ, then the list in ascending order.
__global__ void __launch_bounds__(kPickThreads) pick_kernel(KvCache c, DecodeRows r,
                                                            const int32_t* budget, SelMetric m,
                                                            const double* scores) {
  extern __shared__ uint64_t key[];  // max_blocks
  __shared__ uint32_t hist[256];
  __shared__ uint32_t wbuf[kPickThreads / 32];
  __shared__ double dbuf[kPickThreads / 32];
  __shared__ uint64_t s_lo, s_hi;
  __shared__ uint32_t s_bin, s_need, s_cnt;
  const int row = blockIdx.y, tid = threadIdx.x, G = r.Hq / c.Hkv;
  const int per = m.group ? G : 1;  // heads that get this list
  const int head = blockIdx.x * per, kv = head / G;
  int seq, len;
  decode_row(c, r, row, seq, len);
  const int last = (len + c.block - 1) / c.block - 1;
  int k = 0;
  if (last >= 0) {
    k = budget[last];
    const int lo = min(last + 1, 2);
    if (k < lo || k > last + 1 || k > r.kcap) {
      if (r.status && tid == 0) *r.status = STEM_ERR_ARG;
      k = min(max(k, lo), min(last + 1, r.kcap));
    }
  }
  int32_t* out = r.sel_idx + (static_cast<int64_t>(row) * r.Hq + head) * r.kcap;
  const int want = max(min(k, last + 1) - 2, 0);  // beside the sink and the diagonal block
  const int ncand = max(last - 1, 0);
  const bool all = want >= ncand;
  uint64_t cut = 0;  // keys of at least cut (shifted) are in, but for ties at the cut
  int shift = 0;
  uint32_t ties = 0;  // how many of those equal to the cut
  if (last > 1 && !all && want > 0) {
    const double* s = scores + (static_cast<int64_t>(row) * r.Hq + head) * c.max_blocks;
    double lse[8];
    const bool product_group = m.group && !m.additive && G > 1;
    uint64_t lo = ~0ull, hi = 0;
    // the group's product metric needs each head's softmax denominator (8 heads at a time)
    double* acc = reinterpret_cast<double*>(key);
    if (product_group) {
      for (int j = tid; j < last; j += kPickThreads) acc[j] = -INFINITY;
      for (int h0 = 0; h0 < G; h0 += 8) {
        const int nh = min(8, G - h0);
        for (int h = 0; h < nh; ++h) {
          const double* sh = s + static_cast<int64_t>(h0 + h) * c.max_blocks;
          double top = -INFINITY, sum = 0.0;
          for (int j = tid; j < last; j += kPickThreads) top = fmax(top, sh[j]);
          top = block_max(top, dbuf);
          if (!(top > -INFINITY)) top = 0.0;
          for (int j = tid; j < last; j += kPickThreads) sum += exp(sh[j] - top);
          lse[h] = top + log(block_sum(sum, dbuf));
        }
        for (int j = tid; j < last; j += kPickThreads) {
          double top = acc[j];
          for (int h = 0; h < nh; ++h)
            top = fmax(top, s[static_cast<int64_t>(h0 + h) * c.max_blocks + j] - lse[h]);
          double sum = 0.0;
          if (top > -INFINITY) {
            sum = exp(acc[j] - top);
            for (int h = 0; h < nh; ++h)
              sum += exp(s[static_cast<int64_t>(h0 + h) * c.max_blocks + j] - lse[h] - top);
            acc[j] = top + log(sum);
          }
        }
      }
    }
    for (int j = tid; j < last; j += kPickThreads) {  // (as above: a block stays with its thread)
      if (j == 0) continue;
      const int page = kv_page(c, seq, j, r.status);
      double x = -INFINITY;
      if (page >= 0) {
        const double w =
            magnitude(m, c.vnorm[static_cast<int64_t>(page) * c.Hkv + kv]);
        if (product_group) {
          x = acc[j] + w;
        } else {
          x = 0.0;
          for (int h = 0; h < per; ++h) x += s[static_cast<int64_t>(h) * c.max_blocks + j];
          x += m.additive ? per * w : w;
        }
      }
      const uint64_t u = rank_of(x);
      key[j] = u;
      lo = min(lo, u);
      hi = max(hi, u);
    }
    if (tid == 0) s_lo = ~0ull, s_hi = 0;
    __syncthreads();
    for (int o = 16; o; o /= 2) {
      lo = min(lo, __shfl_xor_sync(kFull, lo, o));
      hi = max(hi, __shfl_xor_sync(kFull, hi, o));
    }
    if (tid % 32 == 0) {
      atomicMin(reinterpret_cast<unsigned long long*>(&s_lo), lo);
      atomicMax(reinterpret_cast<unsigned long long*>(&s_hi), hi);
    }
    __syncthreads();
    lo = s_lo, hi = s_hi;
    if (lo == hi) {
      cut = hi;
      ties = want;
    } else {
      // digits of 8 bits from the first differing bit down
      int top = 64 - __clzll(lo ^ hi);  // bits [0, top) differ
      uint64_t prefix = top == 64 ? 0 : hi >> top;
      uint32_t need = want;
      for (;;) {
        const int bits = min(8, top);
        shift = top - bits;
        __syncthreads();
        hist[tid] = 0;
        __syncthreads();
        for (int j = 1 + tid; j < last; j += kPickThreads) {
          const uint64_t u = key[j];
          if ((top == 64 ? 0 : u >> top) == prefix)
            atomicAdd(&hist[u >> shift & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        // thread t owns bin 255 - t: keys in higher bins come before it
        const uint32_t n = hist[255 - tid];
        const uint32_t before = block_scan(n, wbuf);
        if (before < need && before + n >= need) {
          s_bin = 255 - tid;
          s_need = need - before;
          s_cnt = n;
        }
        __syncthreads();
        prefix = prefix << bits | s_bin;
        need = s_need;
        top = shift;
        if (s_cnt == need || top == 0) break;
      }
      cut = prefix;
      ties = need;
    }
  }
  // ascending output: thread t owns a run of blocks
  const int run = (last + 1 + kPickThreads - 1) / kPickThreads;
  const int b0 = min(tid * run, last + 1), b1 = min(b0 + run, last + 1);
  uint32_t over = 0, equal = 0;
  for (int j = b0; j < b1; ++j) {
    if (j == 0 || j == last || all) {
      ++over;
    } else if (want > 0) {
      const uint64_t u = key[j] >> shift;
      over += u > cut;
      equal += u == cut;
    }
  }
  const uint32_t before = block_scan(over << 16 | equal, wbuf);
  uint32_t eq = before & 0xffffu;
  uint32_t at = (before >> 16) + min(eq, ties);
  for (int j = b0; j < b1; ++j) {
    bool in = j == 0 || j == last || all;
    if (!in && want > 0) {
      const uint64_t u = key[j] >> shift;
      in = u > cut;
      if (u == cut) in = eq++ < ties;
    }
    if (in) {
      if (at < static_cast<uint32_t>(r.kcap))
        for (int h = 0; h < per; ++h) out[static_cast<int64_t>(h) * r.kcap + at] = j;
      ++at;
    }
  }
  const int kept = min(want + min(last + 1, 2), r.kcap);
  for (int n = kept + tid; n < r.kcap; n += kPickThreads)
    for (int h = 0; h < per; ++h) out[static_cast<int64_t>(h) * r.kcap + n] = -1;
  if (tid < per) r.sel_cnt[static_cast<int64_t>(row) * r.Hq + head + tid] = kept;
}

}  // namespace

cudaError_t launch_decode_select(const KvCache& c, int D, const DecodeRows& r,
                                 const int32_t* budget, SelMetric metric, double* scores,
                                 cudaStream_t st) {
  const dim3 grid((c.max_blocks + kScoreBlocks - 1) / kScoreBlocks, c.Hkv, r.R);
  if (D == 128)
    score_kernel<128><<<grid, kScoreWarps * 32, 0, st>>>(c, r, scores);
  else
    score_kernel<64><<<grid, kScoreWarps * 32, 0, st>>>(c, r, scores);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 pgrid(metric.group ? c.Hkv : r.Hq, r.R);
  pick_kernel<<<pgrid, kPickThreads, c.max_blocks * sizeof(uint64_t), st>>>(c, r, budget, metric,
                                                                            scores);
  return cudaGetLastError();
}

}  // namespace stem
