// Block selection for single query tokens (stem_decode_select): the token's scores against the
// cached blocks' summaries, the metric, and the k(i) blocks it keeps.
//
//   s_hj = q_h . kbar_j / sqrt(D) over the blocks j < i before the diagonal block i (all full),
//   ranked by s + ln n or s + beta e, per head or summed over a kv head's query heads.
//
// Everything that decides between two blocks is held in double precision: a row's k-th and
// (k+1)-th blocks among a thousand can be closer than a float32 dot product is accurate, and the
// choice is meant to be the definition's. It is 2 G D flops a block and kv head against 4 D bytes of
// kbar; a first pass in float32 that left double precision to the blocks near the cut was slower
// (13.0 against 12.3 us for one row of 128K, 39 against 33 for 32 ragged rows of up to 64K).
//
// One cluster of up to 8 CTAs per (row, kv head), so that scores never leave shared memory and a
// single launch does it all: each CTA scores a run of blocks for 8 heads at a time on the
// double-precision MMA (its operands need no shared memory and no reduction between lanes), the
// heads' softmax sums and then the keys are exchanged through distributed shared memory, and each
// list is picked by one CTA of the cluster.
//
// Measured (B200, device time in a graph): one row at the end of 128K tokens (32 heads on 8) 12.4 us,
// where reading kbar takes 0.65; 32 ragged rows of up to 64K (28 heads on 4, blocks of 64) 33 us of
// 5.7. Neither is near the floor: what is left is a chain of exchanges and exact ranking, not bytes.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_launch.h"
#include "decode_rows.cuh"

namespace cg = cooperative_groups;

namespace stem {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = kDecodeHeads;  // heads of a pass
constexpr int kMaxCluster = 8;
constexpr int kSlice = 64;      // a cluster grows to fill the device, but to no fewer blocks a CTA
constexpr int kMaxSlice = 512;  // what a CTA's shared memory holds
static_assert(kMaxCluster * kMaxSlice >= STEM_MAX_NB, "a cluster holds the longest context");

// What a block's V magnitude adds to its key.
__device__ __forceinline__ double magnitude(const SelMetric& m, float n) {
  if (!m.additive) return log(static_cast<double>(n));
  if (m.beta == 0.f) return 0.0;
  const double e = 2.0 * log(static_cast<double>(n));
  return static_cast<double>(m.beta) * (m.clamp && e < 0.0 ? 0.0 : e);
}

// Keys as they are compared: NaN ranks with -infinity, -0 with +0.
__device__ __forceinline__ double as_key(double x) { return isnan(x) ? -INFINITY : x + 0.0; }
// Order-preserving map of a key to an unsigned integer.
__device__ __forceinline__ uint64_t rank_of(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
  return b >> 63 ? ~b : b | 1ull << 63;
}

// The threads that pick one list: a warp (of 8 that pick 8 lists at once) or the whole CTA.
template <int T>
struct Team {
  static constexpr int kBuckets = T == 32 ? 256 : 1024;  // of the first cut of the keys
  static constexpr int kTied = T == 32 ? 128 : 256;      // keys ranked one by one at most
  double lo[T / 32], hi[T / 32];
  double tied_key[kTied];
  uint32_t hist[kBuckets];
  uint32_t kept[STEM_MAX_NB / 32 + 1];  // bit j: block j is kept
  uint32_t scan[T / 32];
  uint32_t cut, need, found, tied;
  uint16_t tied_at[kTied];

  static __device__ __forceinline__ int tid() { return threadIdx.x % T; }
  static __device__ __forceinline__ void sync() {
    if (T == 32)
      __syncwarp();
    else
      __syncthreads();
  }
  // Exclusive prefix sum over the team's threads.
  __device__ __forceinline__ uint32_t prefix(uint32_t x) {
    const int lane = threadIdx.x % 32, warp = tid() / 32;
    uint32_t s = x;
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    if (T == 32) return s - x;
    sync();
    if (lane == 31) scan[warp] = s;
    sync();
    uint32_t before = 0;
    for (int n = 0; n < warp; ++n) before += scan[n];
    return before + s - x;
  }
  __device__ __forceinline__ uint32_t sum(uint32_t x) {
    x = __reduce_add_sync(kFull, x);
    if (T == 32) return x;
    sync();
    if (threadIdx.x % 32 == 0) scan[tid() / 32] = x;
    sync();
    x = 0;
    for (int n = 0; n < T / 32; ++n) x += scan[n];
    return x;
  }
};

// The `want` best of the candidates 1 .. last - 1 by key, ties to the lower block, into s.kept
// (beside the sink 0 and the diagonal block). One pass cuts the keys into equal intervals between
// the smallest and the largest; the few of the interval at the cut are ranked one by one.
template <int T>
__device__ void pick(const double* key, int last, int want, Team<T>& s) {
  const int tid = s.tid();
  const int words = last / 32 + 1;
  const bool all = want >= last - 1;  // (every block is kept)
  for (int w = tid; w < words; w += T) {
    uint32_t x = all ? kFull : w == 0 ? 1u : 0u;
    if (w == last / 32) {
      const int r = last % 32;
      x = (x | 1u << r) & (r == 31 ? kFull : (2u << r) - 1u);
    }
    s.kept[w] = x;
  }
  if (all || want <= 0) {
    s.sync();
    return;
  }
  // Few candidates: each counts those that come before it.
  constexpr int kFew = T == 32 ? 64 : 128;
  if (last <= kFew) {
    s.sync();
    for (int j = 1 + tid; j < last; j += T) {
      const double x = key[j];
      int before = 0;
#pragma unroll 4
      for (int n = 1; n < last; ++n) {
        const double y = key[n];
        before += y > x || (y == x && n < j);
      }
      if (before < want) atomicOr(&s.kept[j / 32], 1u << (j % 32));
    }
    s.sync();
    return;
  }
  double lo = INFINITY, hi = -INFINITY;  // of the finite keys
  for (int j = 1 + tid; j < last; j += T) {
    const double x = key[j];
    if (!isinf(x)) {
      lo = fmin(lo, x);
      hi = fmax(hi, x);
    }
  }
  for (int o = 16; o; o /= 2) {
    lo = fmin(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmax(hi, __shfl_xor_sync(kFull, hi, o));
  }
  for (int b = tid; b < s.kBuckets; b += T) s.hist[b] = 0;
  if (tid % 32 == 0) s.lo[tid / 32] = lo, s.hi[tid / 32] = hi;
  if (tid == 0) s.tied = 0;
  s.sync();
  for (int w = 0; w < T / 32; ++w) lo = fmin(lo, s.lo[w]), hi = fmax(hi, s.hi[w]);
  // (a product that rounds keeps the order: a larger key never falls into a lower interval)
  // (finite, so that no product with it is NaN, which is no bucket)
  const double scale = hi > lo ? fmin((s.kBuckets - 1) / (hi - lo), 1e300) : 0.0;
  auto bucket = [&](double x) -> int {
    if (x == -INFINITY) return 0;
    if (x == INFINITY) return s.kBuckets - 1;
    return min(static_cast<int>((x - lo) * scale), s.kBuckets - 1);
  };
  for (int j = 1 + tid; j < last; j += T) atomicAdd(&s.hist[bucket(key[j])], 1u);
  s.sync();
  {
    constexpr int kRun = Team<T>::kBuckets / T;  // thread t owns a run of buckets from the top down
    uint32_t n = 0;
    for (int i = 0; i < kRun; ++i) n += s.hist[s.kBuckets - 1 - (tid * kRun + i)];
    uint32_t before = s.prefix(n);
    for (int i = 0; i < kRun; ++i) {
      const int b = s.kBuckets - 1 - (tid * kRun + i);
      const uint32_t c = s.hist[b];
      if (before < static_cast<uint32_t>(want) && before + c >= static_cast<uint32_t>(want)) {
        s.cut = b;
        s.need = want - before;
        s.found = c;
      }
      before += c;
    }
  }
  s.sync();
  const int cut = s.cut;
  const uint32_t need = s.need, found = s.found;
  const bool few = found <= s.kTied;
  for (int j = 1 + tid; j < last; j += T) {
    const double x = key[j];
    const int b = bucket(x);
    if (b > cut || (b == cut && found == need)) {
      atomicOr(&s.kept[j / 32], 1u << (j % 32));
    } else if (b == cut && few) {
      const uint32_t n = atomicAdd(&s.tied, 1u);
      s.tied_key[n] = x;
      s.tied_at[n] = static_cast<uint16_t>(j);
    }
  }
  s.sync();
  if (found == need) return;
  if (few) {
    for (uint32_t i = tid; i < found; i += T) {
      const double x = s.tied_key[i];
      const int j = s.tied_at[i];
      uint32_t rank = 0;
      for (uint32_t n = 0; n < found; ++n) {
        const double y = s.tied_key[n];
        rank += y > x || (y == x && s.tied_at[n] < j);
      }
      if (rank < need) atomicOr(&s.kept[j / 32], 1u << (j % 32));
    }
    s.sync();
    return;
  }
  // Many keys in one interval (equal blocks, or a few far outliers): their need-th largest value
  // bit by bit, then the lowest blocks of those equal to it.
  uint64_t t = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t c = t | 1ull << bit;
    uint32_t n = 0;
    for (int j = 1 + tid; j < last; j += T) n += bucket(key[j]) == cut && rank_of(key[j]) >= c;
    if (s.sum(n) >= need) t = c;
  }
  const int run = (last + T - 1) / T;
  const int j0 = max(min(tid * run, last), 1), j1 = min(tid * run + run, last);
  uint32_t above = 0, equal = 0;
  for (int j = j0; j < j1; ++j) {
    if (bucket(key[j]) != cut) continue;
    const uint64_t u = rank_of(key[j]);
    above += u > t;
    equal += u == t;
  }
  const uint32_t ties = need - s.sum(above);
  uint32_t at = s.prefix(equal);
  for (int j = j0; j < j1; ++j) {
    if (bucket(key[j]) != cut) continue;
    const uint64_t u = rank_of(key[j]);
    if (u > t || (u == t && at++ < ties)) atomicOr(&s.kept[j / 32], 1u << (j % 32));
  }
  s.sync();
}

// Writes the blocks of s.kept in ascending order as the lists of `per` heads, -1 behind them.
template <int T, typename F>
__device__ void write_list(Team<T>& s, int last, int kcap, int per, int32_t* idx, int32_t* cnt,
                           F each) {
  const int tid = s.tid(), halves = last < 0 ? 0 : (last / 32 + 1) * 2;
  uint32_t total = 0;
  for (int h0 = 0; h0 < halves; h0 += T) {  // thread t: 16 blocks
    const int h = h0 + tid;
    uint32_t bits = h < halves ? s.kept[h / 2] >> (16 * (h % 2)) & 0xffffu : 0u;
    const uint32_t n = __popc(bits);
    uint32_t at = total + s.prefix(n);
    while (bits) {
      const int j = h * 16 + __ffs(bits) - 1;
      bits &= bits - 1;
      if (at < static_cast<uint32_t>(kcap)) {
        for (int p = 0; p < per; ++p) idx[static_cast<int64_t>(p) * kcap + at] = j;
        each(at, j);
      }
      ++at;
    }
    total += s.sum(n);
  }
  total = min(total, static_cast<uint32_t>(kcap));
  for (int e = total + tid; e < kcap; e += T)
    for (int p = 0; p < per; ++p) idx[static_cast<int64_t>(p) * kcap + e] = -1;
  for (int p = tid; p < per; p += T) cnt[p] = static_cast<int32_t>(total);
  s.sync();
}

union Teams {
  Team<kThreads> cta;
  Team<32> warp[kWarps];
};

struct Sums {
  double lse[kHeads];               // softmax denominators of the pass's heads (ln)
  double top[kMaxCluster][kHeads];  // each CTA's maximum and sum, in every CTA
  double sum[kMaxCluster][kHeads];
  uint32_t scan[kWarps];
};

// D += A B with A 16 x 4 (rows g and g + 8), B 4 x 8.
__device__ __forceinline__ void mma_f64(double (&d)[4], double a0, double a1, double b) {
  asm volatile(
      "mma.sync.aligned.m16n8k4.row.col.f64.f64.f64.f64 {%0,%1,%2,%3}, {%4,%5}, {%6}, "
      "{%0,%1,%2,%3};"
      : "+d"(d[0]), "+d"(d[1]), "+d"(d[2]), "+d"(d[3])
      : "d"(a0), "d"(a1), "d"(b));
}

struct Args {
  KvCache c;
  DecodeRows r;
  const int32_t* budget;
  SelMetric m;
  DecodeLists lists;  // of the attention; list NULL: not wanted
  int slice;          // blocks of a CTA
};

// Lists that a CTA of a cluster picks in a pass, with keys of their own.
__host__ __device__ constexpr int lists_of(bool group, int csize) {
  return csize == 1 ? 0 : group ? 1 : (kHeads + csize - 1) / csize;
}

// Dynamic shared memory of a launch (in the order that the kernel lays it out), and the most that any
// launch takes: a cluster is no smaller than its slices of kMaxSlice blocks make it.
constexpr size_t smem_bytes(int max_blocks, int csize, bool group) {
  const size_t slice = (max_blocks + csize - 1) / csize;
  return sizeof(double) * ((kHeads + 2) * slice +
                           static_cast<size_t>(lists_of(group, csize)) * max_blocks) +
         (static_cast<size_t>(max_blocks) + 7) / 4 * 4;
}
constexpr size_t kMaxSmem = smem_bytes(STEM_MAX_NB, kMaxCluster, false);
constexpr bool below_most(int csize) {
  return csize > kMaxCluster ||
         (smem_bytes(std::min(csize * kMaxSlice, STEM_MAX_NB), csize, false) <= kMaxSmem &&
          smem_bytes(std::min(csize * kMaxSlice, STEM_MAX_NB), csize, true) <= kMaxSmem &&
          below_most(2 * csize));
}
static_assert(below_most(1), "kMaxSmem is the most");

// CTAS: CTAs of an SM that the registers are shared out for, 2 or 4 (see launch_decode_select).
template <int D, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) select_kernel(const Args a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Sums s;
  __shared__ Teams team;
  cg::cluster_group cluster = cg::this_cluster();
  const int csize = gridDim.x, rank = blockIdx.x;  // (a cluster is a row of the grid)
  const int row = blockIdx.z, kv = blockIdx.y, G = a.r.Hq / a.c.Hkv;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // shared memory: scores of this CTA's blocks | their V terms | group sums |
  // keys of the lists that this CTA picks (of a cluster of one: the scores' place) | (first CTA)
  // head bits of each block
  double* score = reinterpret_cast<double*>(smem);
  double* w_s = score + kHeads * a.slice;
  double* acc = w_s + a.slice;
  double* key = csize == 1 ? score : acc + a.slice;
  uint32_t* mask = reinterpret_cast<uint32_t*>(acc + a.slice +
                                               lists_of(a.m.group, csize) * a.c.max_blocks);

  // Another CTA's shared memory may be written only once that CTA runs, which its arrival here tells.
  // The wait for it is behind the first scores, so that it hides behind the loads of a CTA that has
  // blocks (one without any comes there at once). The barrier's phases that follow start after it.
  cluster.barrier_arrive();
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  if (rank == 0 && a.lists.list)
    for (int n = tid; n < a.lists.tiles_h; n += kThreads)
      a.lists.arrived[(static_cast<int64_t>(row) * a.c.Hkv + kv) * a.lists.tiles_h + n] = 0;
  int seq, len;
  decode_row(a.c, a.r, row, seq, len);
  const int last = (len + a.c.block - 1) / a.c.block - 1;
  int k = 0;
  if (last >= 0) {
    k = a.budget[last];
    const int lo = min(last + 1, 2);
    if (k < lo || k > last + 1 || k > a.r.kcap) {
      if (a.r.status && tid == 0) *a.r.status = STEM_ERR_ARG;
      k = min(max(k, lo), min(last + 1, a.r.kcap));
    }
  }
  const int want = k - 2;                              // beside the sink and the diagonal block
  const bool scored = want > 0 && want < last - 1;     // (else the scores decide nothing)
  const bool product_group = a.m.group && !a.m.additive && G > 1;
  const int j0 = min(rank * a.slice, max(last, 0)), j1 = min(j0 + a.slice, max(last, 0));
  const int32_t* table = a.c.table + static_cast<int64_t>(seq) * a.c.max_blocks;
  const double scale = 1.0 / sqrt(static_cast<double>(D));
  const int key_row = csize == 1 ? a.slice : a.c.max_blocks;

  if (scored) {
    for (int j = j0 + tid; j < j1; j += kThreads) {
      const int page = kv_page(a.c, seq, j, a.r.status);
      w_s[j - j0] =
          page < 0 ? NAN : magnitude(a.m, a.c.vnorm[static_cast<int64_t>(page) * a.c.Hkv + kv]);
      acc[j - j0] = a.m.additive || G == 1 ? 0.0 : -INFINITY;
    }
  }
  for (int h0 = 0; h0 < G; h0 += kHeads) {
    const int nh = min(kHeads, G - h0);
    const int64_t head0 = static_cast<int64_t>(row) * a.r.Hq + kv * G + h0;
    if (scored) {
      // ---- scores on the double-precision MMA: rows are blocks, columns heads. Lane 4g + t holds
      // block g's (and g + 8's) and head g's channels 16i + 4t + e, which are column t of step (i, e).
      const int g = lane / 4, t = lane % 4;
      double q[D / 16][4];
      const uint2* qp = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.r.q) +
                                                       (head0 + (g < nh ? g : 0)) * D + 4 * t);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint2 u = g < nh ? qp[i * 4] : make_uint2(0, 0);
        q[i][0] = static_cast<double>(__uint_as_float(u.x << 16)) * scale;
        q[i][1] = static_cast<double>(__uint_as_float(u.x & 0xffff0000u)) * scale;
        q[i][2] = static_cast<double>(__uint_as_float(u.y << 16)) * scale;
        q[i][3] = static_cast<double>(__uint_as_float(u.y & 0xffff0000u)) * scale;
      }
      for (int b = j0 + warp * 16; b < j1; b += kWarps * 16) {
        const float4* p[2];
        bool there[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int j = b + g + 8 * y;
          const int page = j < j1 ? table[j] : -1;
          there[y] = page >= 0 && page < a.c.num_pages;
          p[y] = reinterpret_cast<const float4*>(
              a.c.kbar + (static_cast<int64_t>(there[y] ? page : 0) * a.c.Hkv + kv) * D + 4 * t);
        }
        double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int i0 = 0; i0 < D / 16; i0 += 4) {
          float4 x[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              x[i][y] = there[y] ? p[y][(i0 + i) * 4] : make_float4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f64(v, x[i][0].x, x[i][1].x, q[i0 + i][0]);
            mma_f64(v, x[i][0].y, x[i][1].y, q[i0 + i][1]);
            mma_f64(v, x[i][0].z, x[i][1].z, q[i0 + i][2]);
            mma_f64(v, x[i][0].w, x[i][1].w, q[i0 + i][3]);
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int j = b + g + 8 * y;
          if (j >= j1) continue;
          score[2 * t * a.slice + j - j0] = there[y] ? v[2 * y] : -INFINITY;
          score[(2 * t + 1) * a.slice + j - j0] = there[y] ? v[2 * y + 1] : -INFINITY;
        }
      }
    }
    if (h0 == 0) cluster.barrier_wait();  // (every CTA of the cluster runs)
    if (scored) {
      __syncthreads();
      if (product_group) {
        // ---- each head's softmax denominator: a warp per head, then over the cluster
        for (int h = warp; h < nh; h += kWarps) {
          const double* sh = score + h * a.slice;
          double top = -INFINITY, sum = 0.0;
          for (int n = lane; n < j1 - j0; n += 32) top = fmax(top, sh[n]);
          for (int o = 16; o; o /= 2) top = fmax(top, __shfl_xor_sync(kFull, top, o));
          const double base = top > -INFINITY ? top : 0.0;
          for (int n = lane; n < j1 - j0; n += 32) sum += exp(sh[n] - base);
          for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(kFull, sum, o);
          if (lane < csize) {
            Sums* to = cluster.map_shared_rank(&s, lane);
            to->top[rank][h] = top;
            to->sum[rank][h] = sum;
          }
        }
        cluster.sync();
        if (tid < nh) {
          double top = -INFINITY, sum = 0.0;
          for (int c = 0; c < csize; ++c) top = fmax(top, s.top[c][tid]);
          if (!(top > -INFINITY)) top = 0.0;
          for (int c = 0; c < csize; ++c) {
            // a CTA without a finite score (of a short row, say) has no part in it: its sum is 0 (or
            // NaN), and exp(-top) might be infinite (a choice of exponents, not a branch around exp,
            // which would run the CTAs' one after the other)
            const double base = s.top[c][tid] > -INFINITY ? s.top[c][tid] : top;
            sum += s.sum[c][tid] * exp(base - top);
          }
          s.lse[tid] = top + log(sum);
        }
        __syncthreads();
      }
      // ---- keys, or the group's sum so far
      if (a.m.group) {
        for (int n = tid; n < j1 - j0; n += kThreads) {
          double x = acc[n];
          if (product_group) {
            // ln of the probabilities' sum; relative to the largest where the plain sum would lose
            // digits to the range's end (and after the first 8 heads)
            double sum = 0.0;
            if (h0 == 0)
              for (int h = 0; h < nh; ++h) sum += exp(score[h * a.slice + n] - s.lse[h]);
            if (sum > 1e-280 || isnan(sum)) {
              x = log(sum);
            } else {
              double top = x;
              for (int h = 0; h < nh; ++h) top = fmax(top, score[h * a.slice + n] - s.lse[h]);
              if (top > -INFINITY) {
                sum = exp(x - top);
                for (int h = 0; h < nh; ++h) sum += exp(score[h * a.slice + n] - s.lse[h] - top);
                x = top + log(sum);
              }
            }
          } else {
            for (int h = 0; h < nh; ++h) x += score[h * a.slice + n];
          }
          acc[n] = x;
          // (in a cluster of one the key takes the place of the block's first score)
          if (h0 + nh == G)
            *cluster.map_shared_rank(key + j0 + n, 0) =
                as_key(x + (a.m.additive ? G * w_s[n] : w_s[n]));
        }
      } else {
        for (int n = tid; n < nh * a.slice; n += kThreads) {
          const int h = n / a.slice, e = n % a.slice;
          if (e >= j1 - j0) continue;
          *cluster.map_shared_rank(key + (h / csize) * key_row + j0 + e, h % csize) =
              as_key(score[n] + w_s[e]);
        }
      }
    }
    if (a.m.group && h0 + nh < G) {
      cluster.sync();  // (the next heads' sums go where these were read)
      continue;
    }
    if (!a.m.group && rank == 0 && a.lists.list)
      for (int w = tid; w < last / 4 + 1; w += kThreads) mask[w] = 0;
    if (scored || !a.m.group) cluster.sync();
    // ---- pick
    if (a.m.group) {  // one list for all heads: the first CTA's
      if (rank == 0) {
        Team<kThreads>& tm = team.cta;
        if (last >= 0) pick(key, last, want, tm);
        const int64_t li = static_cast<int64_t>(row) * a.c.Hkv + kv;
        Entry* list = a.lists.list ? a.lists.list + li * a.lists.most : nullptr;
        const int64_t head = static_cast<int64_t>(row) * a.r.Hq + kv * G;
        write_list(tm, last, a.r.kcap, G, a.r.sel_idx + head * a.r.kcap, a.r.sel_cnt + head,
                   [&](uint32_t at, int j) {
                     if (list) list[at] = entry_of(a.c, seq, j, 0xffu, a.r.status);
                   });
        if (list && tid == 0) a.lists.count[li] = max(min(k, a.r.kcap), 0);
      }
      continue;
    }
    // a list a head: spread over the cluster, and with four or more in a CTA over its warps
    uint32_t* mask0 = cluster.map_shared_rank(mask, 0);
    auto head_list = [&](auto& tm, int h) {
      if (last >= 0) pick(key + (h / csize) * key_row, last, want, tm);
      write_list(tm, last, a.r.kcap, 1, a.r.sel_idx + (head0 + h) * a.r.kcap,
                 a.r.sel_cnt + head0 + h, [&](uint32_t, int j) {
                   if (a.lists.list) atomicOr(&mask0[j / 4], 1u << (8 * (j % 4) + h));
                 });
    };
    if (csize <= 2) {
      const int h = rank + warp * csize;
      if (h < nh) head_list(team.warp[warp], h);
    } else {
      for (int h = rank; h < nh; h += csize) head_list(team.cta, h);
    }
    cluster.sync();
    if (rank == 0 && a.lists.list) {
      const int64_t item = (static_cast<int64_t>(row) * a.c.Hkv + kv) * a.lists.tiles_h + h0 / kHeads;
      write_union<kThreads>(a.c, a.lists, item, seq, last, nh, mask, s.scan, a.r.status);
    }
    __syncthreads();
  }
  cluster.sync();  // (no CTA leaves while another may still write to it)
}

}  // namespace

cudaError_t launch_decode_select(const KvCache& c, int D, const DecodeRows& r,
                                 const int32_t* budget, SelMetric metric, const DecodeLists& lists,
                                 cudaStream_t st) {
  // Clusters grow while the device has room for more CTAs and a CTA has blocks to share.
  const int64_t lists_all = static_cast<int64_t>(r.R) * c.Hkv;
  int csize = 1;
  while (csize < kMaxCluster &&
         (c.max_blocks > csize * kMaxSlice ||
          (lists_all * csize < sm_count() && c.max_blocks > csize * kSlice)))
    csize *= 2;
  const Args a{c, r, budget, metric, lists, (c.max_blocks + csize - 1) / csize};
  const size_t bytes = smem_bytes(c.max_blocks, csize, metric.group);
  // Where more CTAs are launched than run at once at 2 an SM, 4 of them with fewer registers each:
  // 64 rows of up to 16K with 32 heads on 8 take 15.8 us instead of 20.5 (lists of their own 13.7
  // instead of 17.5). Where all run at once the registers are worth more: 33.4 us instead of 36.5 for
  // 32 rows of up to 64K with 28 on 4, 12.3 instead of 12.7 for one of 128K.
  const bool many = lists_all * csize > 2 * sm_count();
  void (*kernel)(const Args) = D == 128 ? (many ? select_kernel<128, 4> : select_kernel<128, 2>)
                                        : (many ? select_kernel<64, 4> : select_kernel<64, 2>);
  // (the same value in every call: another thread's, between this and the launch, changes nothing)
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kMaxSmem));
  if (e != cudaSuccess) return e;
  return launch_after(kernel, dim3(csize, c.Hkv, r.R), kThreads, bytes, csize, st, a);
}

}  // namespace stem
