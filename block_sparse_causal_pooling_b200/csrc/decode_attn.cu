// Attention of single query tokens over the kept blocks of a paged cache (stem_decode_attn).
//
// For one row and kv head: z_th = q_h . K_t / sqrt(D) over the tokens t of the kept blocks,
// o_h = sum_t softmax_t(z_th) V_t. The K and V bytes are read once and each meets only the G query
// heads of its kv head (2 to 8 flops a byte at 16 bits), so HBM bounds the kernel and the tensor
// pipe has room to spare. It uses mma.sync.m16n8k16 with tokens (for V: channels) as the 16 rows
// and 8 query heads as the 8 columns: tcgen05's 128-row tiles would need the expanded codes in
// shared memory, four times the bytes of 4-bit codes, for 8 useful columns or rows.
//
// Codes of 4 and 8 bits go to the MMA without a conversion: a masked word holds a pair of fp16
// subnormals code * 2^-24 (times 16 for the upper nibble of a byte, undone in q or at the end).
//   K: sum_d q_d c_d over a 32-channel group is one short chain of MMAs; the group's scale multiplies
//      its result (4 FMA a tile and group). What the offset adds over all groups, sum_y s_ty off_yh with
//      off_yh = -offset * sum_d q_d, is one more MMA, of the scales. q is scaled by a power of two per
//      head so that its largest entry is in [2^14, 2^15): bf16's 8 significant bits survive in fp16.
//   V: the scale goes to the weight: a_th = p_th s_t f rounded once to fp16, with f a power of two
//      that follows the largest scale seen (like the running maximum of the softmax), so that none
//      overflows. sum_t a_th (c_td - off) = sum a c - off * sum a; the last sum comes from one more MMA
//      against a constant, so both sums see the same rounded a. A weight below fp16's normal range is
//      off by up to 2^-25, which the sum of a group's weights shows: where it is so small that n
//      tokens could be off by 2^-12 of it together (a group of channels, or the tokens that a head
//      looks at, far below the largest scale), the CTA goes over its entries again, first for the
//      largest p s of each head and group, then with an f for each. So whatever the scales are, the
//      weights are off by no more than 2^-11 of each and 2^-12 of their sum.
// The tensor pipe cuts the products of a chain at 2^-25 of the largest and takes a subnormal's
// exponent for -14 (measured), so a product keeps its bits down to 2^-15 code steps times the largest
// q (or weight) of the chain. bf16 entries of q above 2^-8 of the largest lose nothing; the value sums
// lose less than 2^-10 of the half step by which the code itself may be off.
// At 16 bits the operands are bf16 as stored and each weight is two bf16 numbers (2^-15 of it are lost):
// HBM bounds that kernel, so that its MMAs for V twice over cost little (32 ragged rows of per-head
// lists of up to 16K 102.6 us, 101.2 with one number, which lost 2^-8 of each weight).
//
// A warp streams whole tiles (16 tokens of K and V, contiguous in the page) through a ring of its own
// in shared memory with cp.async: no barrier between warps until the end. Softmax statistics and
// sums are float32. Warps, then CTAs of one (row, kv head), are joined by (max, sum, numerator).
//
// Measured (B200; 16 sequences, 32 heads on 8 kv heads of 128, every block; device time in a graph),
// at 4K, 8K, 16K and 32K tokens: 16 bits 56, 95, 176 and 334 us, 8 bits 40, 62, 108 and 196 us, 4 bits
// 34, 50, 81 and 145 us; at 32K 6.4, 5.8 and 4.2 TB/s (a copy reaches 6.47). A line through the four
// has a slope of 6.8, 6.4 and 4.8 TB/s and starts at 17 to 18 us. Few rows are bound by latency, long
// lists at 16 and 8 bits by HBM, at 4 bits by the instructions that unpack and scale.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "decode_launch.h"
#include "decode_rows.cuh"

namespace stem {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kHeadTile = kDecodeHeads;
// Steps of a CTA below which an item is not split further: two a warp. (A selection and its attention of
// one row of 16 blocks of 64 at 16 bits: 13.1 us with 8 steps a CTA, 13.3 with 16; one row over 52 blocks
// of 128 at 4 bits: 13.4 and 13.1.)
constexpr int kMinSteps = 8;
// Items in parts are joined by the CTA that brings the last part, which saves a launch, unless they
// have more parts than this on average: then by a kernel of their own, with a CTA for each head.
constexpr int kDirect = 16;
constexpr int kStaged = 128;  // list entries in shared memory at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A logit may exceed the running maximum by this much (in log2 units) before the accumulators are
// rescaled: weights stay below 2^4, and most steps need neither the warp's maximum nor a rescale.
constexpr float kSlack = 4.f;
// The V scales' power of two puts the largest scale in [2^8, 2^9) when it is set, and is set again
// when a scale exceeds 2^11 in its units: weights stay below 2^15, fp16's range. The narrower the
// slacks, the more often both are set again, and the fewer entries are gone over again. (Slacks of 2^5 and
// scales from 2^6: every block of 32 sequences of 64K at 8 bits, weights all on one token, 1310 us where
// these take 703 and weights on many 693. 2^3 and 2^10: 695, but 64 ragged rows of up to 32K 91.6
// instead of 90.6.)
constexpr int kScaleSet = 8, kScaleSlack = 2;
// A sum of weights that n tokens may be off by 2^-12 of, at 2^-25 each, is below n times this.
constexpr float kLeastSum = 0x1p-13f;

template <int FMT, int D>
struct Cfg {
  using L = Kv<FMT, D>;
  static constexpr bool Q = FMT != STEM_KV_BF16;
  static constexpr int TPS = Q ? 2 : 1;  // tiles a warp takes at once
  static constexpr int STAGES = 3;
  static constexpr int WARPS = 4, THREADS = 32 * WARPS;
  // CTAs an SM: as many as the rings allow at 8 and 16 bits; at 4 bits, as many as have the registers
  // that the kernel wants. More of them are no faster. (4 bits, 4 CTAs of 128 registers with some
  // spilled: 94 us for 64 ragged rows of up to 32K where 3 take 90, 27.1 for 8 of up to 64K where 3
  // take 24.1. 8 bits, 3 CTAs with rings of 2 steps: 43 us for 32 ragged rows of up to 16K, 57.4 for
  // every block of 4 of up to 64K, where 2 with rings of 3 take 32 and 55.1.)
  static constexpr int CTAS = FMT == STEM_KV_Q4 ? 3 : 2;
  static constexpr int STEP = kKvTile * TPS;  // tokens
  static constexpr int STEP_BYTES = TPS * L::TILE_BYTES;
  static constexpr int RING = STAGES * STEP_BYTES;  // a warp's
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first of a chain: D = A B.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8x8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// lo and hi as bf16 pairs that add up to them but for 2^-15 of each: their upper halves, and what is left
// with 2^-20 more. So no second part of a weight is 0 or below 0 beside a first that is not: the two
// times an infinite V value are infinite, not NaN.
__device__ __forceinline__ void two_parts(float lo, float hi, uint32_t& first, uint32_t& second) {
  first = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
  second = pack_bf16(fmaf(lo, 0x1p-20f, lo - low16(first)), fmaf(hi, 0x1p-20f, hi - high16(first)));
}

struct Args {
  KvCache c;
  DecodeRows r;
  bool share;
  DecodeLists lists;
  int items;  // a row, a kv head and up to 8 of its query heads each
  // A CTA has one part of one item: `chunk` entries, or a little less. With per_item CTAs for each item
  // the chunk is fixed; where they would not all run at once (per_item 0), it follows from the number
  // of entries that there are, so that about at_once CTAs have the work of all.
  int per_item, chunk, at_once;
  __nv_bfloat16* out;
  float* lse;
  // Parts of items, a slot for each CTA: [slot][8] statistics (max in log2 units, sum) and [slot][8][D]
  // numerators.
  float2* stat;
  float* part;
  bool direct;     // the CTA that brings an item's last part joins them
  int32_t* start;  // [items]: the item's first CTA; [items]: the chunk (where neither is fixed)
};

// ------------------------------------------------------------------ the lists

constexpr int kPlanThreads = 128;

// Turns the kept blocks of each (row, kv head) or item into a list of entries: the page of each
// block and the heads that keep it. One CTA per list. (After a selection of the same call the lists are
// there already.)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Args a) {
  extern __shared__ uint32_t mask[];  // per-head lists: a byte of head bits for each block
  __shared__ uint32_t wbuf[kPlanThreads / 32];
  const int tid = threadIdx.x, row = blockIdx.y, G = a.r.Hq / a.c.Hkv;
  const int64_t list = static_cast<int64_t>(row) * gridDim.x + blockIdx.x;
  Entry* out = a.lists.list + list * a.lists.most;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int here = a.share ? a.lists.tiles_h : 1;  // items of this list
  for (int n = tid; n < here; n += kPlanThreads) a.lists.arrived[list * here + n] = 0;
  int seq, len;
  decode_row(a.c, a.r, row, seq, len);
  const int last = (len + a.c.block - 1) / a.c.block - 1;
  if (last < 0) {
    if (tid == 0) a.lists.count[list] = 0;
    return;
  }
  if (a.share) {
    const int64_t head = static_cast<int64_t>(row) * a.r.Hq + blockIdx.x * G;
    const int cnt = a.r.sel_cnt[head];
    if ((cnt < 0 || cnt > a.r.kcap) && a.r.status) *a.r.status = STEM_ERR_ARG;
    const int n = max(min(cnt, a.r.kcap), 0);
    for (int e = tid; e < n; e += kPlanThreads) {
      const int j = a.r.sel_idx[head * a.r.kcap + e];
      if (j >= 0 && j <= last) {
        out[e] = entry_of(a.c, seq, j, 0xffu, a.r.status);
      } else {
        if (a.r.status) *a.r.status = STEM_ERR_ARG;
        out[e] = Entry{0, 0u};
      }
    }
    if (tid == 0) a.lists.count[list] = n;
    return;
  }
  // the union of the heads' lists, in block order
  const int kv = blockIdx.x / a.lists.tiles_h, h0 = blockIdx.x % a.lists.tiles_h * kHeadTile;
  const int nh = min(G - h0, kHeadTile);
  const int64_t head0 = static_cast<int64_t>(row) * a.r.Hq + kv * G + h0;
  for (int w = tid; w < last / 4 + 1; w += kPlanThreads) mask[w] = 0;
  __syncthreads();
  for (int n = tid; n < nh * a.r.kcap; n += kPlanThreads) {
    const int h = n / a.r.kcap, e = n % a.r.kcap;
    const int j = a.r.sel_idx[(head0 + h) * a.r.kcap + e];
    const int cnt = a.r.sel_cnt[head0 + h];
    if (e == 0 && (cnt < 0 || cnt > a.r.kcap) && a.r.status) *a.r.status = STEM_ERR_ARG;
    if (e >= cnt) continue;
    if (j >= 0 && j <= last)
      atomicOr(&mask[j / 4], 1u << (8 * (j % 4) + h));
    else if (a.r.status)
      *a.r.status = STEM_ERR_ARG;
  }
  __syncthreads();
  write_union<kPlanThreads>(a.c, a.lists, list, seq, last, nh, mask, wbuf, a.r.status);
}

// ------------------------------------------------------------------ attention

__device__ __forceinline__ int list_of(const Args& a, int item) {
  return a.share ? item / a.lists.tiles_h : item;
}

// The item that this CTA has a part of (items: none), the item's first CTA, and the chunk. Every CTA
// sums the counts of all items (from L2) for the chunk, then the parts for its place among them.
struct Place {
  int item, first, chunk;
};
template <int WARPS>
__device__ __forceinline__ int cta_scan(int n, int* wsum, int& total) {  // sums before this thread's
  int s = n;
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(kFull, s, o);
    if (threadIdx.x % 32 >= o) s += y;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 31) wsum[threadIdx.x / 32] = s;
  __syncthreads();
  total = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < static_cast<int>(threadIdx.x) / 32) s += wsum[w];
    total += wsum[w];
  }
  return s - n;
}
template <int WARPS>
__device__ __forceinline__ void find_place(const Args& a, Place* sh, int* wsum) {
  const int run = (a.items + WARPS * 32 - 1) / (WARPS * 32);
  const int i0 = min(static_cast<int>(threadIdx.x) * run, a.items), i1 = min(i0 + run, a.items);
  int n = 0, total, parts = 0;
  for (int i = i0; i < i1; ++i) n += a.lists.count[list_of(a, i)];
  cta_scan<WARPS>(n, wsum, total);
  const int chunk = part_entries(total, a.at_once, a.chunk);
  for (int i = i0; i < i1; ++i) parts += (a.lists.count[list_of(a, i)] + chunk - 1) / chunk;
  int s = cta_scan<WARPS>(parts, wsum, total);
  const int cta = blockIdx.x;
  if (cta >= s && cta < s + parts) {
    int i = i0;
    for (;; ++i) {
      const int c = (a.lists.count[list_of(a, i)] + chunk - 1) / chunk;
      if (cta < s + c) break;
      s += c;
    }
    *sh = Place{i, s, chunk};
  } else if (cta >= total && threadIdx.x == 0) {
    *sh = Place{a.items, 0, chunk};
  }
  __syncthreads();
}

// Joins parts of an item, once they are all there: a warp for each head, a lane for 4 channels (at
// 64 channels the warp's halves take parts in turn). Part s is in slot slot0 + s; st holds kJoinStaged
// statistics.
constexpr int kJoinStaged = 512;

// (Not inlined, and its loops mostly not unrolled: it runs once or twice in a CTA, and fetching
// straight-line code for the first time costs more than running it.)
template <int D, int WARPS>
__device__ __noinline__ void join_parts(const Args& a, int64_t head0, int nh, int parts,
                                        float2* st, int slot0) {
  constexpr int kLanes = D / 4, kHalves = 32 / kLanes, kAtOnce = 8;
  const int lane = threadIdx.x % 32, c = lane % kLanes, half = lane / kLanes;
  const int most = kJoinStaged / nh;  // parts staged at a time
  for (int h0 = 0; h0 < nh; h0 += WARPS) {
    const int h = min(h0 + static_cast<int>(threadIdx.x) / 32, nh - 1);  // (the last one twice)
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int s0 = 0; s0 < parts; s0 += most) {
      const int n = min(parts - s0, most);
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < n * nh; i += WARPS * 32)
        st[i] = __ldcg(&a.stat[(slot0 + s0 + i / nh) * kHeadTile + i % nh]);
      __syncthreads();
      float top = m;
#pragma unroll 1
      for (int s = lane; s < n; s += 32) top = fmaxf(top, st[s * nh + h].x);
#pragma unroll
      for (int o = 16; o; o /= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float base = top == -INFINITY ? 0.f : top, f0 = ex2(m - base);
      m = top;
      l *= f0;
      x.x *= f0, x.y *= f0, x.z *= f0, x.w *= f0;
#pragma unroll 1
      for (int s = lane; s < n; s += 32) {
        const float2 v = st[s * nh + h];
        l = fmaf(ex2(v.x - base), v.y, l);
      }
#pragma unroll 1
      for (int i0 = half; i0 < n; i0 += kAtOnce * kHalves) {
        float4 p[kAtOnce];
        const float4* src = reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(h) * D) + c;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {  // (past the end: the last part again, left out below)
          const int e = min(i0 + i * kHalves, n - 1);
          p[i] = __ldcg(src + static_cast<int64_t>(slot0 + s0 + e) * (kHeadTile * D / 4));
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int e = i0 + i * kHalves;
          if (e >= n) continue;  // (not a weight of 0: the part may be infinite)
          const float f = ex2(st[e * nh + h].x - base);
          x.x = fmaf(f, p[i].x, x.x);
          x.y = fmaf(f, p[i].y, x.y);
          x.z = fmaf(f, p[i].z, x.z);
          x.w = fmaf(f, p[i].w, x.w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o /= 2) l += __shfl_xor_sync(kFull, l, o);
    if (kHalves == 2) {
      x.x += __shfl_xor_sync(kFull, x.x, 16);
      x.y += __shfl_xor_sync(kFull, x.y, 16);
      x.z += __shfl_xor_sync(kFull, x.z, 16);
      x.w += __shfl_xor_sync(kFull, x.w, 16);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (half == 0)
      *reinterpret_cast<uint2*>(a.out + (head0 + h) * D + 4 * c) =
          make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    if (lane == 0 && a.lse) a.lse[head0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(Cfg<FMT, D>::THREADS, Cfg<FMT, D>::CTAS) attn_kernel(const Args a) {
  using L = Kv<FMT, D>;
  using C = Cfg<FMT, D>;
  constexpr bool kQuant = C::Q;
  constexpr int NG = L::NG, TPS = C::TPS;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Place s_place;
  __shared__ int s_sum[C::WARPS];
  __shared__ bool s_last;
  __shared__ Entry ent[kStaged];
  __shared__ float s_m[C::WARPS][kHeadTile], s_l[C::WARPS][kHeadTile];

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int G = a.r.Hq / a.c.Hkv;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  int item, first, chunk = a.chunk;  // the item of this CTA, and its first CTA
  if (a.per_item) {
    item = blockIdx.x / a.per_item;
    first = item * a.per_item;
  } else {
    find_place<C::WARPS>(a, &s_place, s_sum);
    item = s_place.item, first = s_place.first, chunk = s_place.chunk;
    if (!a.direct && tid == 0) {
      if (blockIdx.x == 0) a.start[a.items] = chunk;
      if (item < a.items && static_cast<int>(blockIdx.x) == first) a.start[item] = first;
    }
  }
  // rows that keep nothing
  for (int n = blockIdx.x; n < a.items; n += gridDim.x) {
    if (a.lists.count[list_of(a, n)] != 0) continue;
    const int h0 = n % a.lists.tiles_h * kHeadTile, nh = min(G - h0, kHeadTile);
    const int64_t head0 = static_cast<int64_t>(n / a.lists.tiles_h) * G + h0;
    for (int i = tid; i < nh * D; i += C::THREADS)
      a.out[head0 * D + i] = __float2bfloat16_rn(0.f);
    if (tid < nh && a.lse) a.lse[head0 + tid] = -INFINITY;
  }

  if (item >= a.items) return;
  const int n_item = a.lists.count[list_of(a, item)], parts = (n_item + chunk - 1) / chunk;
  const int part = static_cast<int>(blockIdx.x) - first;
  if (part >= parts) return;
  const int entry = n_item * part / parts, n_ent = n_item * (part + 1) / parts - entry;
  const bool whole = parts == 1;
  const int slot = blockIdx.x;
  const Entry* list = a.lists.list + static_cast<int64_t>(list_of(a, item)) * a.lists.most + entry;
  const int row = item / (a.c.Hkv * a.lists.tiles_h), kv = item / a.lists.tiles_h % a.c.Hkv;
  const int h0 = item % a.lists.tiles_h * kHeadTile;
  const int nh = min(G - h0, kHeadTile);
  const int64_t head0 = static_cast<int64_t>(row) * a.r.Hq + kv * G + h0;
  int seq, len;
  decode_row(a.c, a.r, row, seq, len);

  float* o_s = reinterpret_cast<float*>(smem);  // [C::WARPS][8][D], over the rings at the end
  // ---- the queries, as B operands: head g, channels 8t .. 8t + 7 of each group
  uint32_t qf[NG][4];
  {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.r.q) +
                                                    (head0 + (g < nh ? g : 0)) * D + 8 * t);
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      const uint4 u = g < nh ? p[y * (kKvGroup / 8)] : make_uint4(0, 0, 0, 0);
      qf[y][0] = u.x, qf[y][1] = u.y, qf[y][2] = u.z, qf[y][3] = u.w;
    }
  }
  float qscale = kLog2e / sqrtf(static_cast<float>(D));  // of head g: logits in log2 units
  float off[NG];
  if constexpr (kQuant) {
    uint32_t top = 0;  // largest |q|: bf16 bits order like the numbers, two at a time
#pragma unroll
    for (int y = 0; y < NG; ++y)
#pragma unroll
      for (int n = 0; n < 4; ++n) top = __vmaxu2(top, qf[y][n] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    // exponent that brings the largest |q| to [2^14, 2^15); within +-100, so that it and what
    // undoes it are float32 numbers
    const int up = top < 0x0080u || top >= 0x7f80u
                       ? 0
                       : min(max(14 - (static_cast<int>(top >> 7) - 127), -100), 100);
    qscale *= __uint_as_float(static_cast<uint32_t>(127 + 24 - up) << 23);
    const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float x0 = low16(qf[y][n]) * f, x1 = high16(qf[y][n]) * f;
        // (fp16 holds both exactly, but for entries 2^-30 of the largest)
        sum += x0 + x1;
        qf[y][n] = pack_f16(x0, x1);
        if (FMT == STEM_KV_Q4 && (n & 1)) {  // meets upper nibbles, which weigh 16 times as much
          const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&qf[y][n]),
                                    __floats2half2_rn(0.0625f, 0.0625f));
          qf[y][n] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      off[y] = -static_cast<float>(L::OFFSET) * 0x1p-24f * sum;
    }
  }
  uint32_t ob0 = 0, ob1 = 0;  // B operand of the offsets' MMA
  if constexpr (kQuant) {
    // What the codes' offset adds to a logit, sum_y s_ty off_yh, is one MMA of the scales as they
    // are (bf16) with off in three bf16 pieces along k: groups (0, 1), (2, 3) or, of 64 channels,
    // (0, 1) alone, from lane t = 0 on.
    const int piece = NG == 4 ? t / 2 : t;
    auto pieces = [&](float x, float& hi, float& mid, float& lo) {
      hi = low16(pack_bf16(x, 0.f));
      mid = low16(pack_bf16(x - hi, 0.f));
      lo = x - hi - mid;
    };
    float h0_, m0_, l0_, h1_, m1_, l1_;
    pieces(NG == 4 && (t & 1) ? off[NG - 2] : off[0], h0_, m0_, l0_);
    pieces(NG == 4 && (t & 1) ? off[NG - 1] : off[1], h1_, m1_, l1_);
    ob0 = piece == 0   ? pack_bf16(h0_, h1_)
          : piece == 1 ? pack_bf16(m0_, m1_)
          : piece == 2 ? pack_bf16(l0_, l1_)
                       : 0u;
    ob1 = NG == 4 && t < 2 ? pack_bf16(l0_, l1_) : 0u;
  }
  const float qs0 = __shfl_sync(kFull, qscale, 8 * t), qs1 = __shfl_sync(kFull, qscale, 8 * t + 4);

  float acc[2 * NG][4];  // rows: channels; columns: heads 2t, 2t + 1
  float asum[4];         // row y: sum of group y's weights
  float m0, m1, l0, l1;  // running maximum (log2 units) and sum of the weights as the MMA sees them
  float lim0, lim1;      // largest logits (as the MMA gives them) within the maximum's slack
  float vf0, vf1;        // power of two of the V scales that each head meets
  int vlim0, vlim1;      // largest scales (bf16 bits) that they are good for
  uint32_t seen[NG / 2];        // largest V scale (bf16 bits) of each group, two groups a word
  float f0[kQuant ? NG : 1];    // going over the entries again: the largest p s of each group, then
  float f1[kQuant ? NG : 1];    // the power of two that it gets
  unsigned char* ring = smem + warp * C::RING;
  const int spb_log = a.c.block / C::STEP == 2 ? 1 : a.c.block / C::STEP == 4 ? 2 : 3;
  const int64_t page_bytes = static_cast<int64_t>(a.c.Hkv) * a.c.record;
  const unsigned char* head_pages = a.c.at(0, kv) + lane * 16;

  // Goes over the steps of the entries that one of `heads` keeps. again (at 8 and 4 bits): with the
  // statistics as the first time left them, for the largest p s of each group into f0 and f1, or with
  // weights in units of f0 and f1 (exact).
  auto stream = [&](uint32_t heads, auto again, bool exact) {
    constexpr bool kAgain = decltype(again)::value;
#pragma unroll
    for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) asum[e] = 0.f;
    if constexpr (!kAgain) {
      m0 = m1 = lim0 = lim1 = -INFINITY;
      l0 = l1 = 0.f;
      vf0 = vf1 = 1.f;
      vlim0 = vlim1 = -1;
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) seen[w] = 0;
    }
    for (int e0 = 0; e0 < n_ent; e0 += kStaged) {
      __syncthreads();
      const int n_now = min(n_ent - e0, kStaged);
      for (int n = tid; n < n_now; n += C::THREADS) ent[n] = list[e0 + n];
      __syncthreads();
      // Warp w takes steps [u0, u1) of the staged entries, one after the other: two walkers, one
      // that fetches and one that computes, look at an entry when they come to it.
      const int units = n_now << spb_log, per_entry = 1 << spb_log;
      const int u0 = units * warp / C::WARPS, u1 = units * (warp + 1) / C::WARPS;
      auto tokens = [&](const Entry& e) -> int {  // of an entry; 0 or less: nothing to do
        return e.what >> 16 & heads ? len - static_cast<int>(e.what & 0xffffu) * a.c.block : 0;
      };
      int fu = u0, ftok = 0;
      const unsigned char* fsrc = nullptr;
      auto fetch = [&](int stage) {
        if (fu < u1) {
          if (fu == u0 || (fu & (per_entry - 1)) == 0) {
            const Entry e = ent[fu >> spb_log];
            const int skip = fu & (per_entry - 1);
            ftok = tokens(e) - skip * C::STEP;
            fsrc = head_pages + e.page * page_bytes + skip * C::STEP_BYTES;
          }
          if (ftok > 0) {
            unsigned char* dst = ring + stage * C::STEP_BYTES + lane * 16;
#pragma unroll
            for (int n = 0; n < C::STEP_BYTES / 512; ++n) cp16(dst + n * 512, fsrc + n * 512);
            if (C::STEP_BYTES % 512 != 0 && lane < C::STEP_BYTES % 512 / 16)
              cp16(dst + C::STEP_BYTES / 512 * 512, fsrc + C::STEP_BYTES / 512 * 512);
          }
          ftok -= C::STEP;
          fsrc += C::STEP_BYTES;
          ++fu;
        }
        cp_commit();
      };
#pragma unroll
      for (int n = 0; n < C::STAGES - 1; ++n) fetch(n);
      int stage = 0, valid = 0;
      uint32_t hb = 0;
      for (int u = u0; u < u1; ++u) {
        // the next step to fetch takes the stage that the step before this one has left
        fetch(stage == 0 ? C::STAGES - 1 : stage - 1);
        cp_wait<C::STAGES - 1>();
        __syncwarp();
        if (u == u0 || (u & (per_entry - 1)) == 0) {
          const Entry e = ent[u >> spb_log];
          valid = tokens(e) - (u & (per_entry - 1)) * C::STEP;
          hb = e.what >> 16 & heads;
        }
        if (valid > 0) {
          const unsigned char* step = ring + stage * C::STEP_BYTES;
          // ---- logits: rows are tokens g and g + 8 of a tile, columns heads 2t and 2t + 1
          float z[TPS][4];
          uint32_t sv[TPS][2][2];  // V scales of tokens g, g + 8: two groups a word
          if constexpr (!kQuant) {
#pragma unroll
            for (int y = 0; y < NG; ++y) {
              const uint4 ka = *reinterpret_cast<const uint4*>(step + L::word(0, y, 0, lane));
              const uint4 kb = *reinterpret_cast<const uint4*>(step + L::word(1, y, 0, lane));
              if (y == 0)
                mma_bf16_new(z[0], ka.x, kb.x, ka.y, kb.y, qf[y][0], qf[y][1]);
              else
                mma_bf16(z[0], ka.x, kb.x, ka.y, kb.y, qf[y][0], qf[y][1]);
              mma_bf16(z[0], ka.z, kb.z, ka.w, kb.w, qf[y][2], qf[y][3]);
            }
          } else {
            uint32_t kw[TPS][2][NG * L::WPG], sk[TPS][2][2];
#pragma unroll
            for (int i = 0; i < TPS; ++i) {
              const unsigned char* tile = step + i * L::TILE_BYTES;
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const unsigned char* s = tile + 2 * L::CODES + (g + 8 * r) * L::SCROW;
                if constexpr (NG == 4) {
                  const uint4 x = *reinterpret_cast<const uint4*>(s);
                  sk[i][r][0] = x.x, sk[i][r][1] = x.y, sv[i][r][0] = x.z, sv[i][r][1] = x.w;
                } else {
                  const uint2 x = *reinterpret_cast<const uint2*>(s);
                  sk[i][r][0] = x.x, sv[i][r][0] = x.y;
                  sk[i][r][1] = sv[i][r][1] = 0;
                }
              }
              const uint32_t s0 = NG == 4 && (t & 1) ? sk[i][0][1] : sk[i][0][0];
              const uint32_t s1 = NG == 4 && (t & 1) ? sk[i][1][1] : sk[i][1][0];
              mma_bf16_new(z[i], s0, s1, s0, s1, ob0, ob1);
#pragma unroll
              for (int p = 0; p < L::PIECES; ++p) {
                const uint4 x = *reinterpret_cast<const uint4*>(tile + p * 512 + lane * 16);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int n = 0; n < 4; ++n)
                  kw[i][(p * 4 + n) / (NG * L::WPG)][(p * 4 + n) % (NG * L::WPG)] = w[n];
              }
            }
#pragma unroll
            for (int y = 0; y < NG; ++y) {
#pragma unroll
              for (int i = 0; i < TPS; ++i) {
                float d[4];
                if constexpr (FMT == STEM_KV_Q4) {
                  const uint32_t a0 = kw[i][0][y], a1 = kw[i][1][y];
                  mma_f16_new(d, a0 & 0x000f000fu, a1 & 0x000f000fu, a0 & 0x00f000f0u,
                              a1 & 0x00f000f0u, qf[y][0], qf[y][1]);
                  mma_f16(d, a0 >> 8 & 0x000f000fu, a1 >> 8 & 0x000f000fu, a0 >> 8 & 0x00f000f0u,
                          a1 >> 8 & 0x00f000f0u, qf[y][2], qf[y][3]);
                } else {
                  const uint32_t a0 = kw[i][0][2 * y], a1 = kw[i][1][2 * y];
                  const uint32_t b0 = kw[i][0][2 * y + 1], b1 = kw[i][1][2 * y + 1];
                  mma_f16_new(d, a0 & 0x00ff00ffu, a1 & 0x00ff00ffu, a0 >> 8 & 0x00ff00ffu,
                              a1 >> 8 & 0x00ff00ffu, qf[y][0], qf[y][1]);
                  mma_f16(d, b0 & 0x00ff00ffu, b1 & 0x00ff00ffu, b0 >> 8 & 0x00ff00ffu,
                          b1 >> 8 & 0x00ff00ffu, qf[y][2], qf[y][3]);
                }
                const float s0 = y & 1 ? high16(sk[i][0][y / 2]) : low16(sk[i][0][y / 2]);
                const float s1 = y & 1 ? high16(sk[i][1][y / 2]) : low16(sk[i][1][y / 2]);
                z[i][0] = fmaf(s0, d[0], z[i][0]);
                z[i][1] = fmaf(s0, d[1], z[i][1]);
                z[i][2] = fmaf(s1, d[2], z[i][2]);
                z[i][3] = fmaf(s1, d[3], z[i][3]);
              }
            }
          }
          // ---- tokens past the row's length and heads that do not keep the block: weight 0, and
          // scale 0, whatever their bytes hold
          bool on0 = true, on1 = true;
          if (valid < C::STEP || hb != 0xffu) {
            on0 = hb >> (2 * t) & 1;
            on1 = hb >> (2 * t + 1) & 1;
#pragma unroll
            for (int i = 0; i < TPS; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const bool in = i * kKvTile + 8 * r + g < valid;
                if (!(in && on0)) z[i][2 * r] = -INFINITY;
                if (!(in && on1)) z[i][2 * r + 1] = -INFINITY;
                if (kQuant && !in) sv[i][r][0] = sv[i][r][1] = 0;
              }
          }
          // ---- running maximum and scale: exact only when a logit or a scale leaves its slack
          if constexpr (!kAgain) {
            float n0 = fmaxf(z[0][0], z[0][2]), n1 = fmaxf(z[0][1], z[0][3]);
            bool move = false;
            if constexpr (kQuant) {
              n0 = fmaxf(n0, fmaxf(z[1][0], z[1][2]));
              n1 = fmaxf(n1, fmaxf(z[1][1], z[1][3]));
              uint32_t top = 0;
#pragma unroll
              for (int w = 0; w < NG / 2; ++w) {
                const uint32_t here = __vmaxu2(__vmaxu2(sv[0][0][w], sv[0][1][w]),
                                               __vmaxu2(sv[1][0][w], sv[1][1][w]));
                seen[w] = __vmaxu2(seen[w], here);
                top = w == 0 ? here : __vmaxu2(top, here);
              }
              const int most = static_cast<int>(max(top & 0xffffu, top >> 16));
              move = (on0 && most > vlim0) || (on1 && most > vlim1);
            }
            move |= n0 > lim0 || n1 > lim1;
            if (__any_sync(kFull, move)) {
              n0 *= qs0;
              n1 *= qs1;
#pragma unroll
              for (int o = 4; o < 32; o *= 2) {
                n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, o));
                n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, o));
              }
              n0 = fmaxf(n0, m0);
              n1 = fmaxf(n1, m1);
              const float a0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0);
              const float a1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
              m0 = n0;
              m1 = n1;
              lim0 = (n0 + kSlack) * (1.f / qs0);
              lim1 = (n1 + kSlack) * (1.f / qs1);
              l0 *= a0;
              l1 *= a1;
              float c0 = a0, c1 = a1;
              if constexpr (kQuant) {
                uint32_t top = 0;  // largest finite scale: bf16 bits order like the numbers
#pragma unroll
                for (int i = 0; i < TPS; ++i)
#pragma unroll
                  for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int w = 0; w < NG / 2; ++w) {
                      const uint32_t lo = sv[i][r][w] & 0xffffu, hi = sv[i][r][w] >> 16;
                      top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                    }
                top = __reduce_max_sync(kFull, top);
                const uint32_t ex = top >> 7;  // biased exponent
                const float f = __uint_as_float(min(254u + kScaleSet - ex, 245u) << 23);
                const int lim = static_cast<int>((ex + kScaleSlack + 1) << 7) - 1;
                if (on0 && static_cast<int>(top) > vlim0) {
                  if (vlim0 >= 0) c0 *= f / vf0;
                  vf0 = f;
                  vlim0 = lim;
                }
                if (on1 && static_cast<int>(top) > vlim1) {
                  if (vlim1 >= 0) c1 *= f / vf1;
                  vf1 = f;
                  vlim1 = lim;
                }
              }
#pragma unroll
              for (int n = 0; n < 2 * NG; ++n) {
                acc[n][0] *= c0;
                acc[n][1] *= c1;
                acc[n][2] *= c0;
                acc[n][3] *= c1;
              }
              asum[0] *= c0;
              asum[1] *= c1;
              asum[2] *= c0;
              asum[3] *= c1;
            }
          }
          const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
          float p[TPS][4];
#pragma unroll
          for (int i = 0; i < TPS; ++i) {
            p[i][0] = ex2(fmaf(z[i][0], qs0, -b0));
            p[i][1] = ex2(fmaf(z[i][1], qs1, -b1));
            p[i][2] = ex2(fmaf(z[i][2], qs0, -b0));
            p[i][3] = ex2(fmaf(z[i][3], qs1, -b1));
          }
          // ---- O^T += V^T P: rows are channels, P^T is P transposed in registers
          if constexpr (!kQuant) {
            const unsigned char* vt = step + L::CODES;
            l0 += p[0][0] + p[0][2];
            l1 += p[0][1] + p[0][3];
            uint32_t pa, pb, ra, rb;
            two_parts(p[0][0], p[0][1], pa, ra);
            two_parts(p[0][2], p[0][3], pb, rb);
            const uint32_t w0 = transpose8(pa), w1 = transpose8(pb);
            const uint32_t r0 = transpose8(ra), r1 = transpose8(rb);
            // V rows of tokens that are not there may hold anything: 0 * NaN is not 0
            uint32_t ka = kFull, kb = kFull;
            if (valid < kKvTile) {
              ka = (2 * t < valid ? 0xffffu : 0u) | (2 * t + 1 < valid ? 0xffff0000u : 0u);
              kb = (2 * t + 8 < valid ? 0xffffu : 0u) | (2 * t + 9 < valid ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int y = 0; y < NG; ++y) {
              uint4 va = *reinterpret_cast<const uint4*>(vt + L::word(0, y, 0, lane));
              uint4 vb = *reinterpret_cast<const uint4*>(vt + L::word(1, y, 0, lane));
              va.x &= ka, va.y &= ka, va.z &= ka, va.w &= ka;
              vb.x &= kb, vb.y &= kb, vb.z &= kb, vb.w &= kb;
              mma_bf16(acc[2 * y], va.x, va.y, vb.x, vb.y, w0, w1);
              mma_bf16(acc[2 * y + 1], va.z, va.w, vb.z, vb.w, w0, w1);
              mma_bf16(acc[2 * y], va.x, va.y, vb.x, vb.y, r0, r1);
              mma_bf16(acc[2 * y + 1], va.z, va.w, vb.z, vb.w, r0, r1);
            }
          } else {
            uint32_t vw[TPS][2][NG * L::WPG];
#pragma unroll
            for (int i = 0; i < TPS; ++i) {
              if constexpr (!kAgain) {
                l0 += p[i][0] + p[i][2];
                l1 += p[i][1] + p[i][3];
#pragma unroll
                for (int n = 0; n < 4; ++n) p[i][n] *= n & 1 ? vf1 : vf0;
              }
#pragma unroll
              for (int q = 0; q < L::PIECES; ++q) {
                const uint4 x = *reinterpret_cast<const uint4*>(step + i * L::TILE_BYTES + L::CODES +
                                                                q * 512 + lane * 16);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int n = 0; n < 4; ++n)
                  vw[i][(q * 4 + n) / (NG * L::WPG)][(q * 4 + n) % (NG * L::WPG)] = w[n];
              }
            }
#pragma unroll
            for (int y = 0; y < NG; ++y) {
              const uint32_t one = g == y ? 0x3c003c00u : 0u;
#pragma unroll
              for (int i = 0; i < TPS; ++i) {
                const float s0 = y & 1 ? high16(sv[i][0][y / 2]) : low16(sv[i][0][y / 2]);
                const float s1 = y & 1 ? high16(sv[i][1][y / 2]) : low16(sv[i][1][y / 2]);
                float a[4] = {p[i][0] * s0, p[i][1] * s0, p[i][2] * s1, p[i][3] * s1};
                if constexpr (kAgain) {
                  if (!exact) {  // (fmaxf leaves out the 0 * NaN of a masked token)
                    f0[y] = fmaxf(f0[y], fmaxf(a[0], a[2]));
                    f1[y] = fmaxf(f1[y], fmaxf(a[1], a[3]));
                    continue;
                  }
#pragma unroll
                  for (int n = 0; n < 4; ++n) {
                    // (p s has passed float32's range only where f is below 1)
                    const float f = n & 1 ? f1[y] : f0[y];
                    a[n] = f < 1.f ? p[i][n] * ((n < 2 ? s0 : s1) * f) : a[n] * f;
                    if (z[i][n] == -INFINITY) a[n] = 0.f;  // masked: whatever its scale
                  }
                }
                const uint32_t w0 = transpose8(pack_f16(a[0], a[1]));
                const uint32_t w1 = transpose8(pack_f16(a[2], a[3]));
                mma_f16(asum, one, 0u, one, 0u, w0, w1);
                if constexpr (FMT == STEM_KV_Q4) {
                  const uint32_t va = vw[i][0][y], vb = vw[i][1][y];
                  mma_f16(acc[2 * y], va & 0x000f000fu, va & 0x00f000f0u, vb & 0x000f000fu,
                          vb & 0x00f000f0u, w0, w1);
                  mma_f16(acc[2 * y + 1], va >> 8 & 0x000f000fu, va >> 8 & 0x00f000f0u,
                          vb >> 8 & 0x000f000fu, vb >> 8 & 0x00f000f0u, w0, w1);
                } else {
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint32_t va = vw[i][0][2 * y + x], vb = vw[i][1][2 * y + x];
                    mma_f16(acc[2 * y + x], va & 0x00ff00ffu, va >> 8 & 0x00ff00ffu,
                            vb & 0x00ff00ffu, vb >> 8 & 0x00ff00ffu, w0, w1);
                  }
                }
              }
            }
          }
        }
        __syncwarp();
        valid -= C::STEP;
        stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      }
      cp_wait<0>();
      __syncwarp();
    }

    // ---- numerators in units of V: o = sum_t p_t V_t relative to 2^m
    if constexpr (kQuant) {
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        const float inv0 = 1.f / (kAgain ? f0[y] : vf0), inv1 = 1.f / (kAgain ? f1[y] : vf1);
        const float off0 = static_cast<float>(L::OFFSET) * __shfl_sync(kFull, asum[0], 4 * y + t);
        const float off1 = static_cast<float>(L::OFFSET) * __shfl_sync(kFull, asum[1], 4 * y + t);
        // the second 8 rows of a 4-bit tile come from upper nibbles
        const float second = FMT == STEM_KV_Q4 ? 0x1p20f : 0x1p24f;
#pragma unroll
        for (int n = 2 * y; n < 2 * y + 2; ++n) {
          acc[n][0] = (acc[n][0] * 0x1p24f - off0) * inv0;
          acc[n][1] = (acc[n][1] * 0x1p24f - off1) * inv1;
          acc[n][2] = (acc[n][2] * second - off0) * inv0;
          acc[n][3] = (acc[n][3] * second - off1) * inv1;
        }
      }
    }
    if constexpr (!kAgain) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) {
        l0 += __shfl_xor_sync(kFull, l0, o);
        l1 += __shfl_xor_sync(kFull, l1, o);
      }
    }
  };

  // Joins the warps' results for the heads in `heads` and writes them.
  auto finish = [&](uint32_t heads) {
    __syncthreads();
    if (g == 0) {
      s_m[warp][2 * t] = m0, s_m[warp][2 * t + 1] = m1;
      s_l[warp][2 * t] = l0, s_l[warp][2 * t + 1] = l1;
    }
    float* o = o_s + warp * kHeadTile * D;
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      const int d = kKvGroup * y + 4 * g;
      *reinterpret_cast<float4*>(o + 2 * t * D + d) =
          make_float4(acc[2 * y][0], acc[2 * y][2], acc[2 * y + 1][0], acc[2 * y + 1][2]);
      *reinterpret_cast<float4*>(o + (2 * t + 1) * D + d) =
          make_float4(acc[2 * y][1], acc[2 * y][3], acc[2 * y + 1][1], acc[2 * y + 1][3]);
    }
    __syncthreads();
    // each head's warps' weights, relative to the largest maximum, in place of their maxima
    if (tid < kHeadTile) {
      float m = s_m[0][tid];
#pragma unroll
      for (int w = 1; w < C::WARPS; ++w) m = fmaxf(m, s_m[w][tid]);
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) {  // (a warp that saw nothing of the head weighs 0)
        const float f = ex2(s_m[w][tid] - base);
        s_m[w][tid] = f;
        l = fmaf(f, s_l[w][tid], l);
      }
      if (heads >> tid & 1) {
        s_l[0][tid] = l == 0.f ? 0.f : 1.f / l;
        if (!whole)
          a.stat[slot * kHeadTile + tid] = make_float2(m, l);
        else if (a.lse && tid < nh)
          a.lse[head0 + tid] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
    __syncthreads();
    for (int n = tid; n < nh * (D / 4); n += C::THREADS) {
      const int h = n / (D / 4), d = n % (D / 4);
      if (!(heads >> h & 1)) continue;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) {
        const float f = s_m[w][h];
        const float4 v = reinterpret_cast<const float4*>(o_s + (w * kHeadTile + h) * D)[d];
        x.x = fmaf(f, v.x, x.x);
        x.y = fmaf(f, v.y, x.y);
        x.z = fmaf(f, v.z, x.z);
        x.w = fmaf(f, v.w, x.w);
      }
      if (whole) {
        const float inv = s_l[0][h];
        reinterpret_cast<uint2*>(a.out + (head0 + h) * D)[d] =
            make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
      } else {
        reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(slot) * kHeadTile + h) * D)[d] = x;
      }
    }
  };

  stream(0xffu, std::false_type{}, false);
  if constexpr (kQuant) {
    // Weights that may be off (lane (y, t) has the sums of group y for heads 2t and 2t + 1), and the NaN
    // of a weight 0 with a scale that is NaN, of a block that another head keeps.
#pragma unroll
    for (int w = 0; w < NG / 2; ++w)
#pragma unroll
      for (int o = 4; o < 32; o *= 2) seen[w] = __vmaxu2(seen[w], __shfl_xor_sync(kFull, seen[w], o));
    bool unsure = false;
    if (g < NG && 2 * t < nh) {
      const uint32_t pair = NG == 4 && g >= 2 ? seen[NG / 2 - 1] : seen[0];
      const bool any = (g & 1 ? pair >> 16 : pair & 0xffffu) != 0;  // (not all of the group's V are 0)
      const float least = static_cast<float>(n_ent) * (a.c.block / C::WARPS) * kLeastSum;
      unsure = any && ((l0 > 0.f && asum[0] < least) || (l1 > 0.f && asum[1] < least));
      unsure |= !a.share && (isnan(asum[0]) || isnan(asum[1]));
    }
    if (__syncthreads_or(unsure)) {
#pragma unroll
      for (int y = 0; y < NG; ++y) f0[y] = f1[y] = 0.f;
      stream(0xffu, std::true_type{}, false);
#pragma unroll
      for (int y = 0; y < NG; ++y) {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          f0[y] = fmaxf(f0[y], __shfl_xor_sync(kFull, f0[y], o));
          f1[y] = fmaxf(f1[y], __shfl_xor_sync(kFull, f1[y], o));
        }
        // the largest weight to [2^14, 2^15), or below where it is infinite (less than 2^(4 + 126)) or
        // next to nothing
        auto power = [](float w) {
          const int up = 14 + 127 - static_cast<int>(__float_as_uint(w) >> 23);
          return __uint_as_float(static_cast<uint32_t>(127 + (isinf(w) ? -117 : min(up, 126))) << 23);
        };
        f0[y] = power(f0[y]);
        f1[y] = power(f1[y]);
      }
      stream(0xffu, std::true_type{}, true);
    }
    finish(0xffu);
  } else {
    // A head that does not keep a block still meets its V rows with weight 0, and 0 * NaN or 0 * inf is
    // not 0. That shows as a NaN: such a CTA goes over its entries once more for each head alone, so
    // that a head meets only blocks it keeps.
    bool odd = false;
    if (!a.share && nh > 1) {
      bool nan = false;
#pragma unroll
      for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) nan |= isnan(acc[n][e]);
      odd = __syncthreads_or(nan);
    }
    if (!odd) {
      finish(0xffu);
    } else {
      for (int h = 0; h < nh; ++h) {
        stream(1u << h, std::false_type{}, false);
        finish(1u << h);
      }
    }
  }
  // ---- of an item in parts, the CTA that brings the last one joins them
  if (!whole && a.direct) {
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&a.lists.arrived[item], 1) == parts - 1;
    __syncthreads();
    if (s_last) {
      __threadfence();  // (the other CTAs' parts are visible)
      join_parts<D, C::WARPS>(a, head0, nh, parts, reinterpret_cast<float2*>(smem), first);
    }
  }
}

// Joins the items that several CTAs have a part of: one CTA per (row, query head). Threads first turn
// the parts' maxima into weights, then groups of D threads sum the numerators of every kGroups-th part.
constexpr int kJoinThreads = 512;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Args a) {
  constexpr int kGroups = kJoinThreads / D, kJoinWarps = kJoinThreads / 32;
  extern __shared__ float weight[];  // [most]
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps], s_o[kGroups][D];
  const int row = blockIdx.y, head = blockIdx.x, tid = threadIdx.x;
  const int G = a.r.Hq / a.c.Hkv, h = head % G % kHeadTile;
  const int item = (row * a.c.Hkv + head / G) * a.lists.tiles_h + head % G / kHeadTile;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  const int n = a.lists.count[list_of(a, item)];
  if (n == 0) return;
  const int chunk = a.per_item ? a.chunk : a.start[a.items], parts = (n + chunk - 1) / chunk;
  if (parts == 1) return;  // (its CTA has written the output)
  const int slot0 = a.per_item ? item * a.per_item : a.start[item];
  float m = -INFINITY;
  for (int s = tid; s < parts; s += kJoinThreads) m = fmaxf(m, a.stat[(slot0 + s) * kHeadTile + h].x);
  for (int o = 16; o; o /= 2) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if (tid % 32 == 0) s_m[tid / 32] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_m[w]);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int s = tid; s < parts; s += kJoinThreads) {
    const float2 st = a.stat[(slot0 + s) * kHeadTile + h];
    const float f = ex2(st.x - base);
    weight[s] = f;
    l = fmaf(f, st.y, l);
  }
  for (int o = 16; o; o /= 2) l += __shfl_xor_sync(kFull, l, o);
  if (tid % 32 == 0) s_l[tid / 32] = l;
  __syncthreads();
  const int d = tid % D, grp = tid / D;
  const float* part = a.part + static_cast<int64_t>(h) * D + d;
  float x = 0.f;
#pragma unroll 8
  for (int s = grp; s < parts; s += kGroups)
    x = fmaf(weight[s], part[static_cast<int64_t>(slot0 + s) * kHeadTile * D], x);
  s_o[grp][d] = x;
  __syncthreads();
  if (grp == 0) {
    l = s_l[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) l += s_l[w];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) x += s_o[i][d];
    const int64_t o = static_cast<int64_t>(row) * a.r.Hq + head;
    a.out[o * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : x / l);
    if (d == 0 && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// Sizes of a call, and where its arrays are in the workspace.
struct Sizes {
  int tiles_h, most, ctas, per_item, chunk, at_once;
  int64_t items, lists;
  size_t list, count, arrived, start, stat, part, total;
};
Sizes sizes_of(int format, int D, int block, int Hkv, int max_blocks, int R, int Hq, int kcap,
               bool share) {
  Sizes s;
  const int G = Hq / Hkv;
  s.tiles_h = (G + kHeadTile - 1) / kHeadTile;
  s.items = static_cast<int64_t>(R) * Hkv * s.tiles_h;
  s.lists = share ? static_cast<int64_t>(R) * Hkv : s.items;
  // one list, or the union of its heads' lists
  s.most = share ? kcap
                 : static_cast<int>(std::min<int64_t>(
                       static_cast<int64_t>(std::min(G, kHeadTile)) * kcap, max_blocks));
  const int per_sm = format == STEM_KV_Q4 ? Cfg<STEM_KV_Q4, 128>::CTAS
                     : format == STEM_KV_Q8 ? Cfg<STEM_KV_Q8, 128>::CTAS
                                            : Cfg<STEM_KV_BF16, 128>::CTAS;
  const int steps = block / (format == STEM_KV_BF16 ? Cfg<STEM_KV_BF16, 128>::STEP
                                                    : Cfg<STEM_KV_Q4, 128>::STEP);
  s.at_once = sm_count() * per_sm;
  s.chunk = std::max(1, kMinSteps / steps);
  s.per_item = (s.most + s.chunk - 1) / s.chunk;
  int64_t ctas = s.items * s.per_item;
  if (ctas > s.at_once) {
    // a chunk that is an at_once-th of the entries, or more, leaves at most this many parts
    ctas = std::min<int64_t>(ctas, s.items + s.at_once);
    s.per_item = 0;
  }
  s.ctas = static_cast<int>(ctas);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  s.list = take(sizeof(Entry) * static_cast<size_t>(s.lists) * s.most);
  s.count = take(sizeof(int32_t) * static_cast<size_t>(s.lists));
  const size_t slots = static_cast<size_t>(s.ctas);
  s.arrived = take(sizeof(int32_t) * static_cast<size_t>(s.items));
  s.start = take(sizeof(int32_t) * static_cast<size_t>(s.items + 1));
  s.stat = take(sizeof(float2) * slots * kHeadTile);
  s.part = take(sizeof(float) * slots * kHeadTile * D);
  s.total = o;
  return s;
}

template <int FMT, int D>
cudaError_t launch(const Args& a, int ctas, bool planned, cudaStream_t st) {
  using C = Cfg<FMT, D>;
  static_assert(C::RING >= kHeadTile * D * 4 && C::WARPS * C::RING >= kJoinStaged * sizeof(float2),
                "the rings hold the warps' results, then the parts' statistics, at the end");
  cudaError_t e = cudaSuccess;
  if (!planned) {
    const size_t mask = a.share ? 0 : 4 * ((a.c.max_blocks + 3) / 4);
    const int lists = a.share ? a.c.Hkv : a.c.Hkv * a.lists.tiles_h;
    e = launch_after(plan_kernel, dim3(lists, a.r.R), kPlanThreads, mask, 1, st, a);
    if (e != cudaSuccess) return e;
  }
  constexpr size_t bytes = static_cast<size_t>(C::WARPS) * C::RING;
  // (per device and context; 0.1 us)
  e = cudaFuncSetAttribute(attn_kernel<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e != cudaSuccess) return e;
  e = launch_after(attn_kernel<FMT, D>, dim3(ctas), C::THREADS, bytes, 1, st, a);
  if (e != cudaSuccess || a.direct) return e;
  return launch_after(join_kernel<D>, dim3(a.r.Hq, a.r.R), kJoinThreads,
                      sizeof(float) * a.lists.most, 1, st, a);
}

}  // namespace

DecodeLists decode_lists(const KvCache& c, int format, int D, const DecodeRows& r, bool share,
                         unsigned char* ws) {
  const Sizes s = sizes_of(format, D, c.block, c.Hkv, c.max_blocks, r.R, r.Hq, r.kcap, share);
  DecodeLists l;
  l.list = reinterpret_cast<Entry*>(ws + s.list);
  l.count = reinterpret_cast<int32_t*>(ws + s.count);
  l.arrived = reinterpret_cast<int32_t*>(ws + s.arrived);
  l.most = s.most;
  l.tiles_h = s.tiles_h;
  return l;
}

cudaError_t launch_decode_attn(const KvCache& c, int format, int D, const DecodeRows& r, bool share,
                               bool planned, void* out, float* lse, unsigned char* ws,
                               cudaStream_t st) {
  const Sizes s = sizes_of(format, D, c.block, c.Hkv, c.max_blocks, r.R, r.Hq, r.kcap, share);
  Args a;
  a.c = c;
  a.r = r;
  a.share = share;
  a.lists = decode_lists(c, format, D, r, share, ws);
  a.items = static_cast<int>(s.items);
  a.per_item = s.per_item;
  a.chunk = s.chunk;
  a.at_once = s.at_once;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.direct = std::min(s.ctas, s.at_once) <= kDirect * s.items;
  a.start = reinterpret_cast<int32_t*>(ws + s.start);
  a.stat = reinterpret_cast<float2*>(ws + s.stat);
  a.part = reinterpret_cast<float*>(ws + s.part);
  if (D == 128) {
    switch (format) {
      case STEM_KV_BF16: return launch<STEM_KV_BF16, 128>(a, s.ctas, planned, st);
      case STEM_KV_Q8: return launch<STEM_KV_Q8, 128>(a, s.ctas, planned, st);
      default: return launch<STEM_KV_Q4, 128>(a, s.ctas, planned, st);
    }
  }
  switch (format) {
    case STEM_KV_BF16: return launch<STEM_KV_BF16, 64>(a, s.ctas, planned, st);
    case STEM_KV_Q8: return launch<STEM_KV_Q8, 64>(a, s.ctas, planned, st);
    default: return launch<STEM_KV_Q4, 64>(a, s.ctas, planned, st);
  }
}

size_t decode_attn_bytes(int format, int D, int block, int Hkv, int max_blocks, int R, int Hq,
                         int kcap, bool share) {
  return sizes_of(format, D, block, Hkv, max_blocks, R, Hq, kcap, share).total;
}

}  // namespace stem
