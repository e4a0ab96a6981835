// Attention of single query tokens over the kept blocks of a paged cache (stem_decode_attn).
//
// For one row and kv head: z_th = q_h . K_t / sqrt(D) over the tokens t of the kept blocks,
// o_h = sum_t softmax_t(z_th) V_t. The K and V bytes are read once and each meets only the G query
// heads of its kv head (2 to 8 flops a byte at 16 bits), so HBM bounds the kernel and the tensor
// pipe has room to spare. It uses mma.sync.m16n8k16 with tokens (for V: channels) as the 16 rows
// and 8 query heads as the 8 columns: tcgen05's 128-row tiles would need the expanded codes in
// shared memory, four times the bytes that were read, to feed a unit that is idle 90% of the time.
//
// Codes of 4 and 8 bits go to the MMA without a conversion: a masked word holds a pair of fp16
// subnormals code * 2^-24 (times 16 for the upper nibble of a byte, undone in q or at the end).
//   K: sum_d q_d (c_d - off) over a 32-channel group is one short chain of MMAs whose accumulator
//      starts at -off * sum_d q_d; the group's scale multiplies its result (4 FMA a tile and group).
//      q is scaled by a power of two per head so that its largest entry is in [2^14, 2^15): bf16's 8
//      significant bits survive in fp16.
//   V: the scale goes to the weight: a_th = p_th s_t f rounded once to fp16, with f a power of two
//      that follows the largest scale seen (like the running maximum of the softmax), so that no
//      range of scales overflows or underflows. sum_t a_th (c_td - off) = sum a c - off * sum a; the
//      last sum comes from one more MMA against a constant, so both sums see the same rounded a.
// The tensor pipe cuts the products of a chain at 2^-25 of the largest and takes a subnormal's
// exponent for -14 (measured), so a product keeps its bits down to 2^-15 code steps times the largest
// q (or weight) of the chain. bf16 entries of q above 2^-8 of the largest lose nothing; the value sums
// lose less than 2^-10 of the half step by which the code itself may be off.
// At 16 bits the operands are bf16 as stored, P is rounded to bf16 and the normaliser sums the
// rounded values.
//
// A warp streams whole tiles (16 tokens of K and V, contiguous in the page) through a ring of its own
// in shared memory with cp.async: no barrier between warps until the end. Softmax statistics and
// sums are float32. Warps, then CTAs of one (row, kv head), are joined by (max, sum, numerator).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "decode_rows.cuh"

namespace stem {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kHeadTile = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int FMT, int D>
struct Cfg {
  using L = Kv<FMT, D>;
  static constexpr int STAGES = FMT == STEM_KV_BF16 ? 3 : 4;
  static constexpr int RING = STAGES * L::TILE_BYTES;  // a warp's
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

struct Args {
  KvCache c;
  DecodeRows r;
  bool share;
  int chunk;   // list entries of a CTA
  int splits;  // CTAs of an item
  __nv_bfloat16* out;
  float* lse;
  float* part;  // [R][Hkv * head tiles][splits][8][D + 2]: numerator, max (log2 units), sum
};

// The entries (block | heads << 16) of this CTA's part of its item's list.
__device__ __forceinline__ int build_list(const Args& a, int row, int kv, int h0, int nh, int last,
                                          uint32_t* ent, uint32_t* mask, uint32_t* wbuf) {
  const int tid = threadIdx.x, G = a.r.Hq / a.c.Hkv;
  const int e0 = blockIdx.x * a.chunk;
  const int64_t head0 = static_cast<int64_t>(row) * a.r.Hq + kv * G;
  if (a.share) {
    const int cnt = a.r.sel_cnt[head0];
    if ((cnt < 0 || cnt > a.r.kcap) && a.r.status) *a.r.status = STEM_ERR_ARG;
    const int n = min(max(min(cnt, a.r.kcap) - e0, 0), a.chunk);
    const int32_t* idx = a.r.sel_idx + head0 * a.r.kcap + e0;
    for (int e = tid; e < n; e += kWarps * 32) {
      const int j = idx[e];
      const bool ok = j >= 0 && j <= last;
      if (!ok && a.r.status) *a.r.status = STEM_ERR_ARG;
      ent[e] = ok ? j | 0xff0000u : 0u;  // no heads: skipped
    }
    __syncthreads();
    return n;
  }
  // union of the heads' lists: a byte of head bits for each block
  const int words = (last + 4) / 4;
  for (int w = tid; w < words; w += kWarps * 32) mask[w] = 0;
  __syncthreads();
  for (int h = 0; h < nh; ++h) {
    const int64_t hd = head0 + h0 + h;
    const int cnt = a.r.sel_cnt[hd];
    if ((cnt < 0 || cnt > a.r.kcap) && a.r.status) *a.r.status = STEM_ERR_ARG;
    for (int e = tid; e < min(cnt, a.r.kcap); e += kWarps * 32) {
      const int j = a.r.sel_idx[hd * a.r.kcap + e];
      if (j >= 0 && j <= last)
        atomicOr(&mask[j / 4], 1u << (8 * (j % 4) + h));
      else if (a.r.status)
        *a.r.status = STEM_ERR_ARG;
    }
  }
  __syncthreads();
  // thread t owns a run of words; entries in block order
  const int run = (words + kWarps * 32 - 1) / (kWarps * 32);
  const int w0 = min(tid * run, words), w1 = min(w0 + run, words);
  uint32_t n = 0;
  for (int w = w0; w < w1; ++w)
    for (int b = 0; b < 4; ++b) n += (mask[w] >> (8 * b) & 0xffu) != 0;
  uint32_t s = n;
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t y = __shfl_up_sync(kFull, s, o);
    if (tid % 32 >= o) s += y;
  }
  if (tid % 32 == 31) wbuf[tid / 32] = s;
  __syncthreads();
  uint32_t total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < tid / 32) s += wbuf[w];
    total += wbuf[w];
  }
  int at = static_cast<int>(s - n) - e0;
  for (int w = w0; w < w1; ++w)
    for (int b = 0; b < 4; ++b) {
      const uint32_t m = mask[w] >> (8 * b) & 0xffu;
      if (!m) continue;
      if (at >= 0 && at < a.chunk) ent[at] = (4 * w + b) | m << 16;
      ++at;
    }
  __syncthreads();
  return min(max(static_cast<int>(total) - e0, 0), a.chunk);
}

template <int FMT, int D>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const Args a) {
  using L = Kv<FMT, D>;
  using C = Cfg<FMT, D>;
  constexpr bool kQuant = FMT != STEM_KV_BF16;
  constexpr int NG = L::NG;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t wbuf[kWarps];
  __shared__ float s_m[kWarps][kHeadTile], s_l[kWarps][kHeadTile];
  uint32_t* ent = reinterpret_cast<uint32_t*>(smem + kWarps * C::RING);
  uint32_t* mask = ent + a.chunk;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int G = a.r.Hq / a.c.Hkv, tiles_h = (G + kHeadTile - 1) / kHeadTile;
  const int row = blockIdx.z, kv = blockIdx.y / tiles_h, h0 = blockIdx.y % tiles_h * kHeadTile;
  const int nh = min(G - h0, kHeadTile);
  int seq, len;
  decode_row(a.c, a.r, row, seq, len);
  const int last = (len + a.c.block - 1) / a.c.block - 1;
  const int64_t head0 = static_cast<int64_t>(row) * a.r.Hq + kv * G + h0;

  const int n_ent = last >= 0 ? build_list(a, row, kv, h0, nh, last, ent, mask, wbuf) : 0;

  // ---- the queries, as B operands: head g, channels 8t .. 8t + 7 of each group
  uint32_t qf[NG][4];
  float qscale = kLog2e / sqrtf(static_cast<float>(D));  // of head g: logits in log2 units
  float cinit[NG][2];
  {
    const bool on = g < nh;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.r.q) +
                                                    (head0 + (on ? g : 0)) * D + 8 * t);
#pragma unroll
    for (int y = 0; y < NG; ++y) {
      const uint4 u = on ? p[y * (kKvGroup / 8)] : make_uint4(0, 0, 0, 0);
      qf[y][0] = u.x, qf[y][1] = u.y, qf[y][2] = u.z, qf[y][3] = u.w;
    }
    if constexpr (kQuant) {
      uint32_t top = 0;
#pragma unroll
      for (int y = 0; y < NG; ++y)
#pragma unroll
        for (int n = 0; n < 4; ++n)
          top = max(top, max(qf[y][n] & 0x7fffu, qf[y][n] >> 16 & 0x7fffu));
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      // exponent that brings the largest |q| to [2^14, 2^15); at least -100, so that what undoes
      // it stays a float32
      const int up = top < 0x0080u || top >= 0x7f80u
                         ? 0
                         : max(14 - (static_cast<int>(top >> 7) - 127), -100);
      qscale *= ldexpf(1.f, min(24 - up, 126));
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const __half2 h = __floats2half2_rn(ldexpf(low16(qf[y][n]), up),
                                              ldexpf(high16(qf[y][n]), up));
          sum += __low2float(h) + __high2float(h);
          // odd words meet upper nibbles, which weigh 16 times as much
          const __half2 w = FMT == STEM_KV_Q4 && (n & 1)
                                ? __hmul2(h, __floats2half2_rn(0.0625f, 0.0625f))
                                : h;
          qf[y][n] = *reinterpret_cast<const uint32_t*>(&w);
        }
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        sum *= -static_cast<float>(L::OFFSET) * 0x1p-24f;
        cinit[y][0] = __shfl_sync(kFull, sum, 8 * t);      // head 2t: lane row 2t
        cinit[y][1] = __shfl_sync(kFull, sum, 8 * t + 4);  // head 2t + 1
      }
    }
  }
  const float qs0 = __shfl_sync(kFull, qscale, 8 * t), qs1 = __shfl_sync(kFull, qscale, 8 * t + 4);

  float acc[2 * NG][4];  // rows: channels; columns: heads 2t, 2t + 1
  float asum[4];         // row y: sum of group y's weights
  float m0, m1, l0, l1, vf;
  unsigned char* ring = smem + warp * C::RING;
  const int tpb = a.c.block / kKvTile;
  const int units = n_ent * tpb;
  bool odd = false;  // a column's result is not a number

  // Streams the tiles of the entries that one of `heads` keeps.
  auto stream = [&](uint32_t heads) {
#pragma unroll
    for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) asum[e] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    vf = 0x1p126f;

    // tokens of unit u, 0 where there is nothing to do
    auto tokens = [&](int u, uint32_t& e) -> int {
      if (u >= units) return 0;
      e = ent[u / tpb];
      if (!(e >> 16 & heads)) return 0;
      const int j = e & 0xffffu;
      return min(max(len - j * a.c.block - u % tpb * kKvTile, 0), kKvTile);
    };
    auto fetch = [&](int u, int stage) {
      uint32_t e = 0;
      if (tokens(u, e) > 0) {
        const int page = kv_page(a.c, seq, e & 0xffffu, a.r.status);
        if (page >= 0) {
          const unsigned char* src =
              a.c.at(page, kv) + static_cast<int64_t>(u % tpb) * L::TILE_BYTES + lane * 16;
          unsigned char* dst = ring + stage * L::TILE_BYTES + lane * 16;
#pragma unroll
          for (int n = 0; n < L::TILE_BYTES / 512; ++n) cp16(dst + n * 512, src + n * 512);
          if (lane < L::TILE_BYTES % 512 / 16)
            cp16(dst + L::TILE_BYTES / 512 * 512, src + L::TILE_BYTES / 512 * 512);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int n = 0; n < C::STAGES - 1; ++n) fetch(warp + n * kWarps, n);
    int stage = 0;
    for (int u = warp; u < units; u += kWarps) {
      cp_wait<C::STAGES - 2>();
      __syncwarp();
      uint32_t e = 0;
      int valid = tokens(u, e);
      if (valid > 0 && kv_page(a.c, seq, e & 0xffffu, a.r.status) < 0) valid = 0;
      if (valid > 0) {
        const unsigned char* tile = ring + stage * L::TILE_BYTES;
        // ---- logits: rows are tokens g and g + 8, columns heads 2t and 2t + 1
        float z[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t sv[2][2];  // V scales of tokens g, g + 8: two groups a word
        if constexpr (!kQuant) {
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            const uint4 ka = *reinterpret_cast<const uint4*>(tile + L::word(0, y, 0, lane));
            const uint4 kb = *reinterpret_cast<const uint4*>(tile + L::word(1, y, 0, lane));
            mma_bf16(z, ka.x, kb.x, ka.y, kb.y, qf[y][0], qf[y][1]);
            mma_bf16(z, ka.z, kb.z, ka.w, kb.w, qf[y][2], qf[y][3]);
          }
        } else {
          uint32_t kw[2][NG * L::WPG], sk[2][2];
#pragma unroll
          for (int p = 0; p < L::PIECES; ++p) {
            const uint4 x = *reinterpret_cast<const uint4*>(tile + p * 512 + lane * 16);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int n = 0; n < 4; ++n)
              kw[(p * 4 + n) / (NG * L::WPG)][(p * 4 + n) % (NG * L::WPG)] = w[n];
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const unsigned char* s = tile + 2 * L::CODES + (g + 8 * i) * L::SCROW;
            if constexpr (NG == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(s);
              sk[i][0] = x.x, sk[i][1] = x.y, sv[i][0] = x.z, sv[i][1] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(s);
              sk[i][0] = x.x, sv[i][0] = x.y;
              sk[i][1] = sv[i][1] = 0;
            }
          }
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            float d[4] = {cinit[y][0], cinit[y][1], cinit[y][0], cinit[y][1]};
            if constexpr (FMT == STEM_KV_Q4) {
              const uint32_t a0 = kw[0][y], a1 = kw[1][y];
              mma_f16(d, a0 & 0x000f000fu, a1 & 0x000f000fu, a0 & 0x00f000f0u, a1 & 0x00f000f0u,
                      qf[y][0], qf[y][1]);
              mma_f16(d, a0 >> 8 & 0x000f000fu, a1 >> 8 & 0x000f000fu, a0 >> 8 & 0x00f000f0u,
                      a1 >> 8 & 0x00f000f0u, qf[y][2], qf[y][3]);
            } else {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                const uint32_t a0 = kw[0][2 * y + w], a1 = kw[1][2 * y + w];
                mma_f16(d, a0 & 0x00ff00ffu, a1 & 0x00ff00ffu, a0 >> 8 & 0x00ff00ffu,
                        a1 >> 8 & 0x00ff00ffu, qf[y][2 * w], qf[y][2 * w + 1]);
              }
            }
            const float s0 = y & 1 ? high16(sk[0][y / 2]) : low16(sk[0][y / 2]);
            const float s1 = y & 1 ? high16(sk[1][y / 2]) : low16(sk[1][y / 2]);
            z[0] = fmaf(s0, d[0], z[0]);
            z[1] = fmaf(s0, d[1], z[1]);
            z[2] = fmaf(s1, d[2], z[2]);
            z[3] = fmaf(s1, d[3], z[3]);
          }
        }
        // ---- running softmax; tokens past the row's length and heads that do not keep the block
        // get weight 0 whatever their bytes hold
        const uint32_t hb = e >> 16 & heads;
        const bool on0 = hb >> (2 * t) & 1, on1 = hb >> (2 * t + 1) & 1;
        const bool lo = g < valid, hi = g + 8 < valid;
        z[0] = lo && on0 ? z[0] * qs0 : -INFINITY;
        z[1] = lo && on1 ? z[1] * qs1 : -INFINITY;
        z[2] = hi && on0 ? z[2] * qs0 : -INFINITY;
        z[3] = hi && on1 ? z[3] * qs1 : -INFINITY;
        float n0 = fmaxf(z[0], z[2]), n1 = fmaxf(z[1], z[3]);
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          n0 = fmaxf(n0, __shfl_xor_sync(kFull, n0, o));
          n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, o));
        }
        n0 = fmaxf(n0, m0);
        n1 = fmaxf(n1, m1);
        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
        float up = 1.f;  // change of the weights' power of two
        if constexpr (kQuant) {
          // largest finite V scale of the tile: bf16 bits order like the numbers
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i == 0 ? !lo : !hi) sv[i][0] = sv[i][1] = 0;
#pragma unroll
            for (int w = 0; w < NG / 2; ++w) {
              const uint32_t x = sv[i][w] & 0xffffu, y = sv[i][w] >> 16;
              top = max(top, max(x < 0x7f80u ? x : 0u, y < 0x7f80u ? y : 0u));
            }
          }
          top = __reduce_max_sync(kFull, top);
          const float f = __uint_as_float(min(267u - (top >> 7), 253u) << 23);
          if (f < vf) {
            up = f / vf;
            vf = f;
          }
        }
        if (__any_sync(kFull, n0 != m0 || n1 != m1 || up != 1.f)) {
          const float a0 = exp2f(m0 - b0), a1 = exp2f(m1 - b1);
          l0 *= a0;
          l1 *= a1;
          const float c0 = a0 * up, c1 = a1 * up;
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
          m0 = n0;
          m1 = n1;
        }
        float p[4] = {exp2f(z[0] - b0), exp2f(z[1] - b1), exp2f(z[2] - b0), exp2f(z[3] - b1)};
        const unsigned char* vt = tile + L::CODES;
        if constexpr (!kQuant) {
          const uint32_t pa = pack_bf16(p[0], p[1]), pb = pack_bf16(p[2], p[3]);
          l0 += low16(pa) + low16(pb);
          l1 += high16(pa) + high16(pb);
          const uint32_t w0 = transpose8(pa), w1 = transpose8(pb);
          // V rows of tokens that are not there may hold anything: 0 * NaN is not 0
          uint32_t keep0 = kFull, keep1 = kFull;
          if (valid < kKvTile) {
            keep0 = (2 * t < valid ? 0xffffu : 0u) | (2 * t + 1 < valid ? 0xffff0000u : 0u);
            keep1 = (2 * t + 8 < valid ? 0xffffu : 0u) | (2 * t + 9 < valid ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            uint4 va = *reinterpret_cast<const uint4*>(vt + L::word(0, y, 0, lane));
            uint4 vb = *reinterpret_cast<const uint4*>(vt + L::word(1, y, 0, lane));
            if (valid < kKvTile) {
              va.x &= keep0, va.y &= keep0, va.z &= keep0, va.w &= keep0;
              vb.x &= keep1, vb.y &= keep1, vb.z &= keep1, vb.w &= keep1;
            }
            mma_bf16(acc[2 * y], va.x, va.y, vb.x, vb.y, w0, w1);
            mma_bf16(acc[2 * y + 1], va.z, va.w, vb.z, vb.w, w0, w1);
          }
        } else {
          l0 += p[0] + p[2];
          l1 += p[1] + p[3];
#pragma unroll
          for (int n = 0; n < 4; ++n) p[n] *= vf;
          uint32_t vw[2][NG * L::WPG];
#pragma unroll
          for (int q = 0; q < L::PIECES; ++q) {
            const uint4 x = *reinterpret_cast<const uint4*>(vt + q * 512 + lane * 16);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int n = 0; n < 4; ++n)
              vw[(q * 4 + n) / (NG * L::WPG)][(q * 4 + n) % (NG * L::WPG)] = w[n];
          }
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            const float s0 = y & 1 ? high16(sv[0][y / 2]) : low16(sv[0][y / 2]);
            const float s1 = y & 1 ? high16(sv[1][y / 2]) : low16(sv[1][y / 2]);
            // (a head that does not keep the block has weight 0 even where the scale is NaN)
            const uint32_t w0 = transpose8(pack_f16(on0 ? p[0] * s0 : 0.f, on1 ? p[1] * s0 : 0.f));
            const uint32_t w1 = transpose8(pack_f16(on0 ? p[2] * s1 : 0.f, on1 ? p[3] * s1 : 0.f));
            const uint32_t one = g == y ? 0x3c003c00u : 0u;
            mma_f16(asum, one, 0u, one, 0u, w0, w1);
            if constexpr (FMT == STEM_KV_Q4) {
              const uint32_t va = vw[0][y], vb = vw[1][y];
              mma_f16(acc[2 * y], va & 0x000f000fu, va & 0x00f000f0u, vb & 0x000f000fu,
                      vb & 0x00f000f0u, w0, w1);
              mma_f16(acc[2 * y + 1], va >> 8 & 0x000f000fu, va >> 8 & 0x00f000f0u,
                      vb >> 8 & 0x000f000fu, vb >> 8 & 0x00f000f0u, w0, w1);
            } else {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t va = vw[0][2 * y + x], vb = vw[1][2 * y + x];
                mma_f16(acc[2 * y + x], va & 0x00ff00ffu, va >> 8 & 0x00ff00ffu,
                        vb & 0x00ff00ffu, vb >> 8 & 0x00ff00ffu, w0, w1);
              }
            }
          }
        }
      }
      __syncwarp();
      fetch(u + (C::STAGES - 1) * kWarps, (stage + C::STAGES - 1) % C::STAGES);
      stage = stage + 1 == C::STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // ---- numerators in units of V: o = sum_t p_t V_t relative to 2^m
    if constexpr (kQuant) {
      const float inv = 1.f / vf;
#pragma unroll
      for (int y = 0; y < NG; ++y) {
        const float off0 = static_cast<float>(L::OFFSET) * __shfl_sync(kFull, asum[0], 4 * y + t);
        const float off1 = static_cast<float>(L::OFFSET) * __shfl_sync(kFull, asum[1], 4 * y + t);
        // the second 8 rows of a 4-bit tile come from upper nibbles
        const float second = FMT == STEM_KV_Q4 ? 0x1p20f : 0x1p24f;
#pragma unroll
        for (int n = 2 * y; n < 2 * y + 2; ++n) {
          acc[n][0] = (acc[n][0] * 0x1p24f - off0) * inv;
          acc[n][1] = (acc[n][1] * 0x1p24f - off1) * inv;
          acc[n][2] = (acc[n][2] * second - off0) * inv;
          acc[n][3] = (acc[n][3] * second - off1) * inv;
        }
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o *= 2) {
      l0 += __shfl_xor_sync(kFull, l0, o);
      l1 += __shfl_xor_sync(kFull, l1, o);
    }
  };

  float* o_s = reinterpret_cast<float*>(smem);  // [kWarps][8][D], over the rings
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
    for (int n = tid; n < nh * D; n += kWarps * 32) {
      const int h = n / D, d = n % D;
      if (!(heads >> h & 1)) continue;
      float m = s_m[0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = fmaxf(m, s_m[w][h]);
      const float base = m == -INFINITY ? 0.f : m;
      float x = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (s_m[w][h] == -INFINITY && s_l[w][h] == 0.f) continue;  // saw nothing of this head
        const float f = exp2f(s_m[w][h] - base);
        x = fmaf(f, o_s[(w * kHeadTile + h) * D + d], x);
        l = fmaf(f, s_l[w][h], l);
      }
      if (a.splits == 1) {
        a.out[(head0 + h) * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : x / l);
        if (d == 0 && a.lse) a.lse[head0 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        float* q = a.part + (((static_cast<int64_t>(row) * gridDim.y + blockIdx.y) * a.splits +
                              blockIdx.x) * kHeadTile + h) * (D + 2);
        q[d] = x;
        if (d == 0) q[D] = m, q[D + 1] = l;
      }
    }
  };

  stream(0xffu);
  // With 16-bit values a head that does not keep a block still meets its V rows with weight 0, and
  // 0 * NaN or 0 * inf is not 0. That shows as a NaN: such a CTA goes over its entries once more for
  // each head alone, so that a head meets only blocks it keeps.
  if constexpr (!kQuant) {
    if (!a.share && nh > 1) {
      bool nan = false;
#pragma unroll
      for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) nan |= isnan(acc[n][e]);
      odd = __syncthreads_or(nan);
    }
  }
  if (!odd) {
    finish(0xffu);
  } else {
    for (int h = 0; h < nh; ++h) {
      stream(1u << h);
      finish(1u << h);
      __syncthreads();
    }
  }
}

// Joins the CTAs of each item: one CTA per (row, query head), a thread per channel.
template <int D>
__global__ void __launch_bounds__(D) join_kernel(const Args a) {
  const int row = blockIdx.y, head = blockIdx.x, d = threadIdx.x;
  const int G = a.r.Hq / a.c.Hkv, tiles_h = (G + kHeadTile - 1) / kHeadTile;
  const int item = head / G * tiles_h + head % G / kHeadTile, h = head % G % kHeadTile;
  const float* p = a.part + ((static_cast<int64_t>(row) * a.c.Hkv * tiles_h + item) * a.splits *
                                 kHeadTile + h) * (D + 2);
  const int64_t step = static_cast<int64_t>(kHeadTile) * (D + 2);
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, p[s * step + D]);
  const float base = m == -INFINITY ? 0.f : m;
  float x = 0.f, l = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float ms = p[s * step + D], ls = p[s * step + D + 1];
    if (ms == -INFINITY && ls == 0.f) continue;
    const float f = exp2f(ms - base);
    x = fmaf(f, p[s * step + d], x);
    l = fmaf(f, ls, l);
  }
  const int64_t o = static_cast<int64_t>(row) * a.r.Hq + head;
  a.out[o * D + d] = __float2bfloat16_rn(l == 0.f ? 0.f : x / l);
  if (d == 0 && a.lse) a.lse[o] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Split of the longest item's list over CTAs.
struct Split {
  int chunk, splits;
};
Split split_of(int Hkv, int max_blocks, int R, int Hq, int kcap, bool share) {
  const int G = Hq / Hkv;
  const int64_t items = static_cast<int64_t>(R) * Hkv * ((G + kHeadTile - 1) / kHeadTile);
  // entries of an item's list: one list, or the union of its heads' lists
  const int64_t most =
      share ? kcap : std::min<int64_t>(static_cast<int64_t>(std::min(G, kHeadTile)) * kcap,
                                       max_blocks);
  const int64_t target = 8 * static_cast<int64_t>(sm_count());
  int64_t chunk = std::max<int64_t>(1, most * items / target);
  Split s;
  s.chunk = static_cast<int>(chunk);
  s.splits = static_cast<int>((most + chunk - 1) / chunk);
  return s;
}

template <int FMT, int D>
cudaError_t launch(const Args& a, cudaStream_t st) {
  using C = Cfg<FMT, D>;
  const int G = a.r.Hq / a.c.Hkv;
  const size_t ring = static_cast<size_t>(kWarps) * C::RING;
  static_assert(C::RING >= kHeadTile * D * 4, "the rings hold the warps' results at the end");
  const size_t bytes = ring + 4 * static_cast<size_t>(a.chunk) + 4 * ((a.c.max_blocks + 3) / 4);
  // the attribute is per device; setting it is cheap and idempotent
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<FMT, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bytes));
  if (e != cudaSuccess) return e;
  const dim3 grid(a.splits, a.c.Hkv * ((G + kHeadTile - 1) / kHeadTile), a.r.R);
  attn_kernel<FMT, D><<<grid, kWarps * 32, bytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  join_kernel<D><<<dim3(a.r.Hq, a.r.R), D, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_attn(const KvCache& c, int format, int D, const DecodeRows& r, bool share,
                               void* out, float* lse, float* partials, cudaStream_t st) {
  const Split s = split_of(c.Hkv, c.max_blocks, r.R, r.Hq, r.kcap, share);
  const Args a{c,   r, share, s.chunk, s.splits, static_cast<__nv_bfloat16*>(out), lse,
               partials};
  if (D == 128) {
    switch (format) {
      case STEM_KV_BF16: return launch<STEM_KV_BF16, 128>(a, st);
      case STEM_KV_Q8: return launch<STEM_KV_Q8, 128>(a, st);
      default: return launch<STEM_KV_Q4, 128>(a, st);
    }
  }
  switch (format) {
    case STEM_KV_BF16: return launch<STEM_KV_BF16, 64>(a, st);
    case STEM_KV_Q8: return launch<STEM_KV_Q8, 64>(a, st);
    default: return launch<STEM_KV_Q4, 64>(a, st);
  }
}

size_t decode_attn_partials(int, int D, int Hkv, int max_blocks, int R, int Hq, int kcap,
                            bool share) {
  const Split s = split_of(Hkv, max_blocks, R, Hq, kcap, share);
  if (s.splits == 1) return 0;
  const int G = Hq / Hkv;
  return static_cast<size_t>(R) * Hkv * ((G + kHeadTile - 1) / kHeadTile) * s.splits * kHeadTile *
         (D + 2);
}

}  // namespace stem
