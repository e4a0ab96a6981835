// The paged K/V cache's writer and reader (stem_cache_append, stem_cache_read).
//
// Writing quantises each row once, as it arrives: with x the 32 channels of a group,
//   s = bf16(max|x| / Q), c = clamp(rint(x / s), -Q, Q), the value it stands for is s * c.
// s and x are bfloat16 (8 significant bits), so x / s is either a tie or at least 2^-17 away from
// one, relative to its size: the correctly rounded float32 quotient gives the code that real
// arithmetic gives. float32 inputs take the same float32 quotient as their definition.
//
// A block's summaries (kbar, vnorm) are computed by the call that writes its last token, from the
// values that the cache stands for, in an order that depends on token positions alone: tokens that
// came with earlier calls are read back from the page. So the summaries are the same bits whether
// a block came at once or token by token, and writing a position again gives what writing it once
// gives.
//
// Bound: HBM (rows in, codes out). One CTA per (block, kv head, sequence); a thread holds the same
// 8 channels of a token pair of every tile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "decode_internal.h"
#include "decode_launch.h"
#include "kv_layout.cuh"

namespace stem {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Eight consecutive channels of one row as they are in memory, and as float32.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      x[2 * n] = __uint_as_float(w[n] << 16);
      x[2 * n + 1] = __uint_as_float(w[n] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ float bits_bf16(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) w[n] = bf16_bits(x[2 * n]) | bf16_bits(x[2 * n + 1]) << 16;
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

// Quantises the 8 channels of this thread; the group's other channels are in the 3 neighbouring
// lanes (a quad works on one row). x becomes the values that the codes stand for; code[] holds
// offset codes (bfloat16 bits for the 16-bit format), the return value the scale's bits.
//
// The quotients are the correctly rounded ones without a division each (a division has a branch,
// which would run the 8 of them one after another: 7 us a tile where this takes a fraction): with
// r = 1/s correctly rounded, q0 = x r, e = x - q0 s (exact in an FMA) and q = q0 + e r is the
// rounded x / s (Markstein's correction). Powers of two keep x and s away from the range's ends.
// max|x| / Q is rounded once from the double product with 1/Q: 24 bits over 7 or 127 are never
// nearer than 2^-32 to a float32 tie unless they are one.
template <int FMT>
__device__ __forceinline__ uint32_t quantise(float (&x)[8], uint32_t (&code)[8]) {
  if constexpr (FMT == STEM_KV_BF16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      code[e] = bf16_bits(x[e]);
      x[e] = bits_bf16(code[e]);
    }
    return 0;
  } else {
    using L = Kv<FMT, 128>;
    constexpr float kTop = static_cast<float>(L::QMAX);
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
    // magnitudes as integers: ordered like the numbers, with infinity and NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    const bool finite = top < 0x7f800000u;
    const float largest = static_cast<float>(static_cast<double>(__uint_as_float(top)) *
                                             (1.0 / static_cast<double>(L::QMAX)));
    const uint32_t sb = finite ? bf16_bits(largest) : 0x7fc0u;
    const float s = bits_bf16(sb);
    const float pow2 = s < 0x1p-60f ? 0x1p64f : s > 0x1p60f ? 0x1p-64f : 1.f;
    const float ss = finite ? s * pow2 : 0.f;
    const float r = s > 0.f && finite ? __frcp_rn(ss) : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = finite ? x[e] * pow2 : 0.f;
      const float q0 = y * r;
      float q = fmaf(fmaf(-q0, ss, y), r, q0);
      q = fminf(fmaxf(q, -kTop), kTop) + kMagic;
      x[e] = s * (q - kMagic);  // exact (at most 8 + 7 bits); NaN for a group that is not finite
      code[e] = __float_as_uint(q) - __float_as_uint(kMagic) + L::OFFSET;
    }
    return sb;
  }
}

// Where thread (pair, chunk) of a tile finds its codes. chunk c holds channels 8c .. 8c + 7:
// group c / 4; as K they are lane column c % 4, as V the lane rows 2 (c % 4) and 2 (c % 4) + 1.
template <int FMT, int D>
struct Place {
  using L = Kv<FMT, D>;
  int pair, g, q;
  __device__ Place(int pair_, int chunk) : pair(pair_), g(chunk / 4), q(chunk % 4) {}

  // K words of token 2 * pair + y
  __device__ __forceinline__ int k(int y, int w) const {
    const int r = 2 * pair + y;
    return L::word(r / 8, g, w, (r % 8) * 4 + q);
  }
  // V words of the pair, channels 4h .. 4h + 3 of the chunk (h = 0, 1)
  __device__ __forceinline__ int v(int h, int w) const {
    return L::word(pair / 4, g, w, (2 * q + h) * 4 + pair % 4);
  }
};

template <int FMT>
__device__ __forceinline__ void k_words(const uint32_t (&c)[8], uint32_t (&w)[4]) {
  if constexpr (FMT == STEM_KV_BF16) {
#pragma unroll
    for (int n = 0; n < 4; ++n) w[n] = c[2 * n] | c[2 * n + 1] << 16;
  } else if constexpr (FMT == STEM_KV_Q8) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
      w[n] = c[4 * n] | c[4 * n + 2] << 8 | c[4 * n + 1] << 16 | c[4 * n + 3] << 24;
  } else {
    w[0] = c[0] | c[2] << 4 | c[4] << 8 | c[6] << 12 | c[1] << 16 | c[3] << 20 | c[5] << 24 |
           c[7] << 28;
  }
}
template <int FMT>
__device__ __forceinline__ void k_codes(const uint32_t (&w)[4], uint32_t (&c)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (FMT == STEM_KV_BF16)
      c[e] = w[e / 2] >> (16 * (e % 2)) & 0xffffu;
    else if constexpr (FMT == STEM_KV_Q8)
      c[e] = w[e / 4] >> (16 * (e % 2) + 8 * (e % 4 / 2)) & 0xffu;
    else
      c[e] = w[0] >> (16 * (e % 2) + 4 * (e / 2)) & 0xfu;
  }
}
// The 16-bit halves that one token has in the V words of 4 channels.
template <int FMT>
__device__ __forceinline__ void v_halves(const uint32_t* c, uint32_t (&h)[4]) {
  if constexpr (FMT == STEM_KV_BF16) {
#pragma unroll
    for (int n = 0; n < 4; ++n) h[n] = c[n];
  } else if constexpr (FMT == STEM_KV_Q8) {
    h[0] = c[0] | c[1] << 8;
    h[1] = c[2] | c[3] << 8;
  } else {
    h[0] = c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12;
  }
}
template <int FMT>
__device__ __forceinline__ void v_codes(const uint32_t (&h)[4], uint32_t* c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (FMT == STEM_KV_BF16)
      c[e] = h[e];
    else if constexpr (FMT == STEM_KV_Q8)
      c[e] = h[e / 2] >> (8 * (e % 2)) & 0xffu;
    else
      c[e] = h[0] >> (4 * e) & 0xfu;
  }
}

template <int FMT>
__device__ __forceinline__ void values(const uint32_t (&c)[8], uint32_t scale, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (FMT == STEM_KV_BF16)
      x[e] = bits_bf16(c[e]);
    else
      x[e] = bits_bf16(scale) * static_cast<float>(static_cast<int>(c[e]) - Kv<FMT, 128>::OFFSET);
  }
}

// K and V values of the pair's tokens y = 0, 1 from a tile in memory.
template <int FMT, int D>
__device__ __forceinline__ void read_pair(const unsigned char* tile, const Place<FMT, D>& at,
                                          float (&xk)[2][8], float (&xv)[2][8]) {
  using L = Kv<FMT, D>;
  uint32_t vw[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int w = 0; w < L::WPG; ++w)
      vw[h][w] = *reinterpret_cast<const uint32_t*>(tile + L::CODES + at.v(h, w));
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    uint32_t sk = 0, sv = 0;
    if constexpr (FMT != STEM_KV_BF16) {
      const unsigned char* row = tile + 2 * L::CODES + (2 * at.pair + y) * L::SCROW;
      sk = *reinterpret_cast<const uint16_t*>(row + 2 * at.g);
      sv = *reinterpret_cast<const uint16_t*>(row + 2 * (L::NG + at.g));
    }
    uint32_t kw[4] = {0, 0, 0, 0}, c[8];
#pragma unroll
    for (int w = 0; w < L::WPG; ++w)
      kw[w] = *reinterpret_cast<const uint32_t*>(tile + at.k(y, w));
    k_codes<FMT>(kw, c);
    values<FMT>(c, sk, xk[y]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t hv[4];
#pragma unroll
      for (int w = 0; w < L::WPG; ++w) hv[w] = vw[h][w] >> (16 * y) & 0xffffu;
      v_codes<FMT>(hv, c + 4 * h);
    }
    values<FMT>(c, sv, xv[y]);
  }
}

struct Rows {
  const int32_t* pos;    // first token of each sequence's rows
  const int32_t* count;  // rows of each sequence, NULL: T
  int T;
  int64_t s_seq, s_head, s_tok;  // strides of k and v, in elements
  int32_t* status;
};

// The block this CTA works on: tokens [lo, hi) of its page. False: nothing to do.
// `parts`: CTAs of a block.
__device__ __forceinline__ bool my_block(const KvCache& c, const Rows& r, int& page, int& first,
                                         int& lo, int& hi, int parts = 1) {
  const int seq = blockIdx.z;
  int j;
  if (!kv_block_rows(c, r.pos[seq], r.count ? r.count[seq] : r.T, r.T, blockIdx.x / parts,
                     r.status, j, first, lo, hi))
    return false;
  page = kv_page(c, seq, j, r.status);
  return page >= 0;
}

constexpr int kThreads = 256;

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(KvCache c, Rows r, const T* k,
                                                          const T* v) {
  using L = Kv<FMT, D>;
  constexpr int CH = D / 8;                    // chunks of a row
  constexpr int SLOTS = kThreads / (8 * CH);  // tiles at a time
  int page, first, lo, hi;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  if (!my_block(c, r, page, first, lo, hi)) return;
  const int head = blockIdx.y, slot = threadIdx.x / (8 * CH);
  const int pair = threadIdx.x / CH % 8, chunk = threadIdx.x % CH;
  const Place<FMT, D> at(pair, chunk);
  unsigned char* rec = c.at(page, head);
  const int64_t base = static_cast<int64_t>(blockIdx.z) * r.s_seq +
                       static_cast<int64_t>(head) * r.s_head + chunk * 8;
  const bool done = hi == c.block;  // the block is complete: all of its tokens are summarised
  float ksum[8] = {0, 0, 0, 0, 0, 0, 0, 0}, vacc = 0.f;
  const int n_end = (hi - 1) / kKvTile + 1;
  // tiles of a thread are n0, n0 + SLOTS, ..: an order that depends on token positions alone
  int n = (done ? 0 : lo / kKvTile) + slot;
  Raw<T> rk[2], rv[2];
  auto fetch = [&](int tile) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int t = tile * kKvTile + 2 * pair + y;
      if (t >= lo && t < hi) {
        const int64_t o = base + static_cast<int64_t>(first + t) * r.s_tok;
        rk[y].load(k + o);
        rv[y].load(v + o);
      } else {
        rk[y].zero();
        rv[y].zero();
      }
    }
  };
  fetch(n);
  for (; n < n_end; n += SLOTS) {  // (a warp has one slot: n is uniform in it)
    unsigned char* tile = rec + static_cast<int64_t>(n) * L::TILE_BYTES;
    const int t0 = n * kKvTile + 2 * pair;
    bool fresh[2];
    float xk[2][8], xv[2][8];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      fresh[y] = t0 + y >= lo && t0 + y < hi;
      rk[y].get(xk[y]);
      rv[y].get(xv[y]);
    }
    fetch(n + SLOTS);
    if (__any_sync(kFull, fresh[0] || fresh[1])) {
      uint32_t hv[2][2][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t ck[8], cv[8], kw[4];
        const uint32_t sk = quantise<FMT>(xk[y], ck), sv = quantise<FMT>(xv[y], cv);
        v_halves<FMT>(cv, hv[y][0]);
        v_halves<FMT>(cv + 4, hv[y][1]);
        if (fresh[y]) {
          k_words<FMT>(ck, kw);
          if constexpr (FMT == STEM_KV_BF16) {
            *reinterpret_cast<uint4*>(tile + at.k(y, 0)) = make_uint4(kw[0], kw[1], kw[2], kw[3]);
          } else {
#pragma unroll
            for (int w = 0; w < L::WPG; ++w)
              *reinterpret_cast<uint32_t*>(tile + at.k(y, w)) = kw[w];
            if (at.q == 0) {
              unsigned char* row = tile + 2 * L::CODES + (2 * pair + y) * L::SCROW;
              *reinterpret_cast<uint16_t*>(row + 2 * at.g) = static_cast<uint16_t>(sk);
              *reinterpret_cast<uint16_t*>(row + 2 * (L::NG + at.g)) = static_cast<uint16_t>(sv);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned char* dst = tile + L::CODES;
        if (fresh[0] && fresh[1]) {
          uint32_t w4[4];
#pragma unroll
          for (int w = 0; w < L::WPG; ++w) w4[w] = hv[0][h][w] | hv[1][h][w] << 16;
          if constexpr (FMT == STEM_KV_BF16) {
            *reinterpret_cast<uint4*>(dst + at.v(h, 0)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
          } else {
#pragma unroll
            for (int w = 0; w < L::WPG; ++w)
              *reinterpret_cast<uint32_t*>(dst + at.v(h, w)) = w4[w];
          }
        } else {
          // a lone token writes its halves and leaves the other token's as they are
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (fresh[y])
#pragma unroll
              for (int w = 0; w < L::WPG; ++w)
                *reinterpret_cast<uint16_t*>(dst + at.v(h, w) + 2 * y) =
                    static_cast<uint16_t>(hv[y][h][w]);
        }
      }
    }
    if (done) {
      if (!(fresh[0] && fresh[1])) {  // tokens that came with earlier calls
        float ok[2][8], ov[2][8];
        read_pair<FMT, D>(tile, at, ok, ov);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (!fresh[y])
#pragma unroll
            for (int e = 0; e < 8; ++e) xk[y][e] = ok[y][e], xv[y][e] = ov[y][e];
      }
      __syncwarp();
      float sq[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ksum[e] += xk[0][e] + xk[1][e];
        sq[0] = fmaf(xv[0][e], xv[0][e], sq[0]);
        sq[1] = fmaf(xv[1][e], xv[1][e], sq[1]);
      }
#pragma unroll
      for (int o = 1; o < CH; o *= 2) {
        sq[0] += __shfl_xor_sync(kFull, sq[0], o);
        sq[1] += __shfl_xor_sync(kFull, sq[1], o);
      }
      const float n0 = sqrtf(sq[0]), n1 = sqrtf(sq[1]);
      if (c.vmax) {  // (NaN stays: a comparison with it is false)
        const float m = n0 > n1 || isnan(n0) ? n0 : n1;
        vacc = vacc > m || isnan(vacc) ? vacc : m;
      } else {
        vacc += n0 + n1;
      }
    }
  }
  if (!done) return;
  // the sums of the slots' pairs, in a fixed order
  constexpr int P = 8 * SLOTS;
  __shared__ float ks[P][D];
  __shared__ float vs[P];
  const int part = slot * 8 + pair;
#pragma unroll
  for (int e = 0; e < 8; e += 4)
    *reinterpret_cast<float4*>(&ks[part][chunk * 8 + e]) =
        make_float4(ksum[e], ksum[e + 1], ksum[e + 2], ksum[e + 3]);
  if (chunk == 0) vs[part] = vacc;
  __syncthreads();
  const int64_t ph = static_cast<int64_t>(page) * c.Hkv + head;
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    float s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = ks[i][d];
#pragma unroll
    for (int o = 1; o < P; o *= 2)
#pragma unroll
      for (int i = 0; i < P; i += 2 * o) s[i] += s[i + o];
    c.kbar[ph * D + d] = s[0] / static_cast<float>(c.block);
  } else if (threadIdx.x == D) {
    float s = vs[0];
    for (int i = 1; i < P; ++i) {
      if (c.vmax)
        s = s > vs[i] || isnan(s) ? s : vs[i];
      else
        s += vs[i];
    }
    c.vnorm[ph] = c.vmax ? s : s / static_cast<float>(c.block);
  }
}

// A CTA reads kReadTiles tiles, each thread its words of one tile at a time.
constexpr int kReadTiles = 4;

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(8 * (D / 8)) read_kernel(KvCache c, Rows r, T* k, T* v) {
  using L = Kv<FMT, D>;
  constexpr int CH = D / 8;
  int page, first, lo, hi;
  const int parts = c.block / (kReadTiles * kKvTile);
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  if (!my_block(c, r, page, first, lo, hi, parts)) return;
  const int head = blockIdx.y, pair = threadIdx.x / CH, chunk = threadIdx.x % CH;
  const Place<FMT, D> at(pair, chunk);
  const unsigned char* rec = c.at(page, head);
  const int64_t base = static_cast<int64_t>(blockIdx.z) * r.s_seq +
                       static_cast<int64_t>(head) * r.s_head + chunk * 8;
  const int n0 = blockIdx.x % parts * kReadTiles;
#pragma unroll
  for (int i = 0; i < kReadTiles; ++i) {
    const int t0 = (n0 + i) * kKvTile + 2 * pair;
    const bool live[2] = {t0 >= lo && t0 < hi, t0 + 1 >= lo && t0 + 1 < hi};
    if (!live[0] && !live[1]) continue;
    float xk[2][8], xv[2][8];
    read_pair<FMT, D>(rec + static_cast<int64_t>(n0 + i) * L::TILE_BYTES, at, xk, xv);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (!live[y]) continue;
      const int64_t o = base + static_cast<int64_t>(first + t0 + y) * r.s_tok;
      store8(k + o, xk[y]);
      store8(v + o, xv[y]);
    }
  }
}

template <int FMT, int D, typename T>
cudaError_t launch(bool write, const KvCache& c, const Rows& r, void* k, void* v,
                   cudaStream_t st) {
  // blocks that T tokens can touch, from any offset in the first
  const unsigned nblk = static_cast<unsigned>((r.T + c.block - 2) / c.block + 1);
  const unsigned parts = write ? 1 : c.block / (kReadTiles * kKvTile);
  const dim3 grid(nblk * parts, c.Hkv, c.nseq);
  return write ? launch_after(append_kernel<FMT, D, T>, grid, kThreads, 0, 1, st, c, r,
                              static_cast<const T*>(k), static_cast<const T*>(v))
               : launch_after(read_kernel<FMT, D, T>, grid, 8 * (D / 8), 0, 1, st, c, r,
                              static_cast<T*>(k), static_cast<T*>(v));
}

template <int FMT, int D>
cudaError_t by_type(bool write, int dtype, const KvCache& c, const Rows& r, void* k, void* v,
                    cudaStream_t st) {
  return dtype == STEM_BF16 ? launch<FMT, D, __nv_bfloat16>(write, c, r, k, v, st)
                            : launch<FMT, D, float>(write, c, r, k, v, st);
}

template <int FMT>
cudaError_t by_dim(bool write, int D, int dtype, const KvCache& c, const Rows& r, void* k, void* v,
                   cudaStream_t st) {
  return D == 128 ? by_type<FMT, 128>(write, dtype, c, r, k, v, st)
                  : by_type<FMT, 64>(write, dtype, c, r, k, v, st);
}

}  // namespace

cudaError_t launch_cache_rows(bool write, int format, int D, int dtype, const KvCache& c, void* k,
                              void* v, int T, int64_t s_seq, int64_t s_head, int64_t s_tok,
                              const int32_t* pos, const int32_t* count, int32_t* status,
                              cudaStream_t st) {
  const Rows r{pos, count, T, s_seq, s_head, s_tok, status};
  switch (format) {
    case STEM_KV_BF16: return by_dim<STEM_KV_BF16>(write, D, dtype, c, r, k, v, st);
    case STEM_KV_Q8: return by_dim<STEM_KV_Q8>(write, D, dtype, c, r, k, v, st);
    default: return by_dim<STEM_KV_Q4>(write, D, dtype, c, r, k, v, st);
  }
}

}  // namespace stem
