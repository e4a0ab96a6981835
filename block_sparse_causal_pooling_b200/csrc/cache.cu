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
// Bound: HBM (rows in, codes out). Measured (B200, device time in a graph, against the bytes at a copy's
// rate): writing a 128K prompt, 8 kv heads of 128, 195 us of 166 at 16 bits, 242 of 127 at 8 and 228 of
// 106 at 4, where packing the codes stands between a tile's loads and the next; 8 ragged chunks of up to
// 1999 tokens at 8 bits, 2 heads of 64, 15 us of 4, a chain of loads for little work a CTA. Reading the same:
// 161, 128 and 108 us, and 7. One token of 16 sequences at 4 bits 5.8 and 2.2 us. One CTA per (block, kv
// head, sequence); a thread holds the same 8 channels of a token pair of every tile.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "decode_internal.h"
#include "decode_launch.h"
#include "kv_layout.cuh"

namespace stem {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
__device__ __forceinline__ float bits_bf16(uint32_t b) { return __uint_as_float(b << 16); }

// Eight consecutive channels of one row as they are in memory, as float32, and their largest
// magnitude as the bits of a float32 (ordered like the numbers, with infinity and NaN on top).
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
  __device__ __forceinline__ uint32_t largest() const {
    constexpr uint32_t kMag = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & kMag, u.y & kMag), __vmaxu2(u.z & kMag, u.w & kMag));
    return max(m << 16, m & 0xffff0000u);
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
  __device__ __forceinline__ uint32_t largest() const {
    float x[8];
    get(x);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    return m;
  }
};

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

// Eight codes of a row and their scale. A 4- or 8-bit code c is held as the bits of the float32
// kMagic + c, kMagic = 1.5 * 2^23 + offset: adding kMagic rounds to an integer (ties to even), the
// bits are kBits + c + offset, and subtracting kMagic gives c as a float32 again. A 16-bit code is
// the bfloat16's bits.
constexpr uint32_t kBits = 0x4b400000u;  // 1.5 * 2^23
template <int FMT>
struct Codes {
  static constexpr float kMagic = 12582912.f + static_cast<float>(Kv<FMT, 128>::OFFSET);
  uint32_t b[8];
  uint32_t scale;  // bfloat16 bits

  __device__ __forceinline__ float code(int e) const {
    return FMT == STEM_KV_BF16 ? bits_bf16(b[e]) : __uint_as_float(b[e]) - kMagic;
  }
  __device__ __forceinline__ float value(int e) const {
    return FMT == STEM_KV_BF16 ? code(e) : bits_bf16(scale) * code(e);  // exact (8 + 7 bits)
  }
};

// Quantises the 8 channels of this thread; the group's other channels are in the 3 neighbouring
// lanes (a quad works on one row). Called by whole warps.
//
// The quotients are the correctly rounded ones without a division each (a division has a branch,
// which would run the 8 of them one after another): with r near 1/s, q0 = x r, e = x - q0 s (exact
// in an FMA) and q = q0 + e r is x / s but for 2^-46 of it before its rounding (Markstein's
// correction), and the quotient of a float32 by the 8 bits of s is never nearer than 2^-34 to a
// rounding border unless it is on one. The same holds for max|x| / Q. |x / s| <= Q 256/255 < Q + 1/2,
// so that codes need no clamp, while s is a normal number. Rows that are not within 2^+-50, or
// not finite, take the plain way.
template <int FMT, typename T>
__device__ __forceinline__ void quantise(const Raw<T>& raw, Codes<FMT>& c) {
  float x[8];
  raw.get(x);
  if constexpr (FMT == STEM_KV_BF16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c.b[e] = bf16_bits(x[e]);
    c.scale = 0;
  } else {
    constexpr float kTop = static_cast<float>(Kv<FMT, 128>::QMAX), kInv = 1.f / kTop;
    uint32_t top = raw.largest();
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    const float amax = __uint_as_float(top);
    // (0, or 2^-50 .. 2^50 as bits)
    if (__all_sync(kFull, top == 0 || top - 0x26800000u < 0x58800000u - 0x26800000u)) {
      const float t0 = amax * kInv;
      c.scale = bf16_bits(fmaf(fmaf(-t0, kTop, amax), kInv, t0));
      const float s = bits_bf16(c.scale);
      const float r = top == 0 ? 0.f : __frcp_rn(s);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q0 = x[e] * r;
        c.b[e] = __float_as_uint(fmaf(fmaf(-q0, s, x[e]), r, q0) + Codes<FMT>::kMagic);
      }
    } else {
      const bool finite = top < 0x7f800000u;
      c.scale = finite ? bf16_bits(__fdiv_rn(amax, kTop)) : 0x7fc0u;
      const float s = bits_bf16(c.scale);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float q = 0.f;
        if (finite && s > 0.f) q = fminf(fmaxf(__fdiv_rn(x[e], s), -kTop), kTop);
        c.b[e] = __float_as_uint(q + Codes<FMT>::kMagic);
      }
    }
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

// The WPG words of a lane's group are neighbours: moved at once.
template <int N>
__device__ __forceinline__ void load_words(const unsigned char* p, uint32_t (&w)[4]) {
  if constexpr (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <int N>
__device__ __forceinline__ void store_words(unsigned char* p, const uint32_t (&w)[4]) {
  if constexpr (N == 4)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 2)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

// sum of b[e] << shift, less what kBits adds: every code at its place in a word.
__device__ __forceinline__ constexpr uint32_t magic_sum() { return 0u; }
template <typename... S>
__device__ __forceinline__ constexpr uint32_t magic_sum(int shift, S... rest) {
  return (kBits << shift) + magic_sum(rest...);
}

template <int FMT>
__device__ __forceinline__ void k_words(const Codes<FMT>& c, uint32_t (&w)[4]) {
  const uint32_t(&b)[8] = c.b;
  if constexpr (FMT == STEM_KV_BF16) {
#pragma unroll
    for (int n = 0; n < 4; ++n) w[n] = b[2 * n] | b[2 * n + 1] << 16;
  } else if constexpr (FMT == STEM_KV_Q8) {
#pragma unroll
    for (int n = 0; n < 2; ++n)
      w[n] = b[4 * n] + (b[4 * n + 2] << 8) + (b[4 * n + 1] << 16) + (b[4 * n + 3] << 24) -
             magic_sum(0, 8, 16, 24);
  } else {
    w[0] = b[0] + (b[2] << 4) + (b[4] << 8) + (b[6] << 12) + (b[1] << 16) + (b[3] << 20) +
           (b[5] << 24) + (b[7] << 28) - magic_sum(0, 4, 8, 12, 16, 20, 24, 28);
  }
}
template <int FMT>
__device__ __forceinline__ void k_codes(const uint32_t (&w)[4], Codes<FMT>& c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (FMT == STEM_KV_BF16)
      c.b[e] = w[e / 2] >> (16 * (e % 2)) & 0xffffu;
    else if constexpr (FMT == STEM_KV_Q8)
      c.b[e] = (w[e / 4] >> (16 * (e % 2) + 8 * (e % 4 / 2)) & 0xffu) | kBits;
    else
      c.b[e] = (w[0] >> (16 * (e % 2) + 4 * (e / 2)) & 0xfu) | kBits;
  }
}
// The 16-bit halves (in the low bits) that one token has in the V words of channels 4h .. 4h + 3.
template <int FMT>
__device__ __forceinline__ void v_halves(const Codes<FMT>& c, int h, uint32_t (&w)[4]) {
  const uint32_t* b = c.b + 4 * h;
  if constexpr (FMT == STEM_KV_BF16) {
#pragma unroll
    for (int n = 0; n < 4; ++n) w[n] = b[n];
  } else if constexpr (FMT == STEM_KV_Q8) {
    w[0] = b[0] + (b[1] << 8) - magic_sum(0, 8);
    w[1] = b[2] + (b[3] << 8) - magic_sum(0, 8);
  } else {
    w[0] = b[0] + (b[1] << 4) + (b[2] << 8) + (b[3] << 12) - magic_sum(0, 4, 8, 12);
  }
}
template <int FMT>
__device__ __forceinline__ void v_codes(const uint32_t (&w)[4], int h, Codes<FMT>& c) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (FMT == STEM_KV_BF16)
      c.b[4 * h + e] = w[e];
    else if constexpr (FMT == STEM_KV_Q8)
      c.b[4 * h + e] = (w[e / 2] >> (8 * (e % 2)) & 0xffu) | kBits;
    else
      c.b[4 * h + e] = (w[0] >> (4 * e) & 0xfu) | kBits;
  }
}

// Scale bits of token 2 * pair + y in a tile: of its K group, or of its V group.
template <int FMT, int D>
__device__ __forceinline__ uint16_t* scale_at(unsigned char* tile, const Place<FMT, D>& at, int y,
                                              bool v) {
  using L = Kv<FMT, D>;
  return reinterpret_cast<uint16_t*>(tile + 2 * L::CODES + (2 * at.pair + y) * L::SCROW) +
         (v ? L::NG : 0) + at.g;
}

// What a pair's tokens have in a tile, as it is in memory.
template <int FMT, int D>
struct Stored {
  uint32_t k[2][4], v[2][4], sk[2], sv[2];

  __device__ __forceinline__ void load(unsigned char* tile, const Place<FMT, D>& at) {
    using L = Kv<FMT, D>;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      load_words<L::WPG>(tile + at.k(y, 0), k[y]);
      load_words<L::WPG>(tile + L::CODES + at.v(y, 0), v[y]);  // (of channels 4y .. 4y + 3)
      if constexpr (FMT != STEM_KV_BF16) {
        sk[y] = *scale_at(tile, at, y, false);
        sv[y] = *scale_at(tile, at, y, true);
      } else {
        sk[y] = sv[y] = 0;
      }
    }
  }
  // K, or V, codes of token y of the pair
  __device__ __forceinline__ void get_k(int y, Codes<FMT>& c) const {
    c.scale = sk[y];
    k_codes(k[y], c);
  }
  __device__ __forceinline__ void get_v(int y, Codes<FMT>& c) const {
    c.scale = sv[y];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
#pragma unroll
      for (int n = 0; n < Kv<FMT, D>::WPG; ++n) w[n] = v[h][n] >> (16 * y) & 0xffffu;
      v_codes(w, h, c);
    }
  }
};

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
// CTAs an SM. Loads of one CTA hide behind the others' work: with 2 and the next tile's rows loaded
// ahead a 128K prompt at 16 bits takes 377 us (written and read back), with 3 and none ahead 356.
constexpr int kAppendCtas = 3;

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kThreads, kAppendCtas)
    append_kernel(KvCache c_, Rows r, const T* k, const T* v) {
  using L = Kv<FMT, D>;
  constexpr int CH = D / 8;                    // chunks of a row
  constexpr int SLOTS = kThreads / (8 * CH);  // tiles at a time
  int page, first, lo, hi;
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  if (!my_block(c_, r, page, first, lo, hi)) return;
  const int head = blockIdx.y, slot = threadIdx.x / (8 * CH);
  const int pair = threadIdx.x / CH % 8, chunk = threadIdx.x % CH;
  const Place<FMT, D> at(pair, chunk);
  unsigned char* rec = c_.at(page, head);
  const int64_t base = static_cast<int64_t>(blockIdx.z) * r.s_seq +
                       static_cast<int64_t>(head) * r.s_head + chunk * 8;
  const bool done = hi == c_.block;  // the block is complete: all of its tokens are summarised
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
  for (; n < n_end; n += SLOTS) {  // (a warp has one slot: n is uniform in it)
    fetch(n);
    unsigned char* tile = rec + static_cast<int64_t>(n) * L::TILE_BYTES;
    const int t0 = n * kKvTile + 2 * pair;
    const bool fresh[2] = {t0 >= lo && t0 < hi, t0 + 1 >= lo && t0 + 1 < hi};
    const bool any = __any_sync(kFull, fresh[0] || fresh[1]);
    Codes<FMT> c[2];
    // tokens that came with earlier calls are read back where the block is summarised
    Stored<FMT, D> old;
    if (done && !(fresh[0] && fresh[1])) old.load(tile, at);
    __syncwarp();
    // ---- K
    if (any) {
      uint32_t w[4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        quantise(rk[y], c[y]);
        if (fresh[y]) {
          k_words(c[y], w);
          store_words<L::WPG>(tile + at.k(y, 0), w);
          if (FMT != STEM_KV_BF16 && at.q == 0)
            *scale_at(tile, at, y, false) = static_cast<uint16_t>(c[y].scale);
        }
      }
    }
    if (done) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (!fresh[y]) old.get_k(y, c[y]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          ksum[e] = FMT == STEM_KV_BF16 ? ksum[e] + c[y].code(e)
                                        : fmaf(bits_bf16(c[y].scale), c[y].code(e), ksum[e]);
      }
    }
    // ---- V
    if (any) {
      uint32_t hv[2][2][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        quantise(rv[y], c[y]);
        v_halves(c[y], 0, hv[y][0]);
        v_halves(c[y], 1, hv[y][1]);
        if (FMT != STEM_KV_BF16 && fresh[y] && at.q == 0)
          *scale_at(tile, at, y, true) = static_cast<uint16_t>(c[y].scale);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        unsigned char* dst = tile + L::CODES + at.v(h, 0);
        if (fresh[0] && fresh[1]) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < L::WPG; ++i) w[i] = hv[0][h][i] | hv[1][h][i] << 16;
          store_words<L::WPG>(dst, w);
        } else {
          // a lone token writes its halves and leaves the other token's as they are
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (fresh[y])
#pragma unroll
              for (int i = 0; i < L::WPG; ++i)
                *reinterpret_cast<uint16_t*>(dst + 4 * i + 2 * y) =
                    static_cast<uint16_t>(hv[y][h][i]);
        }
      }
    }
    if (done) {
      float norm[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (!fresh[y]) old.get_v(y, c[y]);
        float sq = 0.f;  // of codes: a sum of integers below 2^24, exact
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(c[y].code(e), c[y].code(e), sq);
        if (FMT != STEM_KV_BF16) {
          const float s = bits_bf16(c[y].scale);
          sq *= s * s;
        }
        norm[y] = sq;
      }
      __syncwarp();
#pragma unroll
      for (int d = 1; d < CH; d *= 2) {
        norm[0] += __shfl_xor_sync(kFull, norm[0], d);
        norm[1] += __shfl_xor_sync(kFull, norm[1], d);
      }
      const float n0 = sqrtf(norm[0]), n1 = sqrtf(norm[1]);
      if (c_.vmax) {  // (NaN stays: a comparison with it is false)
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
  const int64_t ph = static_cast<int64_t>(page) * c_.Hkv + head;
  if (threadIdx.x < D) {
    const int d = threadIdx.x;
    float s[P];
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = ks[i][d];
#pragma unroll
    for (int o = 1; o < P; o *= 2)
#pragma unroll
      for (int i = 0; i < P; i += 2 * o) s[i] += s[i + o];
    c_.kbar[ph * D + d] = s[0] / static_cast<float>(c_.block);
  } else if (threadIdx.x == D) {
    float s = vs[0];
    for (int i = 1; i < P; ++i) {
      if (c_.vmax)
        s = s > vs[i] || isnan(s) ? s : vs[i];
      else
        s += vs[i];
    }
    c_.vnorm[ph] = c_.vmax ? s : s / static_cast<float>(c_.block);
  }
}

// A CTA reads kReadTiles tiles, each thread its words of one tile at a time.
constexpr int kReadTiles = 2;

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(8 * (D / 8)) read_kernel(KvCache c_, Rows r, T* k, T* v) {
  using L = Kv<FMT, D>;
  constexpr int CH = D / 8;
  int page, first, lo, hi;
  const int parts = c_.block / (kReadTiles * kKvTile);
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
  if (!my_block(c_, r, page, first, lo, hi, parts)) return;
  const int head = blockIdx.y, pair = threadIdx.x / CH, chunk = threadIdx.x % CH;
  const Place<FMT, D> at(pair, chunk);
  unsigned char* rec = c_.at(page, head);
  const int64_t base = static_cast<int64_t>(blockIdx.z) * r.s_seq +
                       static_cast<int64_t>(head) * r.s_head + chunk * 8;
  const int n0 = blockIdx.x % parts * kReadTiles;
#pragma unroll
  for (int i = 0; i < kReadTiles; ++i) {
    const int t0 = (n0 + i) * kKvTile + 2 * pair;
    const bool live[2] = {t0 >= lo && t0 < hi, t0 + 1 >= lo && t0 + 1 < hi};
    if (!live[0] && !live[1]) continue;
    unsigned char* tile = rec + static_cast<int64_t>(n0 + i) * L::TILE_BYTES;
    Stored<FMT, D> got;
    got.load(tile, at);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (!live[y]) continue;
      const int64_t o = base + static_cast<int64_t>(first + t0 + y) * r.s_tok;
      Codes<FMT> c;
      float x[8];
      got.get_k(y, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = c.value(e);
      store8(k + o, x);
      got.get_v(y, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = c.value(e);
      store8(v + o, x);
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
