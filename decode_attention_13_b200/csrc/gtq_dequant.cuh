// Packed tiles to fp16 matrix operands in shared memory, for the tcgen05
// kernels that attend over the packed cache.
//
// Eight warps share a tile.  Keys: rows = tokens, columns = packed coordinates
// (slot s: columns 2s, 2s + 1), K-major with the 128-byte swizzle in two atoms of 64
// columns; a warp takes four neighbouring slots at a time, a lane one of them for tokens g,
// g + 8, ..., g + 56 (g = lane % 8): with the swizzle its 4-byte stores fall into 32
// different banks.  Values: rows = rotated dims, columns = the tile's 64 tokens, one
// swizzled atom; a warp takes 16 dims, a lane two of them for 16 tokens.
//
// An element is cb[code] / 8 * norm, the factor undone in the queries and at the end.  It shares
// out fp16's range: the largest norm (65504) times the largest centroid (4.61) stays within it,
// and so does a query's coordinate (query_scale).  fp16 ends at 2^-24, so an element is good to 2^-25
// at best: that counts where all norms of a head are small, below about 2^-8 for one fp16 an element
// and below about 1 for two.  Where low parts have to hold to their last bits (FINE), the codebook's
// stay as they are and take norm / 8 instead: an 8th of them is an fp16 subnormal, off by up to 2^-22 of
// the norm.  (Not where other roundings to fp16 stand beside them: it costs a chunk 1.5% of its time.)
//
// Keys of widths up to 4 take a pair of codes in one lookup, every lane by its own
// width (mask, table, multiplier), so that four slots of different widths run as
// one instruction stream (code per width, one after another for the widths of a
// warp, made a chunk of 512 rows 1.09 times slower).  Wider codes, and slots that leave a low part, are
// looked up one by one.  All lookups of a portion come before its stores: a load may
// not pass a store whose address the compiler cannot tell apart.
#pragma once

#include "gtq_internal.h"
#include "gtq_tc.cuh"

namespace gtq {

constexpr float kElement = 0.125f;  // an operand's element: this times cb[code] times norm

// Lookup tables in shared memory (fp16 values of the codebook / 8): pair tables of
// widths 3, 2, 1 with a copy per lane, as they lie in the decode image (kTabP32W3
// .. kTabS32W5), a pair table of width 4 in one copy, single codes of all widths
// (kTabSS: hi | lo << 16; FINE: the low parts not divided), and a zero.
constexpr uint32_t kDqPairs = 0;
constexpr uint32_t kDqPairBytes = kTabS32W5 - kTabP32W3;
constexpr uint32_t kDqPair4 = kDqPairs + kDqPairBytes;
constexpr uint32_t kDqSingles = kDqPair4 + 1024u;
constexpr uint32_t kDqZero = kDqSingles + 2048u;
constexpr uint32_t kDqBytes = kDqZero + 128u;
static_assert(kDqBytes % 128 == 0, "dequantisation tables");

__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Copies the tables from the decode image (all threads of the block).
template <bool FINE>
__device__ __forceinline__ void load_dequant_tables(uint8_t* tab, const uint4* image, int tid,
                                                    int n_threads) {
  const uint8_t* img = reinterpret_cast<const uint8_t*>(image);
  const uint32_t* ss = reinterpret_cast<const uint32_t*>(img + kTabSS);
  const uint32_t* pp = reinterpret_cast<const uint32_t*>(img + kTabP32W3);
  auto scaled = [](uint32_t v) { return as_u32(__hmul2(as_h2(v), __float2half2_rn(kElement))); };
  for (int i = tid; i < (int)(kDqPairBytes / 4); i += n_threads)
    reinterpret_cast<uint32_t*>(tab + kDqPairs)[i] = scaled(pp[i]);
  for (int i = tid; i < 512; i += n_threads)
    reinterpret_cast<uint32_t*>(tab + kDqSingles)[i] = as_u32(__hmul2(as_h2(ss[i]), __floats2half2_rn(kElement, FINE ? 1.f : kElement)));
  for (int i = tid; i < 256; i += n_threads)
    reinterpret_cast<uint32_t*>(tab + kDqPair4)[i] =
        scaled(__byte_perm(ss[kSingleOff(4) / 4 + (i & 15)], ss[kSingleOff(4) / 4 + (i >> 4)], 0x5410));
  if (tid < 32) reinterpret_cast<uint32_t*>(tab + kDqZero)[tid] = 0;
}

// The low parts of the pair tables, laid out as the tables themselves (their single codes left out).
__device__ __forceinline__ void load_dequant_tables_lo(uint8_t* tab, const uint4* image, int tid, int n_threads) {
  const uint32_t* ss = reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint8_t*>(image) + kTabSS);
  auto pair = [&](int w, int i) {
    const uint32_t* e = ss + kSingleOff(w) / 4;
    return __byte_perm(e[i & ((1 << w) - 1)], e[i >> w], 0x7632);
  };
#pragma unroll
  for (int w = 1; w <= 3; ++w)
    for (int i = tid; i < (32 << (2 * w)); i += n_threads)
      reinterpret_cast<uint32_t*>(tab + kDqPairs + (kTabP32(w) - kTabP32W3))[i] = pair(w, i >> 5);
  for (int i = tid; i < 256; i += n_threads) reinterpret_cast<uint32_t*>(tab + kDqPair4)[i] = pair(4, i);
  if (tid < 32) reinterpret_cast<uint32_t*>(tab + kDqZero)[tid] = 0;
}

// From the lookup tables, which never change: the compiler may move it anywhere.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// Codes and norms from the cache.  Volatile: the compiler may not move these loads to their use,
// a whole tile later (it did, and every tile then waited for the memory).
__device__ __forceinline__ uint32_t ldg32(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ldg128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v));
}

// Bits [P, P + N) of the word array x, moved to bits [S, S + N) of the result
// (the other bits 0).
template <int P, int N, int S>
__device__ __forceinline__ uint32_t field(const uint32_t* x) {
  constexpr int i = P >> 5, sh = P & 31;
  constexpr uint32_t mask = (N >= 32 ? 0xffffffffu : ((1u << N) - 1)) << S;
  if constexpr (sh + N <= 32) {
    if constexpr (sh >= S) return (x[i] >> (sh - S)) & mask;
    else return (x[i] << (S - sh)) & mask;
  } else {
    static_assert(sh >= S, "field crosses a word below its place");
    return __funnelshift_r(x[i], x[i + 1], sh - S) & mask;
  }
}

// Code I of width W in the words x: its entry (fp16 hi | lo << 16).
template <int W, int I>
__device__ __forceinline__ uint32_t single(const uint32_t* x, uint32_t tab) {
  return lds32(tab + kDqSingles + kSingleOff(W) + field<I * W, W, 2>(x));
}

// fp16 pair (codes 2 U, 2 U + 1 of width W), hi parts.
template <int W, int U>
__device__ __forceinline__ uint32_t code_pair_hi(const uint32_t* x, uint32_t tab, uint32_t lane4) {
  if constexpr (W <= 3)
    return lds32(tab + kDqPairs + (kTabP32(W) - kTabP32W3) + (field<2 * U * W, 2 * W, 7>(x) | lane4));
  else if constexpr (W == 4)
    return lds32(tab + kDqPair4 + field<8 * U, 8, 2>(x));
  else
    return __byte_perm(single<W, 2 * U>(x, tab), single<W, 2 * U + 1>(x, tab), 0x5410);
}

// A lane's slot among four (4 quad .. 4 quad + 3) of a tile's keys.
struct KeyLane {
  uint32_t src;      // byte offset of its portion in the tile
  uint32_t sn;       // of its norms
  uint32_t col;      // of its pair in the operand: row g, swizzled column
  uint32_t w;        // width (0: no code)
  uint32_t base;     // lookup of a pair (widths up to 4): base + index * step
  uint32_t step;
};
__device__ __forceinline__ KeyLane key_lane(const HeadMeta& m, int quad, int lane, uint32_t atom,
                                            uint32_t norms, uint32_t tab) {
  const int g = lane & 7, s = 4 * quad + (lane >> 3);
  const uint32_t lane4 = 4u * (uint32_t)lane;
  KeyLane k;
  k.w = m.slot_width[s];
  k.src = k.w ? m.slot_koff[s] + 2u * (k.w * g) : 0u;
  k.sn = norms + (k.w ? 128u * m.slot_group[s] : 0u) + 16u * (uint32_t)g;
  k.col = (s >> 5) * atom + 128u * (uint32_t)g + (uint32_t)((((s >> 2) & 7) ^ g) << 4) + 4u * (uint32_t)(s & 3);
  k.step = k.w == 4 ? 4u : 128u;
  k.base = tab + (k.w == 1   ? kDqPairs + (kTabP32W1 - kTabP32W3) + lane4
                  : k.w == 2 ? kDqPairs + (kTabP32W2 - kTabP32W3) + lane4
                  : k.w == 3 ? kDqPairs + lane4
                  : k.w == 4 ? kDqPair4
                             : kDqZero);
  return k;
}

// Words and norms of a portion as they come from a tile: 2 words from the one that
// its first byte lies in for widths up to 4, 5 for any (the words behind a portion
// are inside the tile).
struct KeyRaw {
  uint32_t x[5];
  uint4 n;
};
template <int NW>
__device__ __forceinline__ void load_keys(KeyRaw& r, const uint8_t* tile, const KeyLane& k) {
  const uint8_t* p = tile + (k.src & ~3u);
#pragma unroll
  for (int i = 0; i < NW; ++i) r.x[i] = ldg32(p + 4 * i);
  r.n = ldg128(tile + k.sn);
}

// Widths up to 4, no low parts: four of the portion's 8 pairs are 8 w bits, at most a word.  dst:
// the operand's row of the tile's first token.
__device__ __forceinline__ void keys_by_pair(const KeyLane& k, const KeyRaw& r, uint32_t dst) {
  const uint32_t w2 = 2 * k.w, odd = (k.src & 2u) * 8u, mask = (1u << w2) - 1;
  uint32_t x[2];
  x[0] = __funnelshift_r(r.x[0], r.x[1], odd);
  x[1] = __funnelshift_rc(x[0], r.x[1] >> odd, 4 * w2);
  uint32_t v[8];
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i + u] = lds32((x[i] & mask) * k.step + k.base);
      x[i] >>= w2;
    }
  const uint32_t nw[4] = {r.n.x, r.n.y, r.n.z, r.n.w};
  const uint32_t d = dst + k.col;
#pragma unroll
  for (int u = 0; u < 8; u += 2) {
    const __half2 n = as_h2(nw[u >> 1]);
    sts32(d + 1024 * u, as_u32(__hmul2(as_h2(v[u]), __low2half2(n))));
    sts32(d + 1024 * (u + 1), as_u32(__hmul2(as_h2(v[u + 1]), __high2half2(n))));
  }
}

// The same with the products' rests beyond fp16 (fp16 hi + lo of the codebook in two tables `lo_tab`
// bytes apart), `lo_dst` bytes behind the pair itself.
__device__ __forceinline__ void keys_by_pair_split(const KeyLane& k, const KeyRaw& r, uint32_t dst,
                                                   uint32_t lo_tab, uint32_t lo_dst) {
  const uint32_t w2 = 2 * k.w, odd = (k.src & 2u) * 8u, mask = (1u << w2) - 1;
  uint32_t x[2];
  x[0] = __funnelshift_r(r.x[0], r.x[1], odd);
  x[1] = __funnelshift_rc(x[0], r.x[1] >> odd, 4 * w2);
  const uint32_t nw[4] = {r.n.x, r.n.y, r.n.z, r.n.w};
  const __half2 eighth = __float2half2_rn(kElement);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t v[4], l[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t at = (x[i] & mask) * k.step + k.base;
      v[u] = lds32(at);
      l[u] = lds32(at + lo_tab);
      x[i] >>= w2;
    }
    const uint32_t d = dst + k.col + 4096 * i;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const __half2 n = as_h2(nw[2 * i + (u >> 1)]), nn = (u & 1) ? __high2half2(n) : __low2half2(n);
      const __half2 p = __hmul2(as_h2(v[u]), nn);
      sts32(d + 1024 * u, as_u32(p));
      sts32(d + 1024 * u + lo_dst,
            as_u32(__hfma2(as_h2(l[u]), __hmul2(nn, eighth), __hfma2(as_h2(v[u]), nn, __hneg2(p)))));
    }
  }
}

// Any width, code by code.  With `low`, the rests of the products beyond fp16 go to dl, the lane's
// place among core matrices of 8 rows x 16 bytes (lo_rows bytes from one 8 tokens to the next).
template <bool FINE>
__device__ __forceinline__ void keys_by_code(const KeyLane& k, const KeyRaw& r, uint32_t tab,
                                             uint32_t dst, bool low, uint32_t dl, uint32_t lo_rows) {
  const uint32_t w = k.w, mask = (1u << w) - 1, odd = (k.src & 2u) * 8u;
  // entries of width w; no code: index 0 of the zero
  const uint32_t base = tab + (w ? kDqSingles + 2048u - (8u << w) : kDqZero);
  uint32_t x[5];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __funnelshift_r(r.x[i], r.x[i + 1], odd);
  x[4] = 0;
  const uint32_t nw[4] = {r.n.x, r.n.y, r.n.z, r.n.w};
  const uint32_t d = dst + k.col;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    // four pairs are 8 w bits: the second four start in word w / 4
    const uint32_t at = 8 * w;
    const uint32_t a0 = half == 0 ? x[0] : (at >= 64 ? x[2] : (at >= 32 ? x[1] : x[0]));
    const uint32_t a1 = half == 0 ? x[1] : (at >= 64 ? x[3] : (at >= 32 ? x[2] : x[1]));
    const uint32_t a2 = half == 0 ? x[2] : (at >= 64 ? x[4] : (at >= 32 ? x[3] : x[2]));
    uint32_t y0 = half == 0 ? a0 : __funnelshift_r(a0, a1, at & 31u);
    uint32_t y1 = half == 0 ? a1 : __funnelshift_r(a1, a2, at & 31u);
    uint32_t e0[4], e1[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      e0[u] = lds32((y0 & mask) * 4 + base);
      e1[u] = lds32(((y0 >> w) & mask) * 4 + base);
      y0 = __funnelshift_r(y0, y1, 2 * w);
      y1 >>= 2 * w;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const __half2 hi = as_h2(__byte_perm(e0[u], e1[u], 0x5410)), lo = as_h2(__byte_perm(e0[u], e1[u], 0x7632));
      const __half2 n = as_h2(nw[2 * half + (u >> 1)]);
      const __half2 nn = (u & 1) ? __high2half2(n) : __low2half2(n);
      const __half2 p = __hmul2(hi, nn);
      sts32(d + 4096 * half + 1024 * u, as_u32(p));
      // hi * n - fp16(hi * n) is exact in one fma (above the subnormals); lo * n joins it
      if (low)
        sts32(dl + (4 * half + u) * lo_rows,
              as_u32(__hfma2(lo, FINE ? __hmul2(nn, __float2half2_rn(kElement)) : nn, __hfma2(hi, nn, __hneg2(p)))));
    }
  }
}

// Value codes of a lane (portion `lane` of 16 dims) and the norms of its 16 tokens
// 16 a + 8 b + 2 c + l (rows l = 0, 1 of its c).
// Codes of more than 4 bits are fetched when they are due: holding 8 words a lane ahead
// costs every width its registers.
struct ValueRaw {
  uint32_t x[4];
  uint4 e, o;
};
__device__ __forceinline__ void load_values(ValueRaw& r, const uint8_t* tile, int kb, int vb, int step, int lane) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(tile + 1024 * kb + (step * 32 + lane) * 4 * vb);
  if (vb <= 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < vb) r.x[i] = ldg32(p + i);
  }
  const uint4* n = reinterpret_cast<const uint4*>(tile + 1024 * (kb + vb) + 32 * (lane & 3));
  r.e = ldg128(n);
  r.o = ldg128(n + 1);
}
// The norms as pairs over l, word 2 a + b; tokens from n_tok on count 0.
__device__ __forceinline__ void value_norms(const ValueRaw& r, int lane, int n_tok, uint32_t (&n)[8]) {
  const uint32_t e[4] = {r.e.x, r.e.y, r.e.z, r.e.w}, o[4] = {r.o.x, r.o.y, r.o.z, r.o.w};
#pragma unroll
  for (int u = 0; u < 8; ++u) n[u] = __byte_perm(e[u >> 1], o[u >> 1], (u & 1) ? 0x7632 : 0x5410);
  if (n_tok < 64) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int t = 8 * u + 2 * (lane & 3);
      n[u] = t >= n_tok ? 0u : (t + 1 >= n_tok ? n[u] & 0xffffu : n[u]);
    }
  }
}

// Pair I: codes 2 I, 2 I + 1 = tokens l = 0, 1 of (a, b, h) = (I / 4, I / 2 % 2, I % 2).
// All lookups of a batch come before its stores: a load may not pass a store whose address
// the compiler cannot tell apart (one by one measured a third of the rate).
template <int W, int I, int N>
__device__ __forceinline__ void value_lookups(const uint32_t* x, uint32_t tab, uint32_t lane4, uint32_t* v) {
  v[0] = code_pair_hi<W, I>(x, tab, lane4);
  if constexpr (N > 1) value_lookups<W, I + 1, N - 1>(x, tab, lane4, v + 1);
}

template <int W>
__device__ __forceinline__ void value_portion(const ValueRaw& r, const uint32_t* due,
                                              const uint32_t (&n)[8], uint32_t tab, uint32_t lane4,
                                              uint32_t dst, uint32_t g16) {
  uint32_t x[W + 1];
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = W <= 4 ? r.x[i & 3] : ldg32(due + i);
  x[W] = 0;
  uint32_t v[8];
  value_lookups<W, 0, 8>(x, tab, lane4, v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    sts32(dst + 1024 * (i & 1) + ((16u * (i >> 1)) ^ g16), as_u32(__hmul2(as_h2(v[i]), as_h2(n[i >> 1]))));
  value_lookups<W, 8, 8>(x, tab, lane4, v);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    sts32(dst + 1024 * (i & 1) + ((16u * (4 + (i >> 1))) ^ g16),
          as_u32(__hmul2(as_h2(v[i]), as_h2(n[4 + (i >> 1)]))));
}

// 16 dims (16 step .. + 15) of a tile's values into the atom at dst.
__device__ __forceinline__ void dequant_values(const uint8_t* tile, int kb, int vb, int step, int lane,
                                               const ValueRaw& r, const uint32_t (&n)[8], uint32_t tab,
                                               uint32_t dst) {
  const uint32_t lane4 = 4u * (uint32_t)lane, g = (uint32_t)lane >> 2, c = (uint32_t)lane & 3;
  const uint32_t d = dst + (uint32_t)step * 2048 + g * 128 + c * 4;  // dim 16 step + g, + 8: 1024 on
  const uint32_t* due = reinterpret_cast<const uint32_t*>(tile + 1024 * kb + (step * 32 + lane) * 4 * vb);
  switch (vb) {
    case 1: value_portion<1>(r, due, n, tab, lane4, d, g << 4); break;
    case 2: value_portion<2>(r, due, n, tab, lane4, d, g << 4); break;
    case 3: value_portion<3>(r, due, n, tab, lane4, d, g << 4); break;
    case 4: value_portion<4>(r, due, n, tab, lane4, d, g << 4); break;
    case 5: value_portion<5>(r, due, n, tab, lane4, d, g << 4); break;
    case 6: value_portion<6>(r, due, n, tab, lane4, d, g << 4); break;
    case 7: value_portion<7>(r, due, n, tab, lane4, d, g << 4); break;
    default: value_portion<8>(r, due, n, tab, lane4, d, g << 4); break;
  }
}

}  // namespace gtq
