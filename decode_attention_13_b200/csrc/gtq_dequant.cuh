// Packed tiles to fp16 matrix operands in shared memory, for the tcgen05
// kernels that attend over the packed cache.
//
// Keys, one tile of 64 tokens: rows = tokens, columns = packed coordinates
// (slot s: columns 2s, 2s + 1), value cb[code] * norm / 8, K-major with the
// 128-byte swizzle in two atoms of 64 columns.  A lane takes the portion of one
// slot for tokens g, g + 8, ..., g + 56 (g = lane % 8), a warp four neighbouring
// slots: with the swizzle its 4-byte stores fall into 32 different banks.
// Values: rows = rotated dims, columns = the tile's 64 tokens, cb[code] * norm /
// 16, one swizzled atom; a lane takes a portion (two dims, 16 tokens).
// Powers of two keep the largest norm (65504) times the largest centroid in the
// fp16 range; both are undone in the queries and at the end.
//
// A pair of codes is looked up at once where the pair table is small (widths 1
// to 3: one 32-bit copy per lane, no bank conflicts), code by code above.
#pragma once

#include "gtq_internal.h"
#include "gtq_tc.cuh"

namespace gtq {

// Lookup tables in shared memory: pair tables of widths 3, 2, 1 and the single
// codes of width 5 as they lie in the decode image (kTabP32W3 .. kTabS32W6),
// single codes of width 4 (one copy per lane), single codes of all widths.
constexpr uint32_t kDqPairs = 0;
constexpr uint32_t kDqPairBytes = kTabS32W6 - kTabP32W3;
constexpr uint32_t kDqW4 = kDqPairs + kDqPairBytes;
constexpr uint32_t kDqSingles = kDqW4 + (16u << 7);
constexpr uint32_t kDqBytes = kDqSingles + 2048u;
static_assert(kDqBytes % 16 == 0, "dequantisation tables");

// Copies the tables from the decode image (all threads of the block).
__device__ __forceinline__ void load_dequant_tables(uint8_t* tab, const uint4* image, int tid,
                                                    int n_threads) {
  const uint8_t* img = reinterpret_cast<const uint8_t*>(image);
  for (int i = tid; i < (int)(kDqPairBytes / 16); i += n_threads)
    reinterpret_cast<uint4*>(tab + kDqPairs)[i] = reinterpret_cast<const uint4*>(img + kTabP32W3)[i];
  for (int i = tid; i < 512; i += n_threads) {
    const uint32_t* ss = reinterpret_cast<const uint32_t*>(img + kTabSS);
    reinterpret_cast<uint32_t*>(tab + kDqSingles)[i] = ss[i];
    reinterpret_cast<uint32_t*>(tab + kDqW4)[i] = ss[kSingleOff(4) / 4 + (i >> 5)];
  }
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
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

// 16 W bits from byte address `a` (a multiple of 2; of 4 for even W) in shared
// memory, in words.
template <int W>
__device__ __forceinline__ void load_portion(uint32_t a, uint32_t (&x)[5]) {
  if constexpr (W == 8) {
    asm("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(a));
  } else if constexpr (W == 4) {
    asm("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(a));
  } else if constexpr (W % 2 == 0) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) x[i] = lds32(a + 4 * i);
  } else {  // an odd number of halfwords that starts at either half of a word
    constexpr int n = (W + 1) / 2;
    const uint32_t base = a & ~3u, sh = (a & 2u) * 8u;
    uint32_t y[n + 1];
#pragma unroll
    for (int i = 0; i < n; ++i) y[i] = lds32(base + 4 * i);
    y[n] = 0;
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = __funnelshift_r(y[i], y[i + 1], sh);
  }
}

// Entry (fp16 hi | lo << 16) of code I of width W in the words x.
template <int W, int I, bool SHARED>
__device__ __forceinline__ uint32_t single(const uint32_t* x, uint32_t tab, uint32_t lane4) {
  if constexpr (!SHARED && W == 4)
    return lds32(tab + kDqW4 + (field<I * 4, 4, 7>(x) | lane4));
  else if constexpr (!SHARED && W == 5) {
    // the place that a field of 5 bits moves to must not lie above where it starts
    // in a crossing word: 7 only below bit 28, which always holds for a crossing
    return lds32(tab + kDqPairs + (kTabS32W5 - kTabP32W3) + (field<I * 5, 5, 7>(x) | lane4));
  } else
    return lds32(tab + kDqSingles + kSingleOff(W) + field<I * W, W, 2>(x));
}

// fp16 pair (codes 2 U, 2 U + 1 of width W), hi parts.
template <int W, int U>
__device__ __forceinline__ uint32_t code_pair_hi(const uint32_t* x, uint32_t tab, uint32_t lane4) {
  if constexpr (W <= 3) {
    return lds32(tab + kDqPairs + (kTabP32(W) - kTabP32W3) + (field<2 * U * W, 2 * W, 7>(x) | lane4));
  } else {
    const uint32_t e0 = single<W, 2 * U, (W > 5)>(x, tab, lane4);
    const uint32_t e1 = single<W, 2 * U + 1, (W > 5)>(x, tab, lane4);
    return __byte_perm(e0, e1, 0x5410);
  }
}

// norm u (0..7) of four words of fp16 pairs, in both halves
template <int U>
__device__ __forceinline__ uint32_t norm_both(const uint32_t* n) {
  return __byte_perm(n[U >> 1], 0, (U & 1) ? 0x3232 : 0x1010);
}

// One slot's portion: 8 tokens (rows g + 8 u of `dst`, 128 bytes a row, 1024 a
// group of 8), the pair at byte `col` of the (already swizzled) row.
template <int W, int U>
__device__ __forceinline__ void key_pairs(const uint32_t* x, const uint32_t* n, uint32_t tab,
                                          uint32_t lane4, uint32_t dst) {
  sts32(dst + 1024 * U, h2mul(code_pair_hi<W, U>(x, tab, lane4), norm_both<U>(n)));
  if constexpr (U < 7) key_pairs<W, U + 1>(x, n, tab, lane4, dst);
}
// The same with the rest of the product beyond its fp16 value, in plain layout.
template <int W, int U>
__device__ __forceinline__ void key_pairs_split(const uint32_t* x, const uint32_t* n, uint32_t tab,
                                                uint32_t dst, uint32_t dst_lo, uint32_t lo_step) {
  const uint32_t e0 = single<W, 2 * U, true>(x, tab, 0), e1 = single<W, 2 * U + 1, true>(x, tab, 0);
  const uint32_t hi = __byte_perm(e0, e1, 0x5410), lo = __byte_perm(e0, e1, 0x7632);
  const uint32_t nn = norm_both<U>(n);
  const uint32_t p = h2mul(hi, nn);
  sts32(dst + 1024 * U, p);
  // hi * n - fp16(hi * n) is exact in one fma (above the subnormals); lo * n joins it
  sts32(dst_lo + lo_step * U, h2fma(lo, nn, h2fma(hi, nn, p ^ 0x80008000u)));
  if constexpr (U < 7) key_pairs_split<W, U + 1>(x, n, tab, dst, dst_lo, lo_step);
}

template <int W>
__device__ __forceinline__ void key_slot(uint32_t src, uint32_t src_norm, uint32_t tab,
                                         uint32_t lane4, uint32_t dst, bool split, uint32_t dst_lo,
                                         uint32_t lo_step) {
  uint32_t x[5], n[4];
  load_portion<W>(src, x);
  asm("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(n[0]), "=r"(n[1]), "=r"(n[2]), "=r"(n[3]) : "r"(src_norm));
#pragma unroll
  for (int i = 0; i < 4; ++i) n[i] = h2mul(n[i], 0x30003000u);  // 1 / 8
  if (split) key_pairs_split<W, 0>(x, n, tab, dst, dst_lo, lo_step);
  else key_pairs<W, 0>(x, n, tab, lane4, dst);
}

// Four slots (4 quad .. 4 quad + 3) of a tile: `codes` and `norms` are the
// shared addresses of the tile's key codes and key norms, `dst` the tile's first
// row in the operand's first atom (the second one `atom` bytes on).  Slots below
// n_split also leave the products' rests at dst_lo, in core matrices of 8 rows x 16
// bytes: row r, coordinate c at (r / 8) * lo_rows + (c / 8) * 128 + (r % 8) * 16 +
// (c % 8) * 2.
__device__ __forceinline__ void dequant_keys(const HeadMeta& m, int quad, int lane, uint32_t codes,
                                             uint32_t norms, uint32_t tab, uint32_t dst,
                                             uint32_t atom, int n_split, uint32_t dst_lo,
                                             uint32_t lo_rows) {
  const int g = lane & 7, s = 4 * quad + (lane >> 3);
  const uint32_t lane4 = 4u * (uint32_t)lane;
  const uint32_t col = (uint32_t)((((s >> 2) & 7) ^ g) << 4) + 4u * (uint32_t)(s & 3);
  const uint32_t d = dst + (s >> 5) * atom + 128u * (uint32_t)g + col;
  const int w = m.slot_width[s];
  const uint32_t src = codes + m.slot_koff[s] + 2u * (uint32_t)(w * g);
  const uint32_t sn = norms + 128u * m.slot_group[s] + 16u * (uint32_t)g;
  const bool split = s < n_split;
  const uint32_t dl = dst_lo + (uint32_t)(s >> 2) * 128 + 16u * (uint32_t)g + 4u * (uint32_t)(s & 3);
  switch (w) {
    case 1: key_slot<1>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 2: key_slot<2>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 3: key_slot<3>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 4: key_slot<4>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 5: key_slot<5>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 6: key_slot<6>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 7: key_slot<7>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    case 8: key_slot<8>(src, sn, tab, lane4, d, split, dl, lo_rows); break;
    default:  // no code: its query coordinate is 0, but the operand has to be finite
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        sts32(d + 1024 * u, 0);
        if (split) sts32(dl + lo_rows * u, 0);
      }
  }
}

// Norms of a lane's 16 tokens (16 a + 8 b + 2 c + l) as pairs over l, word 2 a + b,
// divided by 16; tokens from n_tok on count 0.
__device__ __forceinline__ void value_norms(uint32_t norms, int lane, int n_tok, uint32_t (&n)[8]) {
  const int c = lane & 3;
  uint32_t e[4], o[4];
  asm("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(e[0]), "=r"(e[1]), "=r"(e[2]), "=r"(e[3]) : "r"(norms + 32u * c));
  asm("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(norms + 32u * c + 16u));
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    uint32_t v = __byte_perm(e[u >> 1], o[u >> 1], (u & 1) ? 0x7632 : 0x5410);
    if (n_tok < 64) {
      const int t = 8 * u + 2 * c;
      if (t >= n_tok) v = 0;
      else if (t + 1 >= n_tok) v &= 0xffffu;
    }
    n[u] = h2mul(v, 0x2c002c00u);  // 1 / 16
  }
}

template <int W, int I>
__device__ __forceinline__ void value_pairs(const uint32_t* x, const uint32_t (&n)[8], uint32_t tab,
                                            uint32_t lane4, uint32_t dst, uint32_t g16) {
  // pair I: codes 2 I, 2 I + 1 = tokens l = 0, 1 of (a, b, h) = (I / 4, I / 2 % 2, I % 2)
  constexpr int u = I >> 1, h = I & 1;
  const uint32_t v = h2mul(code_pair_hi<W, I>(x, tab, lane4), n[u]);
  sts32(dst + 1024 * h + ((16u * u) ^ g16), v);
  if constexpr (I < 15) value_pairs<W, I + 1>(x, n, tab, lane4, dst, g16);
}

template <int W>
__device__ __forceinline__ void value_portion(uint32_t src, const uint32_t (&n)[8], uint32_t tab,
                                              uint32_t lane4, uint32_t dst, uint32_t g16) {
  uint32_t x[9];
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = lds32(src + 4 * i);
  x[W] = 0;
  value_pairs<W, 0>(x, n, tab, lane4, dst, g16);
}

// 16 dims (16 step .. + 15) of a tile's values into the atom at dst.
__device__ __forceinline__ void dequant_values(int vb, int step, int lane, uint32_t codes,
                                               const uint32_t (&n)[8], uint32_t tab, uint32_t dst) {
  const uint32_t lane4 = 4u * (uint32_t)lane, g = (uint32_t)lane >> 2, c = (uint32_t)lane & 3;
  const uint32_t src = codes + (uint32_t)(step * 32 + lane) * 4u * (uint32_t)vb;
  const uint32_t d = dst + (uint32_t)step * 2048 + g * 128 + c * 4;  // dim 16 step + g, + 8: 1024 on
  switch (vb) {
    case 1: value_portion<1>(src, n, tab, lane4, d, g << 4); break;
    case 2: value_portion<2>(src, n, tab, lane4, d, g << 4); break;
    case 3: value_portion<3>(src, n, tab, lane4, d, g << 4); break;
    case 4: value_portion<4>(src, n, tab, lane4, d, g << 4); break;
    case 5: value_portion<5>(src, n, tab, lane4, d, g << 4); break;
    case 6: value_portion<6>(src, n, tab, lane4, d, g << 4); break;
    case 7: value_portion<7>(src, n, tab, lane4, d, g << 4); break;
    default: value_portion<8>(src, n, tab, lane4, d, g << 4); break;
  }
}

}  // namespace gtq
