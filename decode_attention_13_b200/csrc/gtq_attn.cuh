// What the kernels over several new tokens of a sequence share.
#pragma once

#include "gtq_dequant.cuh"
#include "gtq_internal.h"
#include "gtq_tc.cuh"

namespace gtq {

constexpr float kLog2e = 1.4426950408889634f;

// Rows that sequence b brings.
__device__ __forceinline__ int64_t chunk_len(const int32_t* lens, int64_t n, int b) {
  if (!lens) return n;
  const int64_t c = lens[b];
  return c < 0 ? 0 : (c < n ? c : n);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// two fp32 additions in one instruction
__device__ __forceinline__ uint64_t pack_f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Maximum of one row's first cnt of 128 scores at tensor-memory column `s`.
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t s, int cnt) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tc_ld32(s + 32 * c, r);
    tc_wait_ld();
    const int left = cnt - 32 * c;
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = !MASK || e + i < left ? __uint_as_float(r[e + i]) : -INFINITY;
      m0 = max3(m0, x[0], x[1]);
      m1 = max3(m1, x[2], x[3]);
    }
  }
  return fmaxf(m0, m1);
}

// Raw queries of one row (16 chunks of 8 fp16, or zeros) into a swizzled operand of 128 rows.
__device__ __forceinline__ void put_query_row(uint8_t* operand, int row, const uint4* src, bool mine) {
  uint8_t* o = operand + row * 128;
  const uint32_t sw = (uint32_t)(row & 7);
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const uint4 v = mine ? src[c] : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(o + (c >> 3) * 16384 + (((c & 7) ^ sw) << 4)) = v;
  }
}
// 8 values, scaled, as fp16 hi and the rest.  An infinity becomes a NaN, as it would in a softmax.
__device__ __forceinline__ void split8(const uint32_t* r, const float* scale, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x = __uint_as_float(r[2 * e]) * scale[2 * e], y = __uint_as_float(r[2 * e + 1]) * scale[2 * e + 1];
    x += x - x;
    y += y - y;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h[e]) : "f"(y), "f"(x));
    const __half2 hh = *reinterpret_cast<__half2*>(&h[e]);
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(l[e]) : "f"(y - __high2float(hh)), "f"(x - __low2float(hh)));
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// Factor of a rotated query coordinate: log2(e) / (sqrt(d) sqrt(m)), and the keys' kElement undone:
// 1.02 / sqrt(m).  A coordinate is at most sqrt(m) times the group's root mean square, so hi stays
// in the fp16 range (split8 would clip it) up to a root mean square of .98 of fp16's largest number.
__device__ __forceinline__ float query_scale(const HeadMeta& m, int pos) {
  return (pos >> 1) < m.n_slots ? kLog2e * 0.08838834764831845f / kElement * m.inv_sqrt_m[m.slot_group[pos >> 1]] : 0.f;
}
// k-step ks (16 columns) of a swizzled operand of 128 rows: what its descriptor moves by
__device__ __forceinline__ uint64_t kstep(uint32_t ks) {
  return (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
}

}  // namespace gtq
