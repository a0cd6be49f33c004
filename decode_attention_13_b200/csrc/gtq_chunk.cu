// Attention of a chunk of new tokens over the packed cache (include/gtq.h,
// gtq_chunk_attn): o = R_V^T sum_t softmax(M q . k_t / sqrt(d)) v_t, k_t and v_t
// in their rotated bases as the cache codes them.
//
// A block takes up to 256 rows of one KV head (row r = query head r % Gq of new
// token r / Gq: rows of one token share their limit) and a stretch of its tokens,
// 128 at a time.  Both products run as tcgen05.mma with fp32 accumulators in
// tensor memory; the codes are turned into fp16 operands once per block in shared
// memory and serve all its rows.
//   * warps 0-3, 4-7   softmax: thread = row (tensor-memory lane).  Scores are read
//     from tensor memory, P goes back over them as fp16 and is the A operand of the
//     second product.  The reference maximum moves only when it grew by more than
//     2^8: then the row's output in tensor memory is rescaled (by its own threads,
//     while no product on it runs).
//   * warps 8-15       tiles of codes to operands (gtq_dequant.cuh)
//   * warp 16          tensor memory, issue of all products
//   * warp 17          bulk copies of the packed tiles and the rotation images
// With 129 rows or more (NQ = 2) the two softmax groups take 128 rows each: while
// one group's products run, the other computes.  With fewer (NQ = 1) they share
// the rows and take the token blocks in turns, each with an output of its own;
// the last product joins them.
// Scores: q (hi) k (hi) over all 128 coordinates, plus q (lo) k (hi) and q (hi) k (lo) over
// the first 16, the widest codes: fp16 roundings then stay on coordinates whose part of a
// logit is small.  q is scaled by log2(e), so probabilities are powers of 2.
// The queries' rotation and the values' way back are products of the same block, with the
// rotations split into fp16 hi + lo and (for the way back) the output too.
// With few blocks' worth of rows, the tokens are split over blocks in stretches of equal
// length; each leaves a normalised output with its maximum and sum, and merge_kernel joins
// them.
#include <algorithm>

#include "gtq_dequant.cuh"
#include "gtq_internal.h"
#include "gtq_tc.cuh"

namespace gtq {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kDqWarps = 8;
constexpr int kChunkThreads = 32 * (kSoftWarps + kDqWarps + 2);
constexpr int kBlockTok = 128;     // tokens of a step
constexpr int kSplitSlots = 8;     // slots (pairs of coordinates) with a low part
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.f;    // growth of the maximum (log2) that moves the reference

// shared memory, from a 1024-byte boundary
constexpr uint32_t kQHi = 32768;                    // queries of 128 rows, fp16 (two swizzled atoms)
constexpr uint32_t kQLo = 4096;                     // their low parts, 16 coordinates
constexpr uint32_t kKBuf = 32768 + 4096;            // keys of a step, and their low parts
constexpr uint32_t kVAtom = 16384;                  // values of a packed tile
constexpr uint32_t kImage = 65536;                  // a rotation, hi and lo
template <int NQ>
struct Map {
  static constexpr uint32_t qhi = 0;
  static constexpr uint32_t qlo = qhi + NQ * kQHi;
  static constexpr uint32_t k = qlo + NQ * kQLo;
  static constexpr uint32_t v = k + 2 * kKBuf;
  static constexpr uint32_t tab = v + 3 * kVAtom;
  static constexpr uint32_t misc = tab + kDqBytes;
  // before the steps: the keys' rotation image; after them: the values' image, then the low
  // parts of the outputs (their high parts lie where the queries were) and, for NQ = 1, the
  // second group's maxima and sums
  static constexpr uint32_t image = qlo;
  static constexpr uint32_t olo = image + kImage;
  static constexpr uint32_t stat = tab - 1024;
  static_assert(olo + NQ * 32768 <= (NQ == 1 ? stat : tab), "operands of the last product");
};
struct Misc {
  alignas(16) HeadMeta m;
  alignas(16) float qscale[kD];
  uint64_t bar[34];
  uint32_t tmem;
};

// barriers
constexpr int kRing = 4;            // stages of codes at most
constexpr int kKsFull = 0;          // [kRing] key codes of a tile landed
constexpr int kKsEmpty = 4;         // [kRing] read
constexpr int kVsFull = 8;          // [kRing] value codes
constexpr int kVsEmpty = 12;
constexpr int kKFull = 16;          // [2] keys of a step written
constexpr int kKEmpty = 18;         // [2] their products done
constexpr int kVFull = 20;          // values of a step written
constexpr int kPvDone = 21;         // the step's second products done
constexpr int kSFull = 22;          // [2] scores written
constexpr int kPFull = 24;          // [2] probabilities written
constexpr int kImg = 26;            // rotation image landed
constexpr int kQRaw = 27;           // raw queries written
constexpr int kQRot = 28;           // products of a rotation done
constexpr int kQFull = 29;          // rotated queries written
constexpr int kOFull = 30;          // all steps' products done
constexpr int kOReady = 31;         // outputs written as operands
constexpr int kDrain = 32;
constexpr int kNumBars = 33;

struct ChunkArgs {
  const uint8_t* packed;
  SeqMap sm;
  int64_t T;
  const __half* q;
  int64_t qs[3];
  __half* out;
  int64_t os[3];
  int64_t n;
  const int32_t* chunk_lens;
  int causal, gq, hkv, kb, vb;
  const HeadMeta* meta;
  const uint8_t* bimg_k;   // per head
  const uint8_t* img_vt;   // R_V^T
  const uint4* dec_image;
  int row_tiles, splits;
  int64_t span;            // tokens of a split, a multiple of kBlockTok
  int ks, vs;              // stages of the rings
  float* part_o;           // [heads][splits][rows padded][128]
  float2* part_ml;         // [heads][splits][rows padded]
  int64_t rows_pad;
  int* status;
};

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

// Probabilities of one row's 128 scores at tensor-memory column `s`, written back as fp16;
// cnt of them count.  Returns their sum; `mx` (-inf if none counts) has been found before.
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t s, int cnt) {
  float mx = -INFINITY;
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tc_ld32(s + 32 * c, r);
    tc_wait_ld();
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float a = __uint_as_float(r[e]), b = __uint_as_float(r[e + 1]);
      m0 = fmaxf(m0, !MASK || 32 * c + e < cnt ? a : -INFINITY);
      m1 = fmaxf(m1, !MASK || 32 * c + e + 1 < cnt ? b : -INFINITY);
    }
    mx = fmaxf(mx, fmaxf(m0, m1));
  }
  return mx;
}
template <bool MASK>
__device__ __forceinline__ float row_exp(uint32_t s, int cnt, float ref) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 2
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32], p[16];
    tc_ld32(s + 32 * c, r);
    tc_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float a = ex2(__uint_as_float(r[e]) - ref), b = ex2(__uint_as_float(r[e + 1]) - ref);
      if (MASK) {
        a = 32 * c + e < cnt ? a : 0.f;
        b = 32 * c + e + 1 < cnt ? b : 0.f;
      }
      s0 += a;
      s1 += b;
      p[e / 2] = pack_h2(a, b);
    }
    tc_st16(s + 16 * c, p);
  }
  tc_wait_st();
  return s0 + s1;
}

template <int NQ>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  using M = Map<NQ>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = su32(sm);
  if (sb & 1023u) {  // the swizzled operands need it; there is no room to spare for a shift
    if (threadIdx.x == 0) atomicOr(a.status, kStatusLayout);
    return;
  }
  Misc& ms = *reinterpret_cast<Misc*>(sm + M::misc);
  const uint32_t ring = sb + M::misc + ((sizeof(Misc) + 127) & ~127u);
  const uint32_t ks_bytes = 1024u * a.kb + 1024u, vs_bytes = 1024u * a.vb + 128u;
  const uint32_t vring = ring + a.ks * ks_bytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv;
  const int rt = blockIdx.x % a.row_tiles, sp = blockIdx.x / a.row_tiles;
  const int64_t len = a.sm.len(b, a.T), cl = chunk_len(a.chunk_lens, a.n, b), n_rows = cl * a.gq;
  const int64_t r0 = (int64_t)rt * (128 * NQ);
  if (r0 >= n_rows) return;
  // tokens [s0, s1) of this block: its stretch, as far as its last row sees
  const int64_t last_row = (r0 + 128 * NQ < n_rows ? r0 + 128 * NQ : n_rows) - 1;
  int64_t seen = a.causal ? len - cl + last_row / a.gq + 1 : len;
  if (seen < 0) seen = 0;
  const int64_t s0 = sp * a.span;
  const int64_t s1 = seen < s0 + a.span ? seen : s0 + a.span;
  const int64_t slot0 = ((int64_t)head * a.splits + sp) * a.rows_pad + r0;  // of the partials
  if (s0 >= s1) {  // nothing to see here
    if (a.splits > 1) {
      for (int r = tid; r < 128 * NQ; r += kChunkThreads) a.part_ml[slot0 + r] = make_float2(-INFINITY, 0.f);
    } else {
      for (int i = tid; i < 128 * NQ * 16; i += kChunkThreads) {
        const int64_t row = r0 + (i >> 4);
        if (row < n_rows)
          *reinterpret_cast<uint4*>(a.out + b * a.os[0] + (h * a.gq + row % a.gq) * a.os[1] +
                                    row / a.gq * a.os[2] + 8 * (i & 15)) = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const int nb = (int)((s1 - s0 + kBlockTok - 1) / kBlockTok);  // steps
  const int nt = (int)((s1 - s0 + kTile - 1) / kTile);          // packed tiles
  const uint32_t bar0 = su32(ms.bar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };

  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(kKsFull + i), 1);
      mbar_init(bar(kKsEmpty + i), kDqWarps);
      mbar_init(bar(kVsFull + i), 1);
      mbar_init(bar(kVsEmpty + i), kDqWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKFull + i), kDqWarps);
      mbar_init(bar(kKEmpty + i), 1);
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kPFull + i), 4);
    }
    mbar_init(bar(kVFull), kDqWarps);
    mbar_init(bar(kPvDone), 1);
    mbar_init(bar(kImg), 1);
    mbar_init(bar(kQRaw), 4 * NQ);
    mbar_init(bar(kQRot), 1);
    mbar_init(bar(kQFull), 4 * NQ);
    mbar_init(bar(kOFull), 1);
    mbar_init(bar(kOReady), 4 * NQ);
    mbar_init(bar(kDrain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < (int)(sizeof(HeadMeta) / 4); i += kChunkThreads)
    reinterpret_cast<uint32_t*>(&ms.m)[i] = reinterpret_cast<const uint32_t*>(a.meta + head)[i];
  load_dequant_tables(sm + M::tab, a.dec_image, tid, kChunkThreads);
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&ms.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  // log2(e) / (sqrt(d) sqrt(m)) and the keys' factor 1 / 8 undone
  if (tid < kD)
    ms.qscale[tid] = (tid >> 1) < ms.m.n_slots
                         ? 8.f * kLog2e * 0.08838834764831845f * ms.m.inv_sqrt_m[ms.m.slot_group[tid >> 1]]
                         : 0.f;
  __syncthreads();
  int failed = 0;

  if (warp < kSoftWarps) {
    // -------------------------------------------------------------- softmax
    const int grp = warp >> 2, lrow = (warp & 3) * 32 + lane;  // row within its 128
    const int tile = NQ == 2 ? grp : 0;
    const int64_t row = r0 + 128 * tile + lrow;
    const bool mine = row < n_rows;
    const int64_t tok = mine ? row / a.gq : 0;
    const int hq = h * a.gq + (mine ? (int)(row % a.gq) : 0);
    const bool warp_on = __any_sync(0xffffffffu, mine);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + 128u * grp, t_o = tmem + lane_off + 256u + 128u * grp;
    uint8_t* qhi = sm + M::qhi + tile * kQHi + lrow * 128;
    const uint32_t sw = (uint32_t)(lrow & 7);
    // raw queries -> operand, rotated by the tensor cores, back as scaled hi + lo
    if (NQ == 2 || grp == 0) {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + b * a.qs[0] + hq * a.qs[1] + tok * a.qs[2]);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const uint4 v = mine ? src[c] : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(qhi + (c >> 3) * 16384 + (((c & 7) ^ sw) << 4)) = v;
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQRaw));
      if (!mbar_wait(bar(kQRot), 0)) failed = 1;
      __syncwarp();
      tc_fence_after();
      uint8_t* qlo = sm + M::qlo + tile * kQLo + (lrow >> 3) * 256 + (lrow & 7) * 16;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tc_ld32(t_s + 32 * c, r);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 8 coordinates each
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int p = 32 * c + 8 * k + 2 * e;
            float x = __uint_as_float(r[8 * k + 2 * e]) * ms.qscale[p];
            float y = __uint_as_float(r[8 * k + 2 * e + 1]) * ms.qscale[p + 1];
            x = fminf(fmaxf(x, -65504.f), 65504.f);
            y = fminf(fmaxf(y, -65504.f), 65504.f);
            hi[e] = pack_h2(x, y);
            const __half2 hh = *reinterpret_cast<__half2*>(&hi[e]);
            lo[e] = pack_h2(x - __low2float(hh), y - __high2float(hh));
          }
          const int ch = 4 * c + k;
          *reinterpret_cast<uint4*>(qhi + (ch >> 3) * 16384 + (((ch & 7) ^ sw) << 4)) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          if (ch < 2) *reinterpret_cast<uint4*>(qlo + ch * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      tc_fence_before();
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));
    }
    // steps
    int64_t end = !mine ? 0 : (a.causal ? len - cl + tok + 1 : len);  // tokens this row sees
    if (end > s1) end = s1;
    float ref = -INFINITY, sum = 0.f;
    int it = 0;
    for (int j = NQ == 2 ? 0 : grp; j < nb && !failed; j += NQ == 2 ? 1 : 2, ++it) {
      if (!mbar_wait(bar(kSFull + grp), it & 1)) { failed = 1; break; }
      __syncwarp();
      tc_fence_after();
      if (warp_on) {
        const int64_t left = end - (s0 + (int64_t)j * kBlockTok);
        const int cnt = left < 0 ? 0 : (left < kBlockTok ? (int)left : kBlockTok);
        const bool whole = __all_sync(0xffffffffu, cnt == kBlockTok);
        const float mx = whole ? row_max<false>(t_s, cnt) : row_max<true>(t_s, cnt);
        const bool grow = mx > ref + kRescale;  // also out of -inf
        if (__any_sync(0xffffffffu, grow)) {
          const float now = grow ? mx : ref;
          const float f = grow ? ex2(ref - now) : 1.f;
          sum *= f;
          ref = now;
          if (it) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t r[16];
              tc_ld16(t_o + 16 * c, r);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tc_st16(t_o + 16 * c, r);
            }
            tc_wait_st();
          }
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        sum += whole ? row_exp<false>(t_s, cnt, base) : row_exp<true>(t_s, cnt, base);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kPFull + grp));
    }
    // outputs: normalised, split into hi + lo operands of the last product
    if (!mbar_wait(bar(kOFull), 0)) failed = 1;
    __syncwarp();
    tc_fence_after();
    float total = sum, top = ref, other = 0.f;
    float own = 1.f;
    float2* stat = reinterpret_cast<float2*>(sm + M::stat);
    if (NQ == 1) {  // the first group joins the second one's part of its rows (same lanes)
      if (grp == 1) stat[lrow] = make_float2(ref, sum);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (grp == 0) {
        const float2 o = stat[lrow];
        top = fmaxf(ref, o.x);
        const float t = top == -INFINITY ? 0.f : top;
        own = ex2(ref - t);
        other = ex2(o.x - t);
        total = sum * own + o.y * other;
      }
    }
    if (NQ == 2 || grp == 0) {
      // 16 / sqrt(128): the values' factor
      const float inv = total > 0.f ? 1.4142135623730951f / total : 0.f;
      const float f0 = inv * own, f1 = inv * other;
      const bool two = NQ == 1 && nb > 1;
      uint8_t* ohi = sm + M::qhi + tile * kQHi + lrow * 128;
      uint8_t* olo = sm + M::olo + tile * 32768 + lrow * 128;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t r[16], u[16];
        if (warp_on) {
          tc_ld16(t_o + 16 * c, r);
          if (two) tc_ld16(t_o + 128 + 16 * c, u);
          tc_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int at = 8 * k + 2 * e + i;
              // a part that saw nothing may hold anything
              float v = warp_on && f0 > 0.f ? __uint_as_float(r[at]) * f0 : 0.f;
              if (two && warp_on && f1 > 0.f) v = fmaf(__uint_as_float(u[at]), f1, v);
              x[i] = v;
            }
            hi[e] = pack_h2(x[0], x[1]);
            const __half2 hh = *reinterpret_cast<__half2*>(&hi[e]);
            lo[e] = pack_h2(x[0] - __low2float(hh), x[1] - __high2float(hh));
          }
          const int ch = 2 * c + k;
          const uint32_t off = (ch >> 3) * 16384 + (((ch & 7) ^ sw) << 4);
          *reinterpret_cast<uint4*>(ohi + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(olo + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      tc_fence_before();
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOReady));
      if (!mbar_wait(bar(kQRot), 1)) failed = 1;
      __syncwarp();
      tc_fence_after();
      if (warp_on && !__any_sync(0xffffffffu, failed)) {
        const bool split = a.splits > 1;
        __half* out = a.out + b * a.os[0] + hq * a.os[1] + tok * a.os[2];
        float* po = a.part_o + (slot0 + 128 * tile + lrow) * kD;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tc_ld32(t_s + 32 * c, r);
          tc_wait_ld();
          if (!mine) {
          } else if (split) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<uint4*>(po)[8 * c + k] =
                  make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_h2(__uint_as_float(r[8 * k + 2 * e]), __uint_as_float(r[8 * k + 2 * e + 1]));
              reinterpret_cast<uint4*>(out)[4 * c + k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
        if (split && mine) a.part_ml[slot0 + 128 * tile + lrow] = make_float2(top, total);
      }
    }
  } else if (warp < kSoftWarps + kDqWarps) {
    // ------------------------------------------------------ codes to operands
    const int dw = warp - kSoftWarps;
    const uint32_t tab = sb + M::tab;
    const HeadMeta& m = ms.m;
    // the keys' buffers lie under the rotation image
    if (!mbar_wait(bar(kQRot), 0)) failed = 1;
    auto keys = [&](int j) {  // keys of step j
      if (j >= 2 && !mbar_wait(bar(kKEmpty + (j & 1)), ((j >> 1) & 1) ^ 1)) return false;
      const uint32_t dst = sb + M::k + (j & 1) * kKBuf;
      for (int half = 0; half < 2; ++half) {
        const int t = 2 * j + half;
        if (t >= nt) break;  // rows behind the last tile: whatever they hold, their scores do not count
        const int st = t % a.ks;
        if (!mbar_wait(bar(kKsFull + st), (t / a.ks) & 1)) return false;
        const uint32_t src = ring + st * ks_bytes;
        // the quads with low parts cost more: they go round the warps
        for (int k = 0; k < 2; ++k)
          dequant_keys(m, ((dw + t) & 7) + 8 * k, lane, src, src + 1024u * a.kb, tab, dst + half * 8192, 16384,
                       kSplitSlots, dst + 32768 + half * 2048, 256);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kKsEmpty + st));
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull + (j & 1)));
      return true;
    };
    auto values = [&](int j) {
      for (int half = 0; half < 2; ++half) {
        const int t = 2 * j + half;
        // three atoms: the second of a step is the one that the step before began with
        if (half == 1 && j >= 1 && !mbar_wait(bar(kPvDone), (j - 1) & 1)) return false;
        const uint32_t dst = sb + M::v + (t % 3) * kVAtom;
        if (t < nt) {
          const int st = t % a.vs;
          if (!mbar_wait(bar(kVsFull + st), (t / a.vs) & 1)) return false;
          const uint32_t src = vring + st * vs_bytes;
          const int64_t left = s1 - (s0 + (int64_t)t * kTile);
          uint32_t n[8];
          value_norms(src + 1024u * a.vb, lane, left < kTile ? (int)left : kTile, n);
          dequant_values(a.vb, dw, lane, src, n, tab, dst);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kVsEmpty + st));
        } else {  // no tile: zeros, since the probabilities' zeros must not meet a NaN
          for (int i = lane; i < 128; i += 32)
            *reinterpret_cast<uint4*>(sm + M::v + (t % 3) * kVAtom + dw * 2048 + 16 * i) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kVFull));
      return true;
    };
    if (!failed && !keys(0)) failed = 1;
    for (int j = 0; j < nb && !failed; ++j) {
      if (j + 1 < nb && !keys(j + 1)) { failed = 1; break; }
      if (!values(j)) { failed = 1; break; }
    }
  } else if (warp == 16) {
    // ------------------------------------------------------------- products
    if (lane == 0) {
      const uint32_t idc = idesc_f16(128);
      auto rotate = [&](uint32_t d, uint32_t x, uint32_t img, bool more, bool with_lo) {
        // d (+)= x . (hi + lo)^T of the image; with_lo: the low part of the image too
#pragma unroll
        for (int part = 0; part < 2; ++part)
          if (part == 0 || with_lo)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t o = (ks >> 2) * 16384 + (ks & 3) * 32;
              tc_mma(d, smem_desc(x + o), smem_desc(img + part * 32768 + o), idc, more || (part | ks) != 0);
            }
      };
      auto scores = [&](int x, int j) {
        const uint32_t qt = NQ == 2 ? x : 0;
        const uint32_t q = sb + M::qhi + qt * kQHi, k = sb + M::k + (j & 1) * kKBuf, d = tmem + 128u * x;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t o = (ks >> 2) * 16384 + (ks & 3) * 32;
          tc_mma(d, smem_desc(q + o), smem_desc(k + o), idc, ks != 0);
        }
        tc_mma(d, smem_desc_plain(sb + M::qlo + qt * kQLo, 128, 256), smem_desc(k), idc, 1);
        tc_mma(d, smem_desc(q), smem_desc_plain(k + 32768, 128, 256), idc, 1);
        tc_commit(bar(kSFull + x));
      };
      auto outputs = [&](int x, int j, bool more) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t v = sb + M::v + ((2 * j + half) % 3) * kVAtom;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma_ta(tmem + 256u + 128u * x, tmem + 128u * x + 32u * half + 8u * ks, smem_desc(v + 32 * ks), idc,
                      more || (half | ks) != 0);
        }
      };
      auto waits = [&](int i, uint32_t par) {
        if (!failed && !mbar_wait(bar(i), par)) failed = 1;
        return !failed;
      };
      waits(kImg, 0);
      if (waits(kQRaw, 0)) {
        tc_fence_after();
        for (int x = 0; x < NQ; ++x) rotate(tmem + 128u * x, sb + M::qhi + x * kQHi, sb + M::image, false, true);
        tc_commit(bar(kQRot));
      }
      waits(kQFull, 0);
      // first scores
      for (int x = 0; x < 2 && !failed; ++x) {
        const int j = NQ == 2 ? 0 : x;
        if (j >= nb || !waits(kKFull + (j & 1), 0)) break;
        tc_fence_after();
        scores(x, j);
        if (NQ == 1 || x == 1) tc_commit(bar(kKEmpty + (j & 1)));
      }
      for (int j = 0; j < nb && !failed; ++j) {
        for (int y = 0; y < NQ; ++y) {
          const int x = NQ == 2 ? y : j & 1;           // group
          const int it = NQ == 2 ? j : j >> 1;         // its step
          const int nj = NQ == 2 ? j + 1 : j + 2;      // its next
          if (!waits(kPFull + x, it & 1) || !waits(kVFull, j & 1)) break;
          tc_fence_after();
          outputs(x, j, it > 0);
          if (y == NQ - 1) tc_commit(bar(kPvDone));
          if (nj < nb) {
            if (!waits(kKFull + (nj & 1), (nj >> 1) & 1)) break;
            tc_fence_after();
            scores(x, nj);
            if (y == NQ - 1) tc_commit(bar(kKEmpty + (nj & 1)));
          }
        }
      }
      tc_commit(bar(kOFull));
      if (waits(kImg, 1) && waits(kOReady, 0)) {
        tc_fence_after();
        const uint32_t img = sb + M::image;
        for (int x = 0; x < NQ; ++x) {
          rotate(tmem + 128u * x, sb + M::qhi + x * kQHi, img, false, true);
          rotate(tmem + 128u * x, sb + M::olo + x * 32768, img, true, false);
        }
        tc_commit(bar(kQRot));
      }
    }
  } else {
    // ------------------------------------------------------------ bulk copies
    if (lane == 0) {
      mbar_expect_tx(bar(kImg), kImage);
      bulk_load(sb + M::image, a.bimg_k + (size_t)head * kImage, kImage, bar(kImg));
      const uint32_t norm_bytes = 128u * ms.m.n_groups;
      const int64_t t0 = s0 / kTile;
      int kt = 0, vt = 0;  // next tile of each ring
      while ((kt < nt || vt < nt) && !failed) {
        // keys run a step (and the next step's two tiles) ahead of the values, as they are used: a
        // ring of one stage still never waits for a tile that is behind it
        const bool key = kt < nt && (kt < vt + 4 || vt >= nt);
        const int t = key ? kt : vt, n = key ? a.ks : a.vs, st = t % n;
        if (t >= n && !mbar_wait(bar((key ? kKsEmpty : kVsEmpty) + st), ((t / n) & 1) ^ 1)) { failed = 1; break; }
        const uint8_t* src = a.sm.tile(const_cast<uint8_t*>(a.packed), head, t0 + t);
        if (key) {
          const uint32_t dst = ring + st * ks_bytes;
          mbar_expect_tx(bar(kKsFull + st), 1024u * a.kb + norm_bytes);
          bulk_load(dst, src, 1024u * a.kb, bar(kKsFull + st));
          if (norm_bytes)
            bulk_load(dst + 1024u * a.kb, src + key_norm_offset(a.kb, a.vb), norm_bytes, bar(kKsFull + st));
          ++kt;
        } else {
          mbar_expect_tx(bar(kVsFull + st), vs_bytes);
          bulk_load(vring + st * vs_bytes, src + 1024u * a.kb, vs_bytes, bar(kVsFull + st));
          ++vt;
        }
      }
      if (!mbar_wait(bar(kOFull), 0)) failed = 1;
      if (!failed) {
        mbar_expect_tx(bar(kImg), kImage);
        bulk_load(sb + M::image, a.img_vt, kImage, bar(kImg));
        if (!mbar_wait(bar(kImg), 1)) failed = 1;
      } else {  // copies in flight: the image, and the last of every stage
        mbar_wait(bar(kImg), 0);
        for (int i = 0; i < a.ks && i < kt; ++i) mbar_wait(bar(kKsFull + i), ((kt - 1 - i) / a.ks) & 1);
        for (int i = 0; i < a.vs && i < vt; ++i) mbar_wait(bar(kVsFull + i), ((vt - 1 - i) / a.vs) & 1);
      }
    }
  }
  if (failed) atomicOr(a.status, kStatusTimeout);
  if (__syncthreads_or(failed)) {
    if (warp == 16 && lane == 0) {
      tc_commit(bar(kDrain));
      mbar_wait(bar(kDrain), 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// One warp per row: the splits' outputs, weighted by what their maxima and sums say.
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ ChunkArgs a) {
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t cl = chunk_len(a.chunk_lens, a.n, b);
  if (row >= cl * a.gq) return;
  const int64_t base = (int64_t)head * a.splits * a.rows_pad + row;
  float top = -INFINITY;
  for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_ml[base + s * a.rows_pad].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  if (top != -INFINITY)
    for (int s = 0; s < a.splits; ++s) {
      const float2 ml = a.part_ml[base + s * a.rows_pad];
      const float w = ml.y * ex2(ml.x - top);
      if (!(w > 0.f)) continue;
      const float4 o = reinterpret_cast<const float4*>(a.part_o + (base + s * a.rows_pad) * kD)[lane];
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
      total += w;
    }
  const float inv = total > 0.f ? 1.f / total : 0.f;
  __half* out = a.out + b * a.os[0] + (h * a.gq + row % a.gq) * a.os[1] + row / a.gq * a.os[2];
  *reinterpret_cast<uint2*>(out + 4 * lane) =
      make_uint2(pack_h2(acc.x * inv, acc.y * inv), pack_h2(acc.z * inv, acc.w * inv));
}

// How a call is cut: rows per block, splits of the tokens, stages.
struct Cut {
  int nq, row_tiles, splits, ks, vs;
  int64_t span, rows_pad;
  uint32_t smem;
};

constexpr uint32_t kSmemMost = 232448;
constexpr uint32_t kMiscBytes = (uint32_t)((sizeof(Misc) + 127) & ~127u);
static_assert(Map<1>::misc + kMiscBytes + (1024 * 8 + 1024) + (1024 * 8 + 128) <= kSmemMost, "widest codes");

Cut cut_of(const gtq_plan* p, int64_t T, int64_t n) {
  Cut c;
  const int64_t rows = n * p->g_q;
  const uint32_t kbytes = 1024u * p->cfg.k_bits + 1024u, vbytes = 1024u * p->cfg.v_bits + 128u;
  auto room = [&](int nq) {
    return (int)kSmemMost - (int)((nq == 2 ? Map<2>::misc : Map<1>::misc) + kMiscBytes);
  };
  // 256 rows a block where there are that many and two tiles of keys and one of values fit beside
  // them (up to 8 bits a dim for both together); then as many tiles in flight as fit
  c.nq = rows > 128 && room(2) >= (int)(2 * kbytes + vbytes) ? 2 : 1;
  c.ks = c.vs = 1;
  for (bool more = true; more;) {
    more = false;
    if (c.ks < kRing && c.ks <= c.vs && room(c.nq) >= (int)((c.ks + 1) * kbytes + c.vs * vbytes)) {
      ++c.ks;
      more = true;
    }
    if (c.vs < kRing && room(c.nq) >= (int)(c.ks * kbytes + (c.vs + 1) * vbytes)) {
      ++c.vs;
      more = true;
    }
  }
  c.smem = (c.nq == 2 ? Map<2>::misc : Map<1>::misc) + kMiscBytes + c.ks * kbytes + c.vs * vbytes;
  c.row_tiles = (int)((rows + 128 * c.nq - 1) / (128 * c.nq));
  c.rows_pad = (int64_t)c.row_tiles * 128 * c.nq;
  // Splits: enough blocks to fill the SMs, and evenly; a block's set-up and end cost about as
  // much as 8 steps, a merge more the more parts there are.
  const int64_t units = (int64_t)p->n_heads * c.row_tiles, steps = (T + kBlockTok - 1) / kBlockTok;
  double best = 1e300;
  int64_t best_steps = steps;
  for (int64_t s = 1; s <= 256 && s <= steps; ++s) {
    const int64_t per = (steps + s - 1) / s, parts = (steps + per - 1) / per;
    const int64_t waves = (units * parts + p->n_sms - 1) / p->n_sms;
    const double cost = (double)waves * (per + 8.0) + (parts > 1 ? 4.0 + 0.02 * parts * units / p->n_sms : 0.0);
    if (cost < best * 0.999) {
      best = cost;
      best_steps = per;
    }
    if (units * s > 64 * (int64_t)p->n_sms) break;
  }
  c.span = best_steps * kBlockTok;
  c.splits = (int)((steps + best_steps - 1) / best_steps);
  return c;
}

}  // namespace

size_t chunk_workspace(const gtq_plan* p, int64_t T, int64_t n) {
  const Cut c = cut_of(p, T, n);
  if (c.splits <= 1) return 256;
  const size_t slots = (size_t)p->n_heads * c.splits * c.rows_pad;
  return slots * (kD * sizeof(float) + sizeof(float2));
}

cudaError_t launch_chunk(const gtq_plan* p, const uint8_t* packed, int64_t T, const SeqMap& sm,
                         const gtq_chunk& ch, const __half* q, __half* out, uint8_t* workspace,
                         cudaStream_t s) {
  const Cut c = cut_of(p, T, ch.n_tokens);
  ChunkArgs a = {};
  a.packed = packed;
  a.sm = sm;
  a.T = T;
  a.q = q;
  a.out = out;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = ch.q_strides[i];
    a.os[i] = ch.out_strides[i];
  }
  a.n = ch.n_tokens;
  a.chunk_lens = ch.chunk_lens_dev;
  a.causal = ch.causal;
  a.gq = p->g_q;
  a.hkv = p->cfg.n_kv_heads;
  a.kb = p->cfg.k_bits;
  a.vb = p->cfg.v_bits;
  a.meta = p->d_meta;
  a.bimg_k = p->d_bimg;
  a.img_vt = p->tab.rvt_image;
  a.dec_image = p->tab.dec_image;
  a.row_tiles = c.row_tiles;
  a.splits = c.splits;
  a.span = c.span;
  a.ks = c.ks;
  a.vs = c.vs;
  a.rows_pad = c.rows_pad;
  a.status = p->d_status;
  const size_t slots = (size_t)p->n_heads * c.splits * c.rows_pad;
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(workspace + slots * kD * sizeof(float));
  auto kernel = c.nq == 2 ? chunk_kernel<2> : chunk_kernel<1>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.smem);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)(c.row_tiles * c.splits), (unsigned)p->n_heads), kChunkThreads, c.smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || c.splits == 1) return e;
  merge_kernel<<<dim3((unsigned)((ch.n_tokens * p->g_q + 7) / 8), (unsigned)p->n_heads), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace gtq
