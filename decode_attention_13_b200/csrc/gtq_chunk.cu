// Attention of a chunk of new tokens over the packed cache (include/gtq.h,
// gtq_chunk_attn): o = R_V^T sum_t softmax(M q . k_t / sqrt(d)) v_t, k_t and v_t
// in their rotated bases as the cache codes them.
//
// A block takes up to 256 rows of one KV head (row r = query head r % Gq of new
// token r / Gq: rows of one token share their limit), or a pair of CTAs up to 512,
// and a stretch of its tokens, 128 at a time.  Both products run as tcgen05.mma with
// fp32 accumulators in tensor memory; the codes are turned into fp16 operands once per
// block in shared memory and serve all its rows.
//   * warps 0-3, 4-7   softmax: thread = row (tensor-memory lane).  Scores are read
//     from tensor memory, P goes back over them as fp16 and is the A operand of the
//     second product.  The reference maximum moves only when it grew by more than
//     2^4: then the row's output in tensor memory is rescaled (by its own threads,
//     while no product on it runs).
//     The first warp of each group of four also issues the group's products, as soon as the
//     group has written its P: one hand-off less than a warp of its own.
//   * warps 8-15       tiles of codes to operands (gtq_dequant.cuh): keys run a step ahead
//     of values, and a warp's loads of the one are in flight while it works on the other.
//     (24 warps, 16 of them here, measured 1.06 times slower over 512 rows: 80 registers a
//     thread are too few for it.)
// With 129 rows or more (NQ = 2) the two softmax groups take 128 rows each: while
// one group's products run, the other computes, and they take turns with the exponentials.
// With fewer (NQ = 1) they share the rows and take the token blocks in turns, each with an
// output of its own; the last product joins them.
// In a pair (cta_group::2) each CTA has 256 rows and turns half of every step's codes: 64 of
// its 128 tokens' keys, 64 of the 128 dims of its values.  The even CTA issues both CTAs'
// products.
// With few blocks' worth of rows, the tokens are split over blocks in stretches of equal
// length; each leaves a normalised output with its maximum and sum, and merge_kernel joins
// them.
//
// Roundings.  fp16, half a step 2^-11: the turned keys, P, the values, the result.  Scores:
// q (hi) k (hi) over all 128 coordinates, plus q (lo) k (hi) and q (hi) k (lo) over
// the first 16, the widest codes, which carry most of a logit (lo of a key is good to 2^-22 of its
// group's norm): the error that is left in a
// logit comes from coordinates whose part of it is small.  P's sum is taken before P is
// rounded.  q is scaled by log2(e), so probabilities are powers of 2.  The queries' rotation
// and the values' way back are products of the same block, with the rotations split into
// fp16 hi + lo and (for the way back) the output too.  All sums are fp32.  Rows come out
// 2.8e-4 to 4.1e-4 off attention in 64 bits (2-norm): the result's own rounding is 2e-4 of it, P's
// and the values' two (centroid, element) are 2e-4 each, independent of one another.  That holds while
// the logits' parts beyond the first 16 coordinates are of a few units.  A logit of 15 spread evenly over 128
// coordinates is off by up to 5e-3, and a row that hangs on it by half as much (2.7e-3 measured).
//
// What bounds it: up to 128 rows, turning codes (about 4000 cycles a step of 128 tokens; 40
// rows over 2 x 131072 tokens, 3 bits, 29 MB: 57 us back to back, 66 us a call on inputs that the
// L2 cache does not hold).  With pairs, the chain from a step's scores over the softmax and P to its
// products, about 5200 cycles a step against 2300 of tcgen05.mma: 8192 rows over 2 x 131072 tokens,
// 3 bits, take 1.44 ms back to back (0.76 PFLOP/s), 4000 rows over 8 x 32768, 2 bits, 0.75 ms (0.72
// PFLOP/s).
#include <algorithm>

#include "gtq_attn.cuh"
#include "gtq_dequant.cuh"
#include "gtq_internal.h"
#include "gtq_tc.cuh"

namespace gtq {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kDqWarps = 8;
constexpr int kChunkThreads = 32 * (kSoftWarps + kDqWarps);
constexpr int kBlockTok = 128;     // tokens of a step
constexpr int kSplitSlots = 8;     // slots (pairs of coordinates) with a low part
// P = 2^(score - ref) is fp16, the row's ref 2^kTop below the maximum that set it, so the largest P
// lies in [2^kTop, 2^15]: a token keeps P's full precision down to 2^-25 of that maximum, and an
// absolute 2^-36 of it below.  (One token with .9999 of a row and a hundredth of the others' value, before
// 16384 of them: rows are off by 6e-4, and by 1.4e-2 with ref at the maximum and kRescale 8.)  kRescale 8, 4, 2, 1: 8192 rows over
// 2 x 131072 tokens take 1460, 1469, 1481, 1522 us.
constexpr float kRescale = 4.f;          // growth of the maximum (log2) that moves the reference
constexpr float kTop = 15.f - kRescale;  // log2 P of a maximum that does

// shared memory, from a 1024-byte boundary
constexpr uint32_t kQHi = 32768;                    // queries of 128 rows, fp16 (two swizzled atoms)
constexpr uint32_t kQLo = 4096;                     // their low parts, 16 coordinates
template <int NQ, bool PAIR>
struct Map {
  // the second operand's rows: all 128, or a CTA's half of them
  static constexpr uint32_t atom = PAIR ? 8192 : 16384;     // 64 columns of them, swizzled
  static constexpr uint32_t klo = 2 * atom;                 // keys of a step: two atoms, then their low parts
  static constexpr uint32_t kbuf = klo + (PAIR ? 2048 : 4096);
  static constexpr uint32_t image_bytes = 4 * atom;         // a rotation: hi and lo, two atoms each
  static constexpr uint32_t qhi = 0;
  static constexpr uint32_t qlo = qhi + NQ * kQHi;
  static constexpr uint32_t k = qlo + NQ * kQLo;
  static constexpr uint32_t v = k + 2 * kbuf;               // values of two steps, an atom a packed tile
  // before the steps: the keys' rotation image; after them: the values' image, then the low
  // parts of the outputs (their high parts lie where the queries were) and, for NQ = 1, the
  // second group's maxima and sums
  static constexpr uint32_t image = qlo;
  static constexpr uint32_t olo = image + image_bytes;
  static constexpr uint32_t olo_end = olo + NQ * 32768 + (NQ == 1 ? 1024 : 0), v_end = v + 4 * atom;
  static constexpr uint32_t tab = olo_end > v_end ? olo_end : v_end;
  static constexpr uint32_t misc = tab + kDqBytes;
  static constexpr uint32_t stat = tab - 1024;
};
struct Misc {
  alignas(16) HeadMeta m;
  alignas(16) float qscale[2][kD];  // each softmax group's
  uint64_t bar[18];
  uint32_t tmem;
};

// barriers
constexpr int kK0Full = 0;          // keys of the first step written
constexpr int kKEmpty = 2;          // [2] their products done
constexpr int kFull = 4;            // [2] values of a step and keys of the next written
constexpr int kVEmpty = 6;          // [2] their products done
constexpr int kSFull = 8;           // [2] scores written
constexpr int kImg = 10;            // rotation image landed
constexpr int kQRot = 11;           // products of a rotation done
constexpr int kQFull = 12;          // rotated queries written
constexpr int kOFull = 13;          // all steps' products done
constexpr int kDrain = 14;          // [2] after a failed wait: a group's products so far are done
constexpr int kHand = 16;           // [2] pairs: a group is done in both CTAs (raw queries, turned queries, every
                                    // step's probabilities, outputs)

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
  float* part_o;           // [heads][splits][rows padded][128]
  float2* part_ml;         // [heads][splits][rows padded]
  int64_t rows_pad;
  int* status;
};

// Probabilities 2^(score - ref), written back over the scores as fp16 (128 scores become 64
// columns); returns their sum, taken before they are rounded.
template <bool MASK>
__device__ __forceinline__ float row_exp(uint32_t s, int cnt, float ref) {
  const uint64_t neg = pack_f2(-ref, -ref);
  uint64_t s0 = 0, s1 = 0;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32], p[16];
    tc_ld32(s + 32 * c, r);
    tc_wait_ld();
    const int left = cnt - 32 * c;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float x, y;
      unpack_f2(add_f2(pack_f2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), neg), x, y);
      x = ex2(x);
      y = ex2(y);
      if (MASK) {
        x = e < left ? x : 0.f;
        y = e + 1 < left ? y : 0.f;
      }
      uint64_t& sum = (e & 2) ? s1 : s0;
      sum = add_f2(sum, pack_f2(x, y));
      p[e / 2] = pack_h2(x, y);
    }
    tc_st16(s + 16 * c, p);
  }
  tc_wait_st();
  float x, y;
  unpack_f2(add_f2(s0, s1), x, y);
  return x + y;
}

template <int NQ, bool PAIR>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  static_assert(NQ == 2 || !PAIR, "pairs have 512 rows");
  using M = Map<NQ, PAIR>;
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = su32(sm);
  if (sb & 1023u) {  // the swizzled operands need it; there is no room to spare for a shift
    if (threadIdx.x == 0) atomicOr(a.status, kStatusLayout);
    return;
  }
  Misc& ms = *reinterpret_cast<Misc*>(sm + M::misc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv;
  const int rank = PAIR ? cluster_rank() : 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int rt = unit % a.row_tiles, sp = unit / a.row_tiles;
  const int64_t len = a.sm.len(b, a.T), cl = chunk_len(a.chunk_lens, a.n, b), n_rows = cl * a.gq;
  constexpr int kUnitRows = 128 * NQ * (PAIR ? 2 : 1);
  const int64_t u0 = (int64_t)rt * kUnitRows;  // (rows fit 28 bits: 2^20 tokens of 128 heads)
  if (u0 >= n_rows) return;
  const int64_t r0 = u0 + rank * (128 * NQ);   // this CTA's own
  // tokens [s0, s1) of this block: its stretch, as far as its (pair's) last row sees
  const int64_t last_row = (u0 + kUnitRows < n_rows ? u0 + kUnitRows : n_rows) - 1;
  int64_t seen = a.causal ? len - cl + (int)last_row / a.gq + 1 : len;
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
  auto wait_on = [&](int i, uint32_t par) { return PAIR ? mbar_wait_pair(bar(i), par) : mbar_wait(bar(i), par); };
  auto commit = [&](int i) { PAIR ? tc_commit_pair(bar(i)) : tc_commit(bar(i)); };
  // a CTA's share of an image's rows: all, or 64 of each atom
  auto load_image = [&](const uint8_t* src) {
    mbar_expect_tx(bar(kImg), M::image_bytes);
    if (PAIR) {
      for (int i = 0; i < 4; ++i)
        bulk_load(sb + M::image + i * M::atom, src + i * 16384 + rank * M::atom, M::atom, bar(kImg));
    } else {
      bulk_load(sb + M::image, src, M::image_bytes, bar(kImg));
    }
  };

  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kHand + i), 2);
      mbar_init(bar(kKEmpty + i), NQ);
      mbar_init(bar(kFull + i), kDqWarps * (PAIR ? 2 : 1));
      mbar_init(bar(kVEmpty + i), NQ);
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kDrain + i), 1);
    }
    mbar_init(bar(kK0Full), kDqWarps * (PAIR ? 2 : 1));
    mbar_init(bar(kImg), 1);
    mbar_init(bar(kQRot), NQ);
    mbar_init(bar(kQFull), 4 * NQ);
    mbar_init(bar(kOFull), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    load_image(a.bimg_k + (size_t)head * 65536);
  }
  if (warp == 0) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&ms.tmem)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&ms.tmem)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ms.tmem, 0);  // the same in all lanes, and known to be
  launch_dependents();
  int failed = 0;

  if (warp < kSoftWarps) {
    // -------------------------------------------------------------- softmax
    const int grp = __shfl_sync(0xffffffffu, warp >> 2, 0), lrow = (warp & 3) * 32 + lane;  // row within its 128
    const bool issuer = __shfl_sync(0xffffffffu, (int)((warp & 3) == 0), 0);
    const int tile = NQ == 2 ? grp : 0;
    const int row = (int)r0 + 128 * tile + lrow;
    const bool mine = row < n_rows;
    const int tok = mine ? row / a.gq : 0;
    const int hq = h * a.gq + (mine ? row - tok * a.gq : 0);
    const bool warp_on = __any_sync(0xffffffffu, mine);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_off + 128u * grp, t_o = tmem + lane_off + 256u + 128u * grp;
    uint8_t* qhi = sm + M::qhi + tile * kQHi + lrow * 128;
    const uint32_t sw = (uint32_t)(lrow & 7);
    // A wait that has failed is not repeated, but every barrier of the group is still met.
    auto waits = [&](int i, uint32_t par) {
      if (!failed && !wait_on(i, par)) failed = 1;
      __syncwarp();
    };
    // The group has written an operand (or, with `img`, also an image is due): its issuer goes on.
    // Pairs: when the same group of both CTAs has, the even CTA's issuer does.
    int handed = 0;
    auto group_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(2 + grp) : "memory"); };
    auto hand = [&](int img) -> bool {
      group_sync();
      if (!issuer) return false;
      if (img >= 0) waits(kImg, (uint32_t)img);
      if (PAIR) {
        if (lane == 0) arrive_even(bar(kHand + grp));
        __syncwarp();
        if (rank) return false;
        waits(kHand + grp, (uint32_t)handed & 1u);
        ++handed;
      }
      tc_fence_after();
      return true;
    };
    // NQ = 2: the groups take turns with the exponentials.  Both at once would share the unit for
    // them, finish together and then share the tensor cores; in turns, one's products run during the
    // other's exponentials.
    auto my_turn = [&] { asm volatile("bar.sync %0, 256;" ::"r"(5 + grp) : "memory"); };
    auto your_turn = [&] { asm volatile("bar.arrive %0, 256;" ::"r"(6 - grp) : "memory"); };
    if (NQ == 2 && grp == 1) your_turn();
    // products of the group, issued by one lane of its first warp
    const uint32_t idc = PAIR ? idesc_f16_pair(128) : idesc_f16(128);
    auto mma = [&](uint32_t d, uint64_t x, uint64_t y, uint32_t acc) {
      PAIR ? tc_mma_pair(d, x, y, idc, acc) : tc_mma(d, x, y, idc, acc);
    };
    auto bstep = [](uint32_t ks) { return (uint64_t)(((ks >> 2) * M::atom + (ks & 3) * 32) >> 4); };
    const uint32_t d_s = tmem + 128u * grp, d_o = tmem + 256u + 128u * grp;
    auto rotate = [&](uint32_t x, bool more, bool with_lo) {
      // scores (+)= x . (hi + lo)^T of the image (with_lo), or x . hi^T
      const uint64_t dx = smem_desc(sb + x), di = smem_desc(sb + M::image);
#pragma unroll 1
      for (int part = 0; part < (with_lo ? 2 : 1); ++part)
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma(d_s, dx + kstep(ks), di + bstep(ks) + part * (2 * M::atom >> 4), more || (part | ks) != 0);
    };
    auto scores = [&](int j) {
      const uint32_t kb = sb + M::k + (j & 1) * M::kbuf;
      const uint64_t dq = smem_desc(sb + M::qhi + tile * kQHi), dk = smem_desc(kb);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) mma(d_s, dq + kstep(ks), dk + bstep(ks), ks != 0);
      mma(d_s, smem_desc_plain(sb + M::qlo + tile * kQLo, 128, 256), dk, 1);
      mma(d_s, dq, smem_desc_plain(kb + M::klo, 128, 256), 1);
      commit(kSFull + grp);
      commit(kKEmpty + (j & 1));
    };
    auto outputs = [&](int j, bool more) {
      const uint64_t dv = smem_desc(sb + M::v + (j & 1) * 2 * M::atom);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        PAIR ? tc_mma_ta_pair(d_o, d_s + 8u * ks, dv + bstep(ks), idc, more || ks != 0)
             : tc_mma_ta(d_o, d_s + 8u * ks, dv + bstep(ks), idc, more || ks != 0);
      commit(kVEmpty + (j & 1));
    };
    const int first = NQ == 2 ? 0 : grp, stride = NQ == 2 ? 1 : 2;  // the group's steps
    // raw queries -> operand, rotated by the tensor cores, back as scaled hi + lo
    if (NQ == 2 || grp == 0) {
      ms.qscale[grp][lrow] = query_scale(a.meta[head], lrow);
      put_query_row(sm + M::qhi + tile * kQHi, lrow,
                    reinterpret_cast<const uint4*>(a.q + b * a.qs[0] + hq * a.qs[1] + tok * a.qs[2]), mine);
      fence_async();
      if (hand(0)) {
        if (elect_one() && !failed) {
          rotate(M::qhi + tile * kQHi, false, true);
          commit(kQRot);
        }
        __syncwarp();
      }
      waits(kQRot, 0);
      tc_fence_after();
      uint8_t* qlo = sm + M::qlo + tile * kQLo + (lrow >> 3) * 256 + (lrow & 7) * 16;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tc_ld32(t_s + 32 * c, r);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 8 coordinates each
          const int ch = 4 * c + k;
          uint4 hi, lo;
          split8(r + 8 * k, ms.qscale[grp] + 8 * ch, hi, lo);
          *reinterpret_cast<uint4*>(qhi + (ch >> 3) * 16384 + (((ch & 7) ^ sw) << 4)) = hi;
          if (ch < 2) *reinterpret_cast<uint4*>(qlo + ch * 128) = lo;
        }
      }
      tc_fence_before();
      fence_async();
      __syncwarp();
      if (!PAIR && lane == 0) mbar_arrive(bar(kQFull));
    }
    // steps
    // tokens this row sees; a row that is not there (zeros, its result goes nowhere) keeps its warp
    // from masking by seeing whole steps
    int64_t end = a.causal ? len - cl + tok + 1 : len;
    if (end > s1) end = s1;
    if (!mine) end = s0 + (int64_t)nb * kBlockTok;
    float ref = -INFINITY, sum = 0.f;
    int it = 0;
    if (PAIR ? hand(-1) : issuer && first < nb) {  // the first scores
      if (!PAIR) waits(kQFull, 0);
      if (first == 0) waits(kK0Full, 0);
      else waits(kFull, 0);
      tc_fence_after();
      if (elect_one() && !failed) scores(first);
      __syncwarp();
    }
#pragma unroll 1
    for (int j = first; j < nb; j += stride, ++it) {
      waits(kSFull + grp, it & 1);
      tc_fence_after();
      const int64_t left = end - (s0 + (int64_t)j * kBlockTok);
      const int cnt = left < 0 ? 0 : (left < kBlockTok ? (int)left : kBlockTok);
      const bool whole = __all_sync(0xffffffffu, cnt == kBlockTok);
      if (warp_on) {
        const float mx = whole ? row_max<false>(t_s, cnt) : row_max<true>(t_s, cnt);
        const bool grow = mx > ref + (kTop + kRescale);  // also out of -inf
        if (__any_sync(0xffffffffu, grow)) {
          const float now = grow ? mx - kTop : ref;
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
      }
      if (NQ == 2) my_turn();
      if (warp_on) {
        const float base = ref == -INFINITY ? 0.f : ref;
        sum += whole ? row_exp<false>(t_s, cnt, base) : row_exp<true>(t_s, cnt, base);
      }
      if (NQ == 2 && (grp == 0 || j + 1 < nb)) your_turn();
      tc_fence_before();
      if (hand(-1)) {
        waits(kFull + (j & 1), (j >> 1) & 1);
        tc_fence_after();
        const int nj = j + stride;
        if (elect_one() && !failed) {
          outputs(j, it > 0);
          if (NQ == 2 && nj < nb) scores(nj);
        }
        __syncwarp();
        if (NQ == 1 && nj < nb) {  // its keys come with the other group's values
          waits(kFull + ((j + 1) & 1), ((j + 1) >> 1) & 1);
          tc_fence_after();
          if (elect_one() && !failed) scores(nj);
          __syncwarp();
        }
      }
    }
    if (issuer && rank == 0 && elect_one()) commit(kOFull);
    __syncwarp();
    // outputs: normalised, split into hi + lo operands of the last product
    waits(kOFull, 0);
    tc_fence_after();
    if (warp == 0 && lane == 0 && !failed) {  // the operands' memory is free: the values' rotation
      load_image(a.img_vt);
    }
    __syncwarp();
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
      // the values' factor (a row with a NaN in its query has a NaN here)
      const float inv = total == 0.f ? 0.f : 0.08838834764831845f / kElement / total;
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
              float v = warp_on && f0 != 0.f ? __uint_as_float(r[at]) * f0 : 0.f;
              if (two && warp_on && f1 != 0.f) v = fmaf(__uint_as_float(u[at]), f1, v);
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
      if (hand(1)) {
        if (elect_one() && !failed) {
          rotate(M::qhi + tile * kQHi, false, true);
          rotate(M::olo + tile * 32768, true, false);
          commit(kQRot);
        }
        __syncwarp();
      }
      waits(kQRot, 1);
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
        // (maxima pass over a NaN: any finite one lets its sum count)
        if (split && mine) a.part_ml[slot0 + 128 * tile + lrow] = make_float2(total != total ? 0.f : top, total);
      }
    }
  } else {
    // ------------------------------------------------------ codes to operands
    const int dw = warp - kSoftWarps, dtid = tid - 32 * kSoftWarps;
    const uint32_t tab = sb + M::tab;
    for (int i = dtid; i < (int)(sizeof(HeadMeta) / 4); i += 32 * kDqWarps)
      reinterpret_cast<uint32_t*>(&ms.m)[i] = reinterpret_cast<const uint32_t*>(a.meta + head)[i];
    load_dequant_tables<false>(sm + M::tab, a.dec_image, dtid, 32 * kDqWarps);
    asm volatile("bar.sync 4, %0;" ::"n"(32 * kDqWarps) : "memory");
    // Keys: quads dw and 15 - dw of both tiles of a step, or (pairs) of this CTA's one, whose tokens
    // are its half of the operand's rows.  Values: 16 dims of both tiles, or (pairs) of one of them,
    // among this CTA's 64 dims.
    constexpr int KT = PAIR ? 1 : 2;
    const uint32_t norms = key_norm_offset(a.kb, a.vb);
    const KeyLane k0 = key_lane(ms.m, dw, lane, M::atom, norms, tab);
    const KeyLane k1 = key_lane(ms.m, 15 - dw, lane, M::atom, norms, tab);
    const bool low = dw < kSplitSlots / 4;  // slots of quad dw leave low parts
    const bool code0 = low || __any_sync(0xffffffffu, k0.w > 4), code1 = __any_sync(0xffffffffu, k1.w > 4);
    const uint32_t lo_lane = (uint32_t)dw * 128 + 16u * (lane & 7) + 4u * (lane >> 3);
    const int vstep = PAIR ? 4 * rank + (dw & 3) : dw;
    auto key_tile = [&](int j, int i) { return 2 * j + (PAIR ? rank : i); };
    auto value_tile = [&](int j, int i) { return 2 * j + (PAIR ? dw >> 2 : i); };
    // addresses: page numbers are read a step ahead of their use
    const int64_t t0 = s0 / kTile;
    const uint8_t* const base = a.packed + (a.sm.table ? (int64_t)h * a.sm.tile_bytes
                                                       : ((int64_t)head * a.sm.n_tiles + t0) * a.sm.tile_bytes);
    const int32_t* const pages = a.sm.table ? a.sm.table + (int64_t)b * a.sm.max_blocks + t0 : nullptr;
    auto read_page = [&](int t, int& page) {
      if (pages && t < nt) page = __ldg(pages + t);
    };
    auto tile_of = [&](int t, int page) {
      return base + (pages ? (int64_t)page * a.sm.hkv : (int64_t)t) * a.sm.tile_bytes;
    };
    int kpage[KT] = {}, vpage[KT] = {};
    const uint8_t *kp[KT], *vp[KT];
    KeyRaw r0[KT], r1[KT];
    ValueRaw rv[KT];
    auto fetch_keys = [&](int j) {
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const int t = key_tile(j, i);
        if (t < nt) {
          kp[i] = tile_of(t, kpage[i]);
          if (code0) load_keys<5>(r0[i], kp[i], k0);
          else load_keys<2>(r0[i], kp[i], k0);
          if (!code1) load_keys<2>(r1[i], kp[i], k1);
        }
        read_page(key_tile(j + 1, i), kpage[i]);
      }
    };
    auto put_keys = [&](int j) {
      const uint32_t dst = sb + M::k + (j & 1) * M::kbuf;
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        // rows behind the last tile: whatever they hold, their scores do not count
        if (key_tile(j, i) >= nt) continue;
        const uint32_t row = dst + i * 8192;
        if (code0) keys_by_code<false>(k0, r0[i], tab, row, low, dst + M::klo + i * 2048 + lo_lane, 256);
        else keys_by_pair(k0, r0[i], row);
        if (!code1) {
          keys_by_pair(k1, r1[i], row);
        } else {  // widths above 4 beyond the first half of the slots: fetched when they are due
          KeyRaw r;
          load_keys<5>(r, kp[i], k1);
          keys_by_code<false>(k1, r, tab, row, false, 0, 0);
        }
      }
    };
    auto arrive = [&](int i) { PAIR ? arrive_even(bar(i)) : mbar_arrive(bar(i)); };
#pragma unroll
    for (int i = 0; i < KT; ++i) {
      read_page(key_tile(0, i), kpage[i]);
      read_page(value_tile(0, i), vpage[i]);
    }
    fetch_keys(0);
    // the keys' buffers lie under the rotation image
    if (!wait_on(kQRot, 0)) failed = 1;
    __syncwarp();
    if (!failed) {
      put_keys(0);
      fence_async();
      __syncwarp();
      if (lane == 0) arrive(kK0Full);
      if (nb > 1) fetch_keys(1);
    }
    // step by step: the keys of step j + 1, then the values of step j (a fence costs as much as
    // a portion's work: one for both)
#pragma unroll 1
    for (int j = 0; j < nb && !failed; ++j) {
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const int t = value_tile(j, i);
        if (t < nt) {
          vp[i] = tile_of(t, vpage[i]);
          load_values(rv[i], vp[i], a.kb, a.vb, vstep, lane);
        }
        read_page(value_tile(j + 1, i), vpage[i]);
      }
      if (j + 1 < nb) {
        if (j >= 1 && !wait_on(kKEmpty + ((j + 1) & 1), (((j + 1) >> 1) & 1) ^ 1)) { failed = 1; break; }
        __syncwarp();
        put_keys(j + 1);
      }
      if (j + 2 < nb) fetch_keys(j + 2);  // in flight during the values
      // and what is due two steps later, towards the L2 cache (the warps take turns; a pair's CTAs a
      // tile each)
      if (lane == 0 && (j & 7) == dw)
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int t = key_tile(j + 4, i);
          if (t < nt)
            bulk_prefetch(base + (pages ? (int64_t)__ldg(pages + t) * a.sm.hkv : (int64_t)t) * a.sm.tile_bytes,
                          (uint32_t)a.sm.tile_bytes);
        }
      if (j >= 2 && !wait_on(kVEmpty + (j & 1), ((j >> 1) & 1) ^ 1)) { failed = 1; break; }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const int t = value_tile(j, i);
        const uint32_t atom = M::v + (2 * (j & 1) + (t & 1)) * M::atom;
        const uint32_t first_row = PAIR ? (uint32_t)rank * 8192u : 0u;  // dim 16 vstep lies 2048 vstep behind dim 0
        if (t < nt) {
          const int64_t left = s1 - (s0 + (int64_t)t * kTile);
          uint32_t n[8];
          value_norms(rv[i], lane, left < kTile ? (int)left : kTile, n);
          dequant_values(vp[i], a.kb, a.vb, vstep, lane, rv[i], n, tab, sb + atom - first_row);
        } else {  // no tile: zeros, since the probabilities' zeros must not meet a NaN
          for (int k = lane; k < 128; k += 32)
            *reinterpret_cast<uint4*>(sm + atom - first_row + vstep * 2048 + 16 * k) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) arrive(kFull + (j & 1));
    }
  }
  if (failed) atomicOr(a.status, kStatusTimeout);
  // After a failed wait, nothing in flight may outlive the block: each issuer waits (bounded) for
  // its products so far, and the images' copies are waited for.
  if (__syncthreads_or(failed)) {
    if (warp == 0 || warp == 4) {
      if (elect_one()) {  // the lane that issued them
        if (rank == 0) commit(kDrain + (warp >> 2));
        wait_on(kDrain + (warp >> 2), 0);
      }
    }
    if (tid == 0) {
      mbar_wait(bar(kImg), 0);
      mbar_wait(bar(kImg), 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) {
    cluster_sync_all();  // nothing of the other CTA is touched past this point
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  } else if (warp == 0) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// The splits' outputs of a row, weighted by what their maxima and sums say.  WPR warps a row: one
// where there are many rows, eight where there are few rows of many splits.
template <int WPR>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ float4 part[8][32];
  __shared__ float part_sum[8];
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (int)blockIdx.x * (8 / WPR) + warp / WPR, mine = warp % WPR;
  const int64_t cl = chunk_len(a.chunk_lens, a.n, b);
  wait_dependency();  // every block: this kernel ends after the one before it
  if ((int64_t)(blockIdx.x * (8 / WPR)) >= cl * a.gq) return;
  const bool on = row < cl * a.gq;
  const int64_t base = (int64_t)head * a.splits * a.rows_pad + row;
  float top = -INFINITY;
  if (on)
    for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_ml[base + s * a.rows_pad].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  if (top != -INFINITY)
#pragma unroll 4
    for (int s = mine; s < a.splits; s += WPR) {
      const float2 ml = a.part_ml[base + s * a.rows_pad];
      const float w = ml.y * ex2(ml.x - top);
      // (what a split without a visible token left is not read as a number)
      const float4 o = w > 0.f ? reinterpret_cast<const float4*>(a.part_o + (base + s * a.rows_pad) * kD)[lane]
                               : make_float4(0.f, 0.f, 0.f, 0.f);
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
      total += w;
    }
  if (WPR > 1) {
    part[warp][lane] = acc;
    if (lane == 0) part_sum[warp] = total;
    __syncthreads();
    if (mine) return;
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      const float4 o = part[warp + k][lane];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
      total += part_sum[warp + k];
    }
  }
  if (!on) return;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int tok = row / a.gq;
  __half* out = a.out + b * a.os[0] + (h * a.gq + row - tok * a.gq) * a.os[1] + tok * a.os[2];
  *reinterpret_cast<uint2*>(out + 4 * lane) =
      make_uint2(pack_h2(acc.x * inv, acc.y * inv), pack_h2(acc.z * inv, acc.w * inv));
}

// One new token a sequence is a decode step: launch_decode reads codes straight into registers
// and has nothing to set up for rows that are not there.  These two kernels are the difference:
// queries and tickets before it, fp16 rows after it.
__global__ void __launch_bounds__(128) token_in_kernel(const __half* q, int64_t qs0, int64_t qs1, int hq,
                                                       uint4* rows, int n_rows, unsigned* tickets, int n_tickets) {
  const int i = blockIdx.x * 128 + threadIdx.x;  // 16 bytes of a row
  if (i < n_rows * 16) {
    const int row = i >> 4;
    rows[i] = reinterpret_cast<const uint4*>(q + (row / hq) * qs0 + (row % hq) * qs1)[i & 15];
  }
  for (int t = i; t < n_tickets; t += gridDim.x * 128) tickets[t] = 0;
}
__global__ void __launch_bounds__(128) token_out_kernel(const float4* rows, int n_rows, __half* out, int64_t os0,
                                                        int64_t os1, int hq, const int32_t* chunk_lens) {
  const int i = blockIdx.x * 128 + threadIdx.x;
  if (i >= n_rows * 16) return;
  const int row = i >> 4, b = row / hq;
  if (chunk_lens && chunk_lens[b] < 1) return;
  const float4 x = rows[2 * i], y = rows[2 * i + 1];
  reinterpret_cast<uint4*>(out + b * os0 + (row % hq) * os1)[i & 15] =
      make_uint4(pack_h2(x.x, x.y), pack_h2(x.z, x.w), pack_h2(y.x, y.y), pack_h2(y.z, y.w));
}

// Workspace of a decode step: queries, results, and the split-merge state that the plan's own
// decodes keep in the plan.
struct TokenSpace {
  size_t rows, out, tickets, partials, total;
  int n_rows, n_tickets;
  explicit TokenSpace(const gtq_plan* p) {
    n_rows = p->cfg.batch * p->cfg.n_q_heads;
    n_tickets = p->n_units * kTicketStride;
    rows = 0;
    out = rows + (size_t)n_rows * kD * sizeof(__half);
    tickets = out + (size_t)n_rows * kD * sizeof(float);
    partials = (tickets + (size_t)n_tickets * sizeof(unsigned) + 255) & ~(size_t)255;
    total = partials + (size_t)p->n_units * PartialSlots(decode_split_cap(p->n_sms, p->n_units)).total * 8 *
                           kPartialStride * sizeof(float);
  }
};
cudaError_t launch_token(const gtq_plan* p, const uint8_t* packed, int64_t T, const SeqMap& sm, const gtq_chunk& ch,
                         const __half* q, __half* out, uint8_t* ws, cudaStream_t s) {
  const TokenSpace t(p);
  gtq_plan own = *p;  // the caller's workspace in the place of the plan's
  own.d_tickets = reinterpret_cast<unsigned*>(ws + t.tickets);
  own.d_partials = reinterpret_cast<float*>(ws + t.partials);
  const int blocks = (t.n_rows * 16 + 127) / 128;
  token_in_kernel<<<blocks, 128, 0, s>>>(q, ch.q_strides[0], ch.q_strides[1], p->cfg.n_q_heads,
                                         reinterpret_cast<uint4*>(ws + t.rows), t.n_rows, own.d_tickets, t.n_tickets);
  cudaError_t e = launch_decode(&own, packed, T, ws + t.rows, GTQ_DTYPE_FP16, reinterpret_cast<float*>(ws + t.out),
                                sm, Fp16Kv(), s);
  if (e != cudaSuccess) return e;
  token_out_kernel<<<blocks, 128, 0, s>>>(reinterpret_cast<const float4*>(ws + t.out), t.n_rows, out,
                                          ch.out_strides[0], ch.out_strides[1], p->cfg.n_q_heads, ch.chunk_lens_dev);
  return cudaGetLastError();
}

// How a call is cut: rows per block and splits of the tokens.
struct Cut {
  int nq, pair, row_tiles, splits;
  int64_t span, rows_pad;
  uint32_t smem;
};

template <int NQ, bool PAIR>
constexpr uint32_t smem_of() {
  return Map<NQ, PAIR>::misc + (uint32_t)sizeof(Misc);
}
static_assert(smem_of<2, false>() <= 232448 && smem_of<2, true>() <= 232448, "shared memory of a block");

Cut cut_of(const gtq_plan* p, int64_t T, int64_t n) {
  Cut c;
  const int64_t rows = n * p->g_q;
  // Up to 128 rows, one tile of them (16 rows over 2 x 131072 tokens: 60 us against 66 with a second,
  // empty one).  Pairs, where they do not have more rows to fill up: 768 rows, which would be 1024,
  // take 224 us against 169.  8 heads of 4096 rows over 32768 tokens, with pairs and without, at 2, 3
  // and 4 bits: paged 751 and 822, 751 and 792, 748 and 860 us; contiguous 775 and 779, 781 and 754, 753
  // and 826.  Contiguous caches at 3 bits are the one case that loses (2 heads of 8192 rows over 131072
  // tokens: 1445 and 1421); why a contiguous cache takes longer than a paged one is not known, so
  // the rule does not go by it.
  const int64_t tiles = (rows + 255) / 256;
  c.nq = rows > 128 ? 2 : 1;
  c.pair = tiles > 1 && 24 * (tiles + (tiles & 1)) <= 25 * tiles;
  c.smem = c.pair ? smem_of<2, true>() : (c.nq == 2 ? smem_of<2, false>() : smem_of<1, false>());
  const int64_t unit = 128 * c.nq * (c.pair ? 2 : 1);
  c.row_tiles = (int)((rows + unit - 1) / unit);
  c.rows_pad = (int64_t)c.row_tiles * unit;
  // Splits: enough blocks (pairs) to fill the SMs, and evenly; a block's set-up and end cost about
  // as much as 6 steps, a merge more the more parts there are.
  const int64_t units = (int64_t)p->n_heads * c.row_tiles, steps = (T + kBlockTok - 1) / kBlockTok;
  const int64_t at_once = c.pair ? p->n_sms / 2 : p->n_sms;
  double best = 1e300;
  int64_t best_steps = steps;
  for (int64_t s = 1; s <= 256 && s <= steps; ++s) {
    const int64_t per = (steps + s - 1) / s, parts = (steps + per - 1) / per;
    const int64_t waves = (units * parts + at_once - 1) / at_once;
    const double cost = (double)waves * (per + 6.0) + (parts > 1 ? 2.0 + 0.01 * parts * c.rows_pad * p->n_heads / 256 / p->n_sms : 0.0);
    if (cost < best * 0.999) {
      best = cost;
      best_steps = per;
    }
    if (units * s > 64 * at_once) break;
  }
  c.span = best_steps * kBlockTok;
  c.splits = (int)((steps + best_steps - 1) / best_steps);
  return c;
}

}  // namespace

size_t chunk_workspace(const gtq_plan* p, int64_t T, int64_t n) {
  if (n == 1) return TokenSpace(p).total;
  const Cut c = cut_of(p, T, n);
  if (c.splits <= 1) return 256;
  const size_t slots = (size_t)p->n_heads * c.splits * c.rows_pad;
  return slots * (kD * sizeof(float) + sizeof(float2));
}

cudaError_t launch_chunk(const gtq_plan* p, const uint8_t* packed, int64_t T, const SeqMap& sm,
                         const gtq_chunk& ch, const __half* q, __half* out, uint8_t* workspace,
                         cudaStream_t s) {
  // One token: 16 sequences x 4 KV heads of 7 queries, up to 16384 tokens each, take 91 us this way
  // and 213 us as a chunk, whose products are then mostly of rows that are not there.
  if (ch.n_tokens == 1) return launch_token(p, packed, T, sm, ch, q, out, workspace, s);
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
  a.rows_pad = c.rows_pad;
  a.status = p->d_status;
  const size_t slots = (size_t)p->n_heads * c.splits * c.rows_pad;
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(workspace + slots * kD * sizeof(float));
  auto kernel = c.pair ? chunk_kernel<2, true> : (c.nq == 2 ? chunk_kernel<2, false> : chunk_kernel<1, false>);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(c.row_tiles * c.splits * (c.pair ? 2 : 1)), (unsigned)p->n_heads);
  cfg.blockDim = dim3(kChunkThreads);
  cfg.dynamicSmemBytes = c.smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c.pair ? 2 : 1;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess || c.splits == 1) return e;
  const int64_t rows = ch.n_tokens * p->g_q;
  // eight warps a row from eight parts on (64 rows in about 70 parts: 61 us for the call, 80 with one
  // warp a row); with fewer, one (8 heads of 1024 rows in a few parts: 232 us, 241 with eight)
  if (c.splits >= 8)
    return launch_overlapped(merge_kernel<8>, dim3((unsigned)rows, (unsigned)p->n_heads), 256, 0, s, a);
  return launch_overlapped(merge_kernel<1>, dim3((unsigned)((rows + 7) / 8), (unsigned)p->n_heads), 256, 0, s, a);
}

}  // namespace gtq
