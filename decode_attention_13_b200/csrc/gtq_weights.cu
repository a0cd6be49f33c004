// Attention weights that a chunk gives every cached token (include/gtq.h,
// gtq_attn_weights): w_t += sum over rows r of exp(s_rt) / sum_t' exp(s_rt').
//
// Two passes over the keys, since a row's sum has to be known before any of its
// weights: pass 0 leaves every row's maximum and sum (one pair per stretch of
// tokens), pass 1 the sums over rows.  Each pass is a kernel like the chunk's
// (gtq_chunk.cu): a block takes up to 128 rows of one KV head and a stretch of its
// tokens, eight warps turn codes into fp16 operands, scores are tcgen05.mma
// products into tensor memory, and two groups of four warps read them in turns.
// Pass 0 has rows on the lanes (a thread keeps one row's maximum and sum); pass 1
// swaps the operands, so that tokens are on the lanes and a thread adds one token's
// weights over the rows, in order: no atomics, the same bits every time.
//
// The result is fp32, so scores are q (hi + lo) . k (hi + lo) without lo . lo: three
// products of fp16 halves carry about 22 bits of each factor (128 rows over 8 x 32768 tokens:
// weights within 1.2e-6 of those in 64 bits, fp32 products 1.1e-6).
//
// With up to kKeepRows rows of a KV head, pass 0 leaves the scores themselves (4 bytes a row
// and token) and kept_kernel takes the place of pass 1: writing and reading them costs less than
// turning the codes into operands again.  Kept and turned again, us back to back, at 8, 16, 24 and 32
// rows: 2 heads of 131072 tokens 48 66, 58 67, 70 67, 81 68; 8 of 32768 47 66, 53 66, 61 67, 70 67; 64 of
// 16384 161 233, 181 233, 209 236, 245 236; 32 of 8192 48 69, 53 69, 60 70, 69 70.
// Rows beyond 128 of a KV head are more blocks, whose sums lie side by side in the
// workspace until add_kernel joins them in order.
//
// Bound by turning codes into operands, as chunks of few rows are: both passes read the keys'
// codes and norms, 18 MB over 2 x 131072 tokens at 3 bits (51 us for 8 rows), 13 MB over
// 8 x 32768 at 2 bits (128 rows: 76 us).  A pair of codes is one lookup for hi and one for lo,
// and each tile of a step has registers of its own, filled a step ahead: code by code and a tile
// ahead took 53 and 80 us.
#include <algorithm>

#include "gtq_attn.cuh"
#include "gtq_dequant.cuh"
#include "gtq_internal.h"
#include "gtq_tc.cuh"

namespace gtq {
namespace {

constexpr int kReadWarps = 8;
constexpr int kDqWarps = 8;
constexpr int kThreadsW = 32 * (kReadWarps + kDqWarps);
constexpr int kStepTok = 128;
constexpr int kRowsW = 128;
constexpr int kKeepRows = 16;  // rows whose scores are kept
constexpr int kAheadW = 8;   // packed tiles between a prefetch and its use

// shared memory: queries and two steps of keys, each fp16 hi and lo (two swizzled atoms a part)
constexpr uint32_t kPart = 32768;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = 2 * kPart;
constexpr uint32_t kOffTab = kOffK + 4 * kPart;
constexpr uint32_t kOffMisc = kOffTab + 2 * kDqBytes;  // pair tables, then their low parts
constexpr uint32_t kImageBytes = 65536;  // the keys' rotation, under the keys until the queries are turned
struct MiscW {
  alignas(16) HeadMeta m;
  alignas(16) float qscale[kD];
  alignas(16) float2 stat[kRowsW];  // pass 0: the second group's rows; pass 1: maximum, 1 / sum
  int end[kRowsW];                  // pass 1: tokens of the stretch that a row sees
  uint64_t bar[12];
  uint32_t tmem;
};
constexpr uint32_t kSmemW = kOffMisc + (uint32_t)sizeof(MiscW);
static_assert(kSmemW <= 232448, "shared memory of a block");

constexpr int kKFull = 0;   // [2] keys of a step written
constexpr int kKEmpty = 2;  // [2] their products done
constexpr int kSFull = 4;   // [2] scores written
constexpr int kImg = 6;
constexpr int kQRot = 7;
constexpr int kQFull = 8;
constexpr int kDrain = 9;   // [2]

struct WeightArgs {
  const uint8_t* packed;
  SeqMap sm;
  int64_t T;
  const __half* q;
  int64_t qs[3];
  int64_t n;
  const int32_t* chunk_lens;
  int causal, gq, hkv, kb, vb;
  const HeadMeta* meta;
  const uint8_t* bimg_k;
  const uint4* dec_image;
  const float* w_in;
  float* w_out;
  int64_t ws[2];
  int row_tiles, splits, n_heads, rows_kept;
  int64_t span, rows_pad;
  float2* part_ml;  // [heads][splits][rows_pad]
  float* part_w;    // [row tiles][heads][T], when there are several row tiles
  float* kept;      // [heads][rows][kept_stride] scores, or null
  int64_t kept_stride;
  int* status;
};

template <int PASS>
__global__ void __launch_bounds__(kThreadsW, 1) weights_kernel(const __grid_constant__ WeightArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = su32(sm);
  if (sb & 1023u) {  // the swizzled operands need it
    if (threadIdx.x == 0) atomicOr(a.status, kStatusLayout);
    return;
  }
  MiscW& ms = *reinterpret_cast<MiscW*>(sm + kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv;
  const int rt = blockIdx.x % a.row_tiles, sp = blockIdx.x / a.row_tiles;
  const int64_t len = a.sm.len(b, a.T), cl = chunk_len(a.chunk_lens, a.n, b), n_rows = cl * a.gq;
  const int64_t r0 = (int64_t)rt * kRowsW, s0 = sp * a.span;
  const int rows = (int)(n_rows - r0 < 0 ? 0 : (n_rows - r0 < kRowsW ? n_rows - r0 : kRowsW));
  int64_t seen = len;
  if (PASS == 0 && a.causal && rows) seen = len - cl + ((int)r0 + rows - 1) / a.gq + 1;
  const int64_t s1 = seen < s0 + a.span ? seen : s0 + a.span;
  float2* ml = a.part_ml + ((int64_t)head * a.splits + sp) * a.rows_pad + r0;
  float* out = nullptr;
  const float* in = nullptr;
  if (PASS == 1) {
    const int64_t at = b * a.ws[0] + h * a.ws[1];
    if (a.row_tiles == 1) {
      out = a.w_out + at;
      in = a.w_in ? a.w_in + at : nullptr;
    } else {
      out = a.part_w + ((int64_t)rt * a.n_heads + head) * a.T;
    }
  }
  if (rows == 0 || s0 >= s1) {
    if (PASS == 1) wait_dependency();  // this kernel ends after the one before it
    if (PASS == 0) {
      for (int r = tid; r < rows; r += kThreadsW) ml[r] = make_float2(-INFINITY, 0.f);
    } else if (a.row_tiles == 1) {  // no row: what was there stays
      for (int64_t t = s0 + tid; t < s1; t += kThreadsW) out[t] = in ? in[t] : 0.f;
    }
    return;
  }
  const int nb = (int)((s1 - s0 + kStepTok - 1) / kStepTok), nt = (int)((s1 - s0 + kTile - 1) / kTile);
  const uint32_t bar0 = su32(ms.bar);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };

  // ---------------------------------------------------------------- set-up
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKFull + i), kDqWarps);
      mbar_init(bar(kKEmpty + i), 1);
      mbar_init(bar(kSFull + i), 1);
      mbar_init(bar(kDrain + i), 1);
    }
    mbar_init(bar(kImg), 1);
    mbar_init(bar(kQRot), 1);
    mbar_init(bar(kQFull), 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_expect_tx(bar(kImg), kImageBytes);
    bulk_load(sb + kOffK, a.bimg_k + (size_t)head * kImageBytes, kImageBytes, bar(kImg));
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(su32(&ms.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ms.tmem, 0);
  launch_dependents();
  int failed = 0;

  if (warp < kReadWarps) {
    // ------------------------------------------------- products and their readers
    const int grp = __shfl_sync(0xffffffffu, warp >> 2, 0), lrow = (warp & 3) * 32 + lane;
    const bool issuer = __shfl_sync(0xffffffffu, (int)((warp & 3) == 0), 0);
    const uint32_t t_s = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128u * grp, d_s = tmem + 128u * grp;
    auto waits = [&](int i, uint32_t par) {  // a failed wait is not repeated; barriers are still met
      if (!failed && !mbar_wait(bar(i), par)) failed = 1;
      __syncwarp();
    };
    auto group_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(2 + grp) : "memory"); };
    // columns of a product: 128 tokens, or the rows in sixteens
    const int n_cols = PASS == 0 ? kStepTok : (rows + 15) & ~15;
    const uint32_t idc = idesc_f16(n_cols);
    auto scores = [&](int j) {
      const uint64_t q = smem_desc(sb + kOffQ), k = smem_desc(sb + kOffK + (j & 1) * 2 * kPart);
      const uint64_t x = PASS == 0 ? q : k, y = PASS == 0 ? k : q;
#pragma unroll 1
      for (int part = 0; part < 3; ++part) {  // lo . hi, hi . lo, hi . hi
        const uint64_t px = x + (part == 0 ? kPart >> 4 : 0), py = y + (part == 1 ? kPart >> 4 : 0);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) tc_mma(d_s, px + kstep(ks), py + kstep(ks), idc, (part | ks) != 0);
      }
      tc_commit(bar(kSFull + grp));
      tc_commit(bar(kKEmpty + (j & 1)));
    };
    if (grp == 0) {  // queries: raw operand, turned by the tensor cores, back as scaled hi + lo
      const int row = (int)r0 + lrow;
      const bool mine = lrow < rows;
      const int tok = mine ? row / a.gq : 0;
      const int hq = h * a.gq + (mine ? row - tok * a.gq : 0);
      ms.qscale[lrow] = query_scale(a.meta[head], lrow);
      put_query_row(sm + kOffQ, lrow,
                    reinterpret_cast<const uint4*>(a.q + b * a.qs[0] + hq * a.qs[1] + tok * a.qs[2]), mine);
      fence_async();
      group_sync();
      if (issuer) {
        waits(kImg, 0);
        tc_fence_after();
        if (elect_one() && !failed) {
          const uint64_t dx = smem_desc(sb + kOffQ), di = smem_desc(sb + kOffK);
#pragma unroll 1
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma(d_s, dx + kstep(ks), di + kstep(ks) + part * (kPart >> 4), idesc_f16(128), (part | ks) != 0);
          tc_commit(bar(kQRot));
        }
        __syncwarp();
      }
      waits(kQRot, 0);
      tc_fence_after();
      uint8_t* qh = sm + kOffQ + lrow * 128;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tc_ld32(t_s + 32 * c, r);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int ch = 4 * c + k;
          uint4 hi, lo;
          split8(r + 8 * k, ms.qscale + 8 * ch, hi, lo);
          uint8_t* o = qh + (ch >> 3) * 16384 + (((ch & 7) ^ (lrow & 7)) << 4);
          *reinterpret_cast<uint4*>(o) = hi;
          *reinterpret_cast<uint4*>(o + kPart) = lo;
        }
      }
      tc_fence_before();
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kQFull));
    }
    if (PASS == 1) {  // every row's softmax, from its stretches; the other group turns the queries
      if (grp == 1) {
        wait_dependency();
        const int r = lrow;
        float top = -INFINITY, total = 0.f;
        if (r < rows) {
          const float2* p = a.part_ml + (int64_t)head * a.splits * a.rows_pad + r0 + r;
#pragma unroll 4
          for (int s = 0; s < a.splits; ++s) top = fmaxf(top, p[s * a.rows_pad].x);
          if (top != -INFINITY)
#pragma unroll 4
            for (int s = 0; s < a.splits; ++s) {
              const float2 v = p[s * a.rows_pad];
              total += v.y * ex2(v.x - top);
            }
        }
        ms.stat[r] = total > 0.f ? make_float2(top, 1.f / total) : make_float2(0.f, 0.f);
        const int64_t end = (a.causal ? len - cl + ((int)r0 + r) / a.gq + 1 : len) - s0;
        ms.end[r] = r >= rows || end < 0 ? 0 : (end < a.span ? (int)end : (int)a.span);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if (issuer && grp < nb) {
      waits(kQFull, 0);
      waits(kKFull + grp, 0);
      tc_fence_after();
      if (elect_one() && !failed) scores(grp);
      __syncwarp();
    }
    // pass 0: the row on this lane
    int64_t end = 0;
    if (PASS == 0) {
      end = a.causal ? len - cl + ((int)r0 + lrow) / a.gq + 1 : len;
      if (end > s1) end = s1;
      // a row that is not there keeps its warp from masking by seeing whole steps
      if (lrow >= rows) end = s0 + (int64_t)nb * kStepTok;
    }
    const int64_t first_end = len - cl + (int)r0 / a.gq;  // last token that the first row sees
    const bool warp_on = PASS == 1 || (warp & 3) * 32 < rows;
    float ref = -INFINITY, sum = 0.f;
    int it = 0;
#pragma unroll 1
    for (int j = grp; j < nb; j += 2, ++it) {
      waits(kSFull + grp, it & 1);
      tc_fence_after();
      const int64_t at = s0 + (int64_t)j * kStepTok;
      if (PASS == 0) {
        if (warp_on) {
          const int64_t left = end - at;
          const int cnt = left < 0 ? 0 : (left < kStepTok ? (int)left : kStepTok);
          const bool whole = __all_sync(0xffffffffu, cnt == kStepTok);
          const float mx = whole ? row_max<false>(t_s, cnt) : row_max<true>(t_s, cnt);
          if (mx > ref) {
            sum *= ex2(ref - mx);
            ref = mx;
          }
          const float base = ref == -INFINITY ? 0.f : ref;
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          uint4* kept = a.kept ? reinterpret_cast<uint4*>(a.kept + ((int64_t)head * a.rows_kept + lrow) * a.kept_stride + at)
                               : nullptr;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            tc_ld32(t_s + 32 * c, r);
            tc_wait_ld();
            if (kept && lrow < rows)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                kept[8 * c + e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float p = ex2(__uint_as_float(r[e]) - base);
              part[e & 3] += whole || 32 * c + e < cnt ? p : 0.f;
            }
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
        }
      } else {
        // the token on this lane, over the rows in their order (four running sums)
        const int tok = j * kStepTok + lrow;  // of the stretch
        const bool all = !a.causal || at + kStepTok - 1 <= first_end;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < n_cols; c += 16) {
          uint32_t r[16];
          tc_ld16(t_s + c, r);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float4 st = *reinterpret_cast<const float4*>(&ms.stat[c + e]);
            float p0 = ex2(__uint_as_float(r[e]) - st.x), p1 = ex2(__uint_as_float(r[e + 1]) - st.z);
            if (!all) {
              const int2 en = *reinterpret_cast<const int2*>(&ms.end[c + e]);
              p0 = tok < en.x ? p0 : 0.f;
              p1 = tok < en.y ? p1 : 0.f;
            }
            part[e & 2] = fmaf(p0, st.y, part[e & 2]);
            part[(e & 2) + 1] = fmaf(p1, st.w, part[(e & 2) + 1]);
          }
        }
        const int64_t t = at + lrow;
        if (t < s1) {
          const float w = (part[0] + part[1]) + (part[2] + part[3]);
          out[t] = in ? in[t] + w : w;
        }
      }
      tc_fence_before();
      group_sync();
      if (issuer && j + 2 < nb) {
        waits(kKFull + (j & 1), ((j + 2) >> 1) & 1);
        tc_fence_after();
        if (elect_one() && !failed) scores(j + 2);
        __syncwarp();
      }
    }
    if (PASS == 0) {
      if (grp == 1) ms.stat[lrow] = make_float2(ref, sum);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (grp == 0 && lrow < rows) {
        const float2 o = ms.stat[lrow];
        const float top = fmaxf(ref, o.x), t = top == -INFINITY ? 0.f : top;
        ml[lrow] = make_float2(top, sum * ex2(ref - t) + o.y * ex2(o.x - t));
      }
    }
  } else {
    // ------------------------------------------------------ codes to operands
    const int dw = warp - kReadWarps, dtid = tid - 32 * kReadWarps;
    for (int i = dtid; i < (int)(sizeof(HeadMeta) / 4); i += 32 * kDqWarps)
      reinterpret_cast<uint32_t*>(&ms.m)[i] = reinterpret_cast<const uint32_t*>(a.meta + head)[i];
    load_dequant_tables<true>(sm + kOffTab, a.dec_image, dtid, 32 * kDqWarps);
    load_dequant_tables_lo(sm + kOffTab + kDqBytes, a.dec_image, dtid, 32 * kDqWarps);
    asm volatile("bar.sync 4, %0;" ::"n"(32 * kDqWarps) : "memory");
    const uint32_t tab = sb + kOffTab, norms = key_norm_offset(a.kb, a.vb);
    const KeyLane k0 = key_lane(ms.m, dw, lane, 16384, norms, tab), k1 = key_lane(ms.m, 15 - dw, lane, 16384, norms, tab);
    const int64_t t0 = s0 / kTile;
    const uint8_t* const base = a.packed + (a.sm.table ? (int64_t)h * a.sm.tile_bytes
                                                       : ((int64_t)head * a.sm.n_tiles + t0) * a.sm.tile_bytes);
    const int32_t* const pages = a.sm.table ? a.sm.table + (int64_t)b * a.sm.max_blocks + t0 : nullptr;
    const bool code0 = __any_sync(0xffffffffu, k0.w > 4), code1 = __any_sync(0xffffffffu, k1.w > 4);
    // a set of registers for each tile of a step: a tile's set is filled again as soon as it is
    // used, a whole step before it is due
    KeyRaw r0k[2], r1k[2];
    int page[2] = {0, 0};
    auto read_page = [&](int t) {
      if (pages && t < nt) page[t & 1] = __ldg(pages + t);
    };
    auto fetch = [&](int t, int i) {
      if (t < nt) {
        const uint8_t* p = base + (pages ? (int64_t)page[i] * a.sm.hkv : (int64_t)t) * a.sm.tile_bytes;
        if (code0) load_keys<5>(r0k[i], p, k0);
        else load_keys<2>(r0k[i], p, k0);
        if (code1) load_keys<5>(r1k[i], p, k1);
        else load_keys<2>(r1k[i], p, k1);
      }
    };
    read_page(0);
    read_page(1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fetch(i, i);
      read_page(2 + i);
    }
    if (!mbar_wait(bar(kQRot), 0)) failed = 1;  // the keys' buffers lie under the rotation image
    __syncwarp();
#pragma unroll 1
    for (int j = 0; j < nb && !failed; ++j) {
      if (j >= 2 && !mbar_wait(bar(kKEmpty + (j & 1)), ((j >> 1) & 1) ^ 1)) { failed = 1; break; }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * j + i;
        if (t >= nt) break;
        const uint32_t row = sb + kOffK + (j & 1) * 2 * kPart + i * 8192;
        if (code0) keys_by_code<true>(k0, r0k[i], tab, row, true, row + kPart + k0.col, 1024);
        else keys_by_pair_split(k0, r0k[i], row, kDqBytes, kPart);
        if (code1) keys_by_code<true>(k1, r1k[i], tab, row, true, row + kPart + k1.col, 1024);
        else keys_by_pair_split(k1, r1k[i], row, kDqBytes, kPart);
        fetch(t + 2, i);
        read_page(t + 4);
        if (t + kAheadW < nt && lane == 0 && (t & 7) == dw) {  // towards the L2 cache (the warps take turns)
          const uint8_t* p = base + (pages ? (int64_t)__ldg(pages + t + kAheadW) * a.sm.hkv
                                           : (int64_t)(t + kAheadW)) * a.sm.tile_bytes;
          bulk_prefetch(p, 1024u * a.kb);
          bulk_prefetch(p + norms, 1024u);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKFull + (j & 1)));
    }
  }
  if (failed) atomicOr(a.status, kStatusTimeout);
  if (__syncthreads_or(failed)) {  // nothing in flight may outlive the block (bounded waits)
    if (warp == 0 || warp == 4) {
      if (elect_one()) {
        tc_commit(bar(kDrain + (warp >> 2)));
        mbar_wait(bar(kDrain + (warp >> 2)), 0);
      }
    }
    if (tid == 0) mbar_wait(bar(kImg), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
}

// Kept scores: a thread takes one token and adds its weights over the rows, in order.
__global__ void __launch_bounds__(256) kept_kernel(const __grid_constant__ WeightArgs a) {
  __shared__ float2 stat[kKeepRows];
  __shared__ int64_t end[kKeepRows];
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv;
  const int64_t len = a.sm.len(b, a.T), cl = chunk_len(a.chunk_lens, a.n, b);
  const int rows = (int)(cl * a.gq), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_dependency();
  if ((int64_t)blockIdx.x * 256 >= len) return;
  for (int r = warp; r < rows; r += 8) {  // every row's softmax, from its stretches
    const float2* p = a.part_ml + (int64_t)head * a.splits * a.rows_pad + r;
    float top = -INFINITY, total = 0.f;
    for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, p[s * a.rows_pad].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top != -INFINITY)
      for (int s = lane; s < a.splits; s += 32) total += p[s * a.rows_pad].y * ex2(p[s * a.rows_pad].x - top);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
      stat[r] = total > 0.f ? make_float2(top, 1.f / total) : make_float2(0.f, 0.f);
      end[r] = a.causal ? len - cl + r / a.gq + 1 : len;
    }
  }
  __syncthreads();
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= len) return;
  const float* s = a.kept + (int64_t)head * a.rows_kept * a.kept_stride + t;
  float part[4] = {0.f, 0.f, 0.f, 0.f};
  // (a stretch that no row sees is not written: nothing is read where a row sees nothing)
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
    if (t < end[r]) part[r & 3] = fmaf(ex2(s[r * a.kept_stride] - stat[r].x), stat[r].y, part[r & 3]);
  const float w = (part[0] + part[1]) + (part[2] + part[3]);
  const int64_t o = b * a.ws[0] + h * a.ws[1] + t;
  a.w_out[o] = a.w_in ? a.w_in[o] + w : w;
}

// Several row tiles: their sums, in order.
__global__ void __launch_bounds__(256) add_kernel(const __grid_constant__ WeightArgs a) {
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= a.sm.len(b, a.T)) return;
  const int64_t n_rows = chunk_len(a.chunk_lens, a.n, b) * a.gq;
  const int tiles = (int)((n_rows + kRowsW - 1) / kRowsW);
  const int64_t o = b * a.ws[0] + h * a.ws[1] + t;
  float w = 0.f;
  for (int r = 0; r < tiles; ++r) w += a.part_w[((int64_t)r * a.n_heads + head) * a.T + t];
  a.w_out[o] = a.w_in ? a.w_in[o] + w : w;
}

struct CutW {
  int row_tiles, splits;
  int64_t span, rows_pad;
};
CutW cut_of(const gtq_plan* p, int64_t T, int64_t n) {
  CutW c;
  const int64_t rows = n * p->g_q;
  c.row_tiles = (int)((rows + kRowsW - 1) / kRowsW);
  c.rows_pad = (int64_t)c.row_tiles * kRowsW;
  // enough blocks to fill the SMs evenly; a block's set-up costs about as much as 4 steps
  const int64_t units = (int64_t)p->n_heads * c.row_tiles, steps = (T + kStepTok - 1) / kStepTok;
  double best = 1e300;
  int64_t best_per = steps;
  for (int64_t s = 1; s <= 256 && s <= steps; ++s) {
    const int64_t per = (steps + s - 1) / s, parts = (steps + per - 1) / per;
    const double cost = (double)((units * parts + p->n_sms - 1) / p->n_sms) * (per + 4.0);
    if (cost < best * 0.999) {
      best = cost;
      best_per = per;
    }
    if (units * s > 64 * (int64_t)p->n_sms) break;
  }
  c.span = best_per * kStepTok;
  c.splits = (int)((steps + best_per - 1) / best_per);
  return c;
}

size_t stat_bytes(const gtq_plan* p, const CutW& c) {
  return ((size_t)p->n_heads * c.splits * c.rows_pad * sizeof(float2) + 255) & ~(size_t)255;
}

// tokens of a row of kept scores: whole steps are written
int64_t kept_stride(const CutW& c) { return c.span * c.splits; }

}  // namespace

size_t weights_workspace(const gtq_plan* p, int64_t T, int64_t n) {
  const CutW c = cut_of(p, T, n);
  if (n * p->g_q <= kKeepRows) return stat_bytes(p, c) + (size_t)p->n_heads * n * p->g_q * kept_stride(c) * sizeof(float);
  return stat_bytes(p, c) + (c.row_tiles > 1 ? (size_t)c.row_tiles * p->n_heads * T * sizeof(float) : 0);
}

cudaError_t launch_weights(const gtq_plan* p, const uint8_t* packed, int64_t T, const SeqMap& sm,
                           const gtq_chunk& ch, const __half* q, const float* w_in, float* w_out,
                           const int64_t* ws, uint8_t* workspace, cudaStream_t s) {
  const CutW c = cut_of(p, T, ch.n_tokens);
  WeightArgs a = {};
  a.packed = packed;
  a.sm = sm;
  a.T = T;
  a.q = q;
  for (int i = 0; i < 3; ++i) a.qs[i] = ch.q_strides[i];
  a.n = ch.n_tokens;
  a.chunk_lens = ch.chunk_lens_dev;
  a.causal = ch.causal;
  a.gq = p->g_q;
  a.hkv = p->cfg.n_kv_heads;
  a.kb = p->cfg.k_bits;
  a.vb = p->cfg.v_bits;
  a.meta = p->d_meta;
  a.bimg_k = p->d_bimg;
  a.dec_image = p->tab.dec_image;
  a.w_in = w_in;
  a.w_out = w_out;
  a.ws[0] = ws[0];
  a.ws[1] = ws[1];
  a.row_tiles = c.row_tiles;
  a.splits = c.splits;
  a.n_heads = p->n_heads;
  a.span = c.span;
  a.rows_pad = c.rows_pad;
  a.part_ml = reinterpret_cast<float2*>(workspace);
  a.part_w = reinterpret_cast<float*>(workspace + stat_bytes(p, c));
  a.status = p->d_status;
  cudaError_t e = cudaFuncSetAttribute(weights_kernel<0>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemW);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(weights_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemW);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(c.row_tiles * c.splits), (unsigned)p->n_heads);
  if (ch.n_tokens * p->g_q <= kKeepRows) {
    a.kept = a.part_w;
    a.kept_stride = kept_stride(c);
    a.rows_kept = (int)(ch.n_tokens * p->g_q);
    weights_kernel<0><<<grid, kThreadsW, kSmemW, s>>>(a);
    return launch_overlapped(kept_kernel, dim3((unsigned)((T + 255) / 256), (unsigned)p->n_heads), 256, 0, s, a);
  }
  weights_kernel<0><<<grid, kThreadsW, kSmemW, s>>>(a);
  e = launch_overlapped(weights_kernel<1>, grid, kThreadsW, kSmemW, s, a);
  if (e != cudaSuccess) return e;
  if (c.row_tiles > 1)
    add_kernel<<<dim3((unsigned)((T + 255) / 256), (unsigned)p->n_heads), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace gtq
