// Eviction (include/gtq.h, gtq_evict): of every (sequence, KV head) the first
// and last tokens and those with the largest weights stay, and their codes move
// to another packed cache.  Two launches.
//
// select_kernel: one cluster of up to 16 blocks per head.  Each block holds its stretch
// of tokens in shared memory as order-preserving integers of their weights (HBM is
// read once; tokens beyond that memory are read again from L2).  The weight that the
// last chosen token has is found digit by digit (11, 11 and 10 bits): each block
// counts the digits of its stretch and adds up its share of the digits over the cluster
// (distributed shared memory), and every block finds the digit where the count from the
// top passes what is still wanted, in the one share that holds it (2 heads of 131072
// tokens, calls back to back: 46 us, and 50 where every block reads all counts; 51 to 53 a call on
// inputs that the L2 cache does not hold).  Then each thread counts 16 neighbouring tokens, one prefix sum
// gives it its place, and it writes the indices of those that stay: tokens above that
// weight, and as many with exactly that weight, lowest index first, as are missing.
// Bound by the latencies of its dozen block- and cluster-wide steps: 26 us for 64 heads of
// 16384 tokens (4 MB of weights), 31 us for 2 heads of 131072.
//
// move_kernel: one block per new tile and head.  The tiles that its 64 tokens
// come from arrive by bulk copy, a batch at a time; a thread owns portions of the
// new tile (all codes of 8 or 16 of its tokens in one slot or pair of dims), shifts
// them together in registers from reads of the old tiles, and adds them to the tile in
// shared memory, which leaves in full.  The bytes of the source tiles are its floor (HBM
// reads them in sectors that hold the codes of many tokens).  Bound by its instructions,
// which take codes apart and together, and by the waits of a block's stages (a quarter kept of
// 64 heads of 16384 tokens, K3V2: 58 us, three fifths of all issue slots, 105 MB of source tiles).
#include <cooperative_groups.h>

#include <algorithm>

#include "gtq_internal.h"

namespace cg = cooperative_groups;

namespace gtq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelCluster = 16;      // blocks per head at most
constexpr int kSelTokens = 4096;     // tokens that are worth a block of their own
constexpr int kPer = 16;             // neighbouring tokens of a thread
constexpr int kHeld = 32768;         // tokens of a block that stay in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMaxBatch = 12;        // source tiles in shared memory at once, at most
// Dynamic shared memory of a block, at most.  The kernels' limits are set to these and never to a
// call's own size: a limit belongs to the process, and another thread's call would launch against it.
constexpr size_t kMaxSelSmem = (kHeld + kHeld / kPer + 1) * sizeof(uint32_t) + kSelThreads * kPer * sizeof(uint16_t);
constexpr size_t kMaxMoveSmem = 110 * 1024;  // two blocks fit on an SM

struct EvictArgs {
  const float* w;
  int64_t ws[2];
  float* w_out;
  int64_t wos[2];
  int32_t* kept;        // [heads][kept_stride]
  int64_t kept_stride;
  int64_t fill;         // entries of kept that are written (behind the last: -1)
  int32_t* new_lens;
  int64_t T, keep, first, recent;
  int hkv;
  SeqMap src, dst;
  const uint8_t* src_packed;
  uint8_t* dst_packed;
  const HeadMeta* meta;
  int kb, vb;
  int held;   // select: tokens in shared memory
  int batch;  // move: source tiles in shared memory
};

// Larger weight, larger integer; -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of one int per thread over the block; `total` for all.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  const int before = warp ? warp_sums[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

// What lies behind the held keys in dynamic shared memory.
__device__ __forceinline__ uint32_t* list_space(uint32_t* keys, int held) { return keys + held + held / 16 + 1; }

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t keys[];  // token i of the stretch at i + i / 16: a thread's 16 neighbours
                                      // then lie in as many banks as its warp's need
  __shared__ __align__(16) int hist[kSelBins];
  __shared__ __align__(16) int slice[2][kSelBins];  // this block's share of the digits, counted over all blocks
  __shared__ int slice_sum[2];
  __shared__ int warp_sums[32];
  __shared__ int found[2];   // digit, and the count above it
  __shared__ int counts[2];  // this block's tokens that are sure to stay, and those at the weight
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t len = a.src.len(b, a.T);
  const int64_t n_keep = len < a.keep ? len : a.keep;
  const int64_t first = a.first < len ? a.first : len;
  const int64_t last = len - a.recent > first ? len - a.recent : first;  // [first, last) compete
  int want = (int)(n_keep - (first + len - last));
  const float* w = a.w + b * a.ws[0] + h * a.ws[1];
  // this block's stretch, a multiple of the threads' neighbours
  const int64_t part = (len + blocks - 1) / blocks;
  const int64_t per = (part + kPer - 1) / kPer * kPer;
  const int64_t t0 = per * rank < len ? per * rank : len;
  const int n = (int)((t0 + per < len ? t0 + per : len) - t0);
  const int c0 = (int)(first - t0 < 0 ? 0 : (first - t0 < n ? first - t0 : n));
  const int c1 = (int)(last - t0 < 0 ? 0 : (last - t0 < n ? last - t0 : n));  // [c0, c1) compete
  w += t0;
  const bool all = n_keep == len;  // nothing is left out (uniform over the cluster)
  const int held = n < a.held ? n : a.held;
  auto key_at = [&](int i) { return i < held ? keys[i + (i >> 4)] : order_key(w[i]); };
  uint32_t prefix = 0;
  if (!all) {
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = slice[0][i] = 0;
    if (tid == 0) slice_sum[0] = 0;
#pragma unroll 4
    for (int i = tid; i < held; i += kSelThreads) keys[i + (i >> 4)] = order_key(w[i]);
    __syncthreads();
    int shift = 32;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      const uint32_t above = pass == 0 ? 0u : ~0u << shift;
      shift -= bits;
      // equal digits are common: a weight of 0 is counted apart, and a thread's run of one
      // digit is added at once
      const int zero_bin = ((0x80000000u & above) == prefix) ? (int)((0x80000000u >> shift) & ((1u << bits) - 1)) : -1;
      int zeros = 0, run = -1, run_n = 0;
#pragma unroll 4
      for (int i = c0 + tid; i < c1; i += kSelThreads) {
        const uint32_t k = key_at(i);
        const int bin = (int)((k >> shift) & ((1u << bits) - 1));
        if (k == 0x80000000u) {
          zeros += zero_bin >= 0;
        } else if ((k & above) == prefix) {
          if (bin != run) {
            if (run_n) atomicAdd(&hist[run], run_n);
            run = bin;
            run_n = 0;
          }
          ++run_n;
        }
      }
      if (run_n) atomicAdd(&hist[run], run_n);
      zeros = __reduce_add_sync(0xffffffffu, zeros);
      if (lane == 0 && zeros) atomicAdd(&hist[zero_bin], zeros);
      cluster.sync();
      // every block adds up its share of the digits, ...
      const int n_bins = 1 << bits, share = n_bins / blocks, quads = share / 4;
      int* const sums = slice[pass & 1];
      int sum = 0;
      static_assert(kSelBins / 4 <= kSelThreads, "one quad of digits a thread");
      if (tid < n_bins / 4) {
        const int r = tid / quads, at = 4 * (tid - r * quads);
        const int4 v = *reinterpret_cast<const int4*>(cluster.map_shared_rank(hist, r) + rank * share + at);
        if (v.x) atomicAdd(&sums[at], v.x);
        if (v.y) atomicAdd(&sums[at + 1], v.y);
        if (v.z) atomicAdd(&sums[at + 2], v.z);
        if (v.w) atomicAdd(&sums[at + 3], v.w);
        sum = v.x + v.y + v.z + v.w;
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0 && sum) atomicAdd(&slice_sum[pass & 1], sum);
      cluster.sync();
      // ... and reads the share in which the count from the top (lane 0) passes `want`
      int in_share = lane < blocks ? *cluster.map_shared_rank(&slice_sum[pass & 1], blocks - 1 - lane) : 0;
      int upto = in_share;
#pragma unroll
      for (int o = 1; o < kSelCluster; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned passes = __ballot_sync(0xffffffffu, upto - in_share < want && upto >= want);
      const int top = passes ? __ffs(passes) - 1 : 0, f = blocks - 1 - top;
      const int above_share = __shfl_sync(0xffffffffu, upto - in_share, top);
      const int d0 = share - 4 - 4 * tid;
      int c[4] = {0, 0, 0, 0};
      if (d0 >= 0) {
        const int4 v = *reinterpret_cast<const int4*>(cluster.map_shared_rank(sums, f) + d0);
        c[0] = v.w;
        c[1] = v.z;
        c[2] = v.y;
        c[3] = v.x;
      }
      int total;
      int over = above_share + block_scan(c[0] + c[1] + c[2] + c[3], warp_sums, total);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (over < want && over + c[e] >= want) {
          found[0] = f * share + d0 + 3 - e;
          found[1] = over;
        }
        over += c[e];
      }
      // (counts are read by others before the exchange's second barrier, shares after it: the other
      // share's last readers have passed the next digit's first barrier)
      for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = slice[(pass + 1) & 1][i] = 0;
      if (tid == 0) slice_sum[(pass + 1) & 1] = 0;
      __syncthreads();
      if (want > 0) {
        prefix |= (uint32_t)found[0] << shift;
        want -= found[1];
      } else {  // only the first and last tokens stay: nothing is above the largest integer
        prefix = ~0u;
      }
    }
  }
  // want: how many of the tokens whose integer is `prefix` stay
  auto klass = [&](int i) {  // 2 stays, 1 at the weight, 0 goes
    if (all || i < c0 || i >= c1) return 2;
    const uint32_t k = key_at(i);
    return k > prefix ? 2 : (k == prefix && want > 0 ? 1 : 0);
  };
  // a thread's 16 neighbours as bits: sure to stay, at the weight
  auto classes = [&](int base, uint32_t& stay, uint32_t& at_weight) {
    stay = at_weight = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int c = base + k < n ? klass(base + k) : 0;
      stay |= (uint32_t)(c == 2) << k;
      at_weight |= (uint32_t)(c == 1) << k;
    }
  };
  uint32_t stay = 0, at_weight = 0;
  int sure = 0, equal = 0;
  for (int base = tid * kPer; base < n; base += kSelThreads * kPer) {
    classes(base, stay, at_weight);
    sure += __popc(stay);
    equal += __popc(at_weight);
  }
  if (tid < 2) counts[tid] = 0;
  __syncthreads();
  {
    int s = sure, q = equal;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if (lane == 0) {
      atomicAdd(&counts[0], s);
      atomicAdd(&counts[1], q);
    }
  }
  cluster.sync();
  int64_t out = 0, eq = 0;  // tokens that stay, and tokens at the weight, before this block's
  for (int r = 0; r < rank; ++r) {
    const int* other = cluster.map_shared_rank(counts, r);
    out += other[0];
    eq += other[1];
  }
  out += eq < want ? eq : want;
  cluster.sync();  // nothing of another block is read past this point
  int32_t* kept = a.kept + (int64_t)head * a.kept_stride;
  float* wo = a.w_out ? a.w_out + b * a.wos[0] + h * a.wos[1] : nullptr;
  uint16_t* list = reinterpret_cast<uint16_t*>(list_space(keys, a.held));  // a turn's kept tokens, in order
  for (int start = 0; start < n; start += kSelThreads * kPer) {
    const int base = start + tid * kPer;
    if (n > kSelThreads * kPer) {  // its classes, where one turn does not take all
      classes(base, stay, at_weight);
      sure = __popc(stay);
      equal = __popc(at_weight);
    }
    int n_sure, n_equal;
    const int sure_before = block_scan(sure, warp_sums, n_sure);
    const int equal_before = block_scan(equal, warp_sums, n_equal);
    // of the tokens at the weight, the first `want` of the head stay
    const int64_t room = want - eq > 0 ? want - eq : 0;
    int left = (int)(room > equal_before ? room - equal_before : 0);
    int at = sure_before + (int)(equal_before < room ? equal_before : room);
    uint32_t both = stay | at_weight;
    while (both) {
      const int k = __ffs(both) - 1;
      both &= both - 1;
      const bool tie = (at_weight >> k) & 1u;
      if (!tie || left > 0) list[at++] = (uint16_t)(tid * kPer + k);
      left -= tie;
    }
    __syncthreads();
    const int total = n_sure + (int)(n_equal < room ? n_equal : room);
    for (int r = tid; r < total; r += kSelThreads) {
      const int i = start + list[r];
      kept[out + r] = (int32_t)(t0 + i);
      if (wo) wo[out + r] = w[i];
    }
    __syncthreads();
    out += total;
    eq += n_equal;
  }
  for (int64_t i = n_keep + (int64_t)rank * kSelThreads + tid; i < a.fill; i += (int64_t)blocks * kSelThreads)
    kept[i] = -1;
  if (h == 0 && rank == 0 && tid == 0) a.new_lens[b] = (int32_t)n_keep;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// At least n <= 32 bits from bit `at` of a word array; the second word is read only where the bits
// reach into it.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* x, int at, int n) {
  const uint32_t* p = x + (at >> 5);
  uint32_t next = 0;
  if ((at & 31) + n > 32) next = p[1];
  return __funnelshift_r(p[0], next, at);
}

// Where a token's codes lie in a batch of source tiles, in bits of shared memory.
struct From {
  int tile;   // its tile, or -1: not in this batch
  int entry;  // its place among a row of 64: (t % 8) * 8 + t / 8, key pairs and norms
  int value;  // its codes of dim 0
};

// The pairs of codes of 8 tokens (g + 8 u) in two slots, shifted together from the last to the first.
// Bit j of `here`: token j of the new tile comes from this batch.
template <int WORDS>
__device__ __forceinline__ void gather_keys(const uint32_t* x, const From* from, uint64_t here, int g, const int (&w2)[2],
                                            const int (&area)[2], uint32_t (&acc)[2][4]) {
#pragma unroll
  for (int u = 7; u >= 0; --u) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int r = WORDS - 1; r > 0; --r) acc[k][r] = __funnelshift_l(acc[k][r - 1], acc[k][r], w2[k]);
      acc[k][0] <<= w2[k];
    }
    if (!((here >> (8 * u)) & 255)) continue;
    const int tile = from[g + 8 * u].tile, entry = from[g + 8 * u].entry;
    if (tile < 0) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      acc[k][0] |= bits_at(x, tile + area[k] + w2[k] * entry, w2[k]) & ((1u << w2[k]) - 1);
  }
}

// The codes of 16 tokens in two dims: for every (a, b) those of tokens 16 a + 8 b + 2 c + l, as
// (dim, l) = (0, 0), (0, 1), (1, 0), (1, 1).  A token's two codes lie 2 vb bits apart in the old tile
// as they do in the new one.
template <int WORDS>
__device__ __forceinline__ void gather_values(const uint32_t* x, const From* from, uint64_t here, int c, int vb, int area,
                                              uint32_t (&acc)[8]) {
  const uint32_t code = (1u << vb) - 1, both = code | code << (2 * vb);
#pragma unroll
  for (int ab = 7; ab >= 0; --ab) {
#pragma unroll
    for (int r = WORDS - 1; r > 0; --r) acc[r] = __funnelshift_lc(acc[r - 1], acc[r], 4 * vb);
    acc[0] = __funnelshift_lc(0u, acc[0], 4 * vb);  // (a whole word at vb = 8)
    if (!((here >> (8 * ab)) & 255)) continue;
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      const int at = from[8 * ab + 2 * c + l].value;
      if (at >= 0) acc[0] |= (bits_at(x, at + area, 3 * vb) & both) << (l * vb);
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictArgs a, int* status) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ HeadMeta m;
  __shared__ int src_tile[kTile];     // distinct source tiles, in order
  __shared__ uint16_t tok[kTile];     // token: place of its tile in that list << 8 | its index there
  __shared__ From from[kTile];
  __shared__ __align__(8) uint32_t in_batch[2];
  __shared__ int n_src;
  __shared__ __align__(8) uint64_t bar;
  const int head = blockIdx.y, b = head / a.hkv;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t len = a.src.len(b, a.T);
  const int64_t n_keep = len < a.keep ? len : a.keep;
  const int64_t tile = blockIdx.x;
  if (tile * kTile >= n_keep) return;
  const int n_tok = (int)(n_keep - tile * kTile < kTile ? n_keep - tile * kTile : kTile);
  const int tb = (int)a.src.tile_bytes;
  uint32_t* out = reinterpret_cast<uint32_t*>(sm);
  const uint32_t stage = (uint32_t)tb + 16;  // a word behind each tile may be read
  if (tid < 32) {  // which tiles the tokens come from: they are in order
    const int32_t* kept = a.kept + (int64_t)head * a.kept_stride + tile * kTile;
    int before = 0;
    int prev_last = -1;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = 32 * half + lane;
      const int s = i < n_tok ? kept[i] : -1;
      const int st = s >> 6;
      int up = __shfl_up_sync(0xffffffffu, st, 1);
      if (lane == 0) up = prev_last;
      const bool fresh = s >= 0 && st != up;
      const unsigned f = __ballot_sync(0xffffffffu, fresh);
      const int at = before + __popc(f & ((2u << lane) - 1)) - 1;
      tok[i] = s >= 0 ? (uint16_t)(at << 8 | (s & 63)) : (uint16_t)0xffff;  // behind the last: in no batch
      if (fresh) src_tile[at] = st;
      before += __popc(f);
      prev_last = __shfl_sync(0xffffffffu, st, 31);
    }
    if (lane == 0) {
      n_src = before;
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&bar)));
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  }
  for (int i = tid; i < tb / 16; i += kMoveThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < (int)(sizeof(HeadMeta) / 4); i += kMoveThreads)
    reinterpret_cast<uint32_t*>(&m)[i] = reinterpret_cast<const uint32_t*>(a.meta + head)[i];
  __syncthreads();
  const int kb = a.kb, vb = a.vb;
  bool ok = true;
  for (int s0 = 0, round = 0; s0 < n_src && ok; s0 += a.batch, ++round) {
    const int n = min(a.batch, n_src - s0);
    if (tid == 0) {
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(&bar)),
                   "r"((uint32_t)(n * tb)) : "memory");
      for (int i = 0; i < n; ++i)
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_addr(sm + tb + i * stage)),
            "l"(a.src.tile(const_cast<uint8_t*>(a.src_packed), head, src_tile[s0 + i])), "r"((uint32_t)tb),
            "r"(smem_addr(&bar))
            : "memory");
    }
    if (tid < kTile) {
      const int j = tid, v = tok[j], i = (v >> 8) - s0, js = v & 63;
      const bool in = (unsigned)i < (unsigned)n;
      const int at = 8 * (tb + i * (int)stage);
      const unsigned any = __ballot_sync(0xffffffffu, in);
      if (lane == 0) in_batch[tid >> 5] = any;
      from[j].tile = in ? at : -1;
      from[j].entry = (js & 7) * 8 + (js >> 3);
      // portion (i8, g, c) holds dims 16 i8 + g and + 8 of 16 tokens
      from[j].value = in ? at + 8192 * kb + vb * (((js & 7) >> 1) * 32 + 4 * (js >> 3) + (js & 1)) : -1;
    }
    {  // bounded wait: after 2 s the call has failed, after 2 s more its copies are given up
      uint64_t began = 0;
      for (unsigned i = 0;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done) : "r"(smem_addr(&bar)), "r"(round & 1), "r"(1000000u) : "memory");
        if (done) break;
        uint64_t now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (!began) began = now;
        else if (now - began > 4000000000ull) break;
        else if (now - began > 2000000000ull) ok = false;
      }
    }
    if (__syncthreads_or(!ok)) { ok = false; break; }
    // keys: portion g of slot s holds the pairs of tokens g + 8 u, 2 w bits each; a thread's two
    // slots share the tokens
    const uint32_t* const words = reinterpret_cast<const uint32_t*>(sm);
    const uint64_t here = *reinterpret_cast<const uint64_t*>(in_batch);
    {
      const int g = tid & 7;
      int w2[2], area[2];
      uint32_t acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int slot = (tid >> 3) + 32 * k;
        w2[k] = 2 * m.slot_width[slot];
        area[k] = 8 * m.slot_koff[slot];
      }
      if (__any_sync(0xffffffffu, max(w2[0], w2[1]) > 8)) gather_keys<4>(words, from, here, g, w2, area, acc);
      else gather_keys<2>(words, from, here, g, w2, area, acc);
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // 16 w bits at a multiple of 16 bits
        const int w = w2[k] >> 1;
        uint16_t* o = reinterpret_cast<uint16_t*>(sm) + (area[k] >> 4) + g * w;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < w) o[i] |= (uint16_t)(acc[k][i >> 1] >> (16 * (i & 1)));
      }
    }
    if (vb) {
      static_assert(kMoveThreads == 256, "one portion of values a thread");
      const int area = (tid >> 2) * 128 * vb;
      uint32_t acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (vb <= 2) gather_values<2>(words, from, here, tid & 3, vb, area, acc);
      else if (vb <= 4) gather_values<4>(words, from, here, tid & 3, vb, area, acc);
      else gather_values<8>(words, from, here, tid & 3, vb, area, acc);
      uint32_t* o = out + 256 * kb + tid * vb;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < vb) o[r] |= acc[r];
    }
    // norms: row of 64 fp16, token j at (j & 7) * 8 + (j >> 3); the value norms, then the groups'
    const int n_rows = (vb ? 1 : 0) + m.n_groups;
    for (int i = tid; i < n_rows * kTile; i += kMoveThreads) {
      const int row = i >> 6, at = i & 63, j = (at & 7) * 8 + (at >> 3);  // entry `at` is of token j
      const int tile = from[j].tile;
      if (tile < 0) continue;
      const int o = 512 * (kb + vb) + row * 64;
      reinterpret_cast<uint16_t*>(sm)[o + at] = reinterpret_cast<const uint16_t*>(sm)[(tile >> 4) + o + from[j].entry];
    }
    __syncthreads();  // the batch is read before the next one lands on it
  }
  if (!ok) {
    if (tid == 0) atomicOr(status, kStatusTimeout);
    return;
  }
  uint4* dst = reinterpret_cast<uint4*>(a.dst.tile(a.dst_packed, head, tile));
  for (int i = tid; i < tb / 16; i += kMoveThreads) dst[i] = reinterpret_cast<const uint4*>(sm)[i];
}

}  // namespace

cudaError_t launch_evict(const gtq_plan* p, const uint8_t* src, int64_t T, const SeqMap& sm,
                         const gtq_eviction& ev, uint8_t* dst, const SeqMap& dm, int32_t* ws_kept,
                         cudaStream_t s) {
  EvictArgs a;
  a.w = ev.weights_dev;
  a.w_out = ev.weights_out_dev;
  for (int i = 0; i < 2; ++i) {
    a.ws[i] = ev.w_strides[i];
    a.wos[i] = ev.w_out_strides[i];
  }
  a.kept = ev.kept_dev ? ev.kept_dev : ws_kept;
  a.kept_stride = ev.kept_dev ? ev.keep : T;
  a.fill = ev.kept_dev ? ev.keep : 0;
  a.new_lens = ev.new_lens_dev;
  a.T = T;
  a.keep = ev.keep;
  a.first = ev.n_first;
  a.recent = ev.n_recent;
  a.hkv = p->cfg.n_kv_heads;
  a.src = sm;
  a.dst = dm;
  a.src_packed = src;
  a.dst_packed = dst;
  a.meta = p->d_meta;
  a.kb = p->cfg.k_bits;
  a.vb = p->cfg.v_bits;
  // Blocks for a head: while its tokens are worth them, and no more than one wave of SMs (64 heads
  // of 16384 tokens: 43 us with 4 blocks, 26 with 2; of 32768: 121 with 8, 31 with 2).
  int blocks = 1;
  while (blocks < 8 && T > (int64_t)blocks * kSelTokens && 2 * blocks * p->n_heads <= p->n_sms) blocks *= 2;
  // Clusters of 16 have to find 16 SMs close together, and wait longer for one another: for long
  // sequences of few heads (4 heads of 262144 tokens: 93 us, 109 with 8 blocks; of 70000: 45 and 43;
  // 8 heads of 262144: 177 and 158).
  if (blocks == 8 && T > 8 * 4 * (int64_t)kSelTokens && 2 * kSelCluster * p->n_heads <= p->n_sms) blocks = kSelCluster;
  const int64_t stretch = (T + blocks - 1) / blocks + kPer;
  a.held = (int)std::min<int64_t>(stretch, kHeld);
  const size_t sel_smem = (size_t)(a.held + a.held / 16 + 1) * sizeof(uint32_t) +
                          std::min<int64_t>(stretch, kSelThreads * kPer) * sizeof(uint16_t);
  cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSelSmem);
  if (e == cudaSuccess)  // clusters above 8 blocks
    e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = sel_smem;
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)p->n_heads);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select_kernel, a);
  if (e != cudaSuccess) return e;
  const int64_t most = std::min(ev.keep, T);
  // source tiles of a new tile: about T / keep and two cut ones.  More at once cost blocks on an SM
  // (64 heads, a quarter kept: 84 us for the call, 97 with two tiles more); two blocks fit in any case
  const int64_t span = (T + most - 1) / most + 2;
  const int64_t room = (int64_t)kMaxMoveSmem / (int64_t)(p->tile_bytes + 16) - 1;
  a.batch = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(span, kMaxBatch), room));
  const size_t smem = p->tile_bytes + a.batch * (p->tile_bytes + 16);
  e = cudaFuncSetAttribute(move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxMoveSmem);
  if (e != cudaSuccess) return e;
  move_kernel<<<dim3((unsigned)((most + kTile - 1) / kTile), (unsigned)p->n_heads), kMoveThreads, smem, s>>>(
      a, p->d_status);
  return cudaGetLastError();
}

}  // namespace gtq
