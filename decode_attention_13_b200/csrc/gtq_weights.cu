// Attention weights that a chunk gives every cached token (include/gtq.h,
// gtq_attn_weights).
#include <algorithm>

#include "gtq_internal.h"
#include "gtq_unpack.cuh"

namespace gtq {
namespace {

constexpr int kRows = 16;       // rows of a block
constexpr int kThreadsC = 256;
constexpr float kScale = 0.08838834764831845f;  // 1 / sqrt(128)

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
  int causal;
  int gq, hkv, kb, vb;
  const HeadMeta* meta;
  const float* mrow;
  const float* rv;
  const uint8_t* singles;  // centroids as fp16 hi | lo (kTabSS of the decode image)
  const float* w_in;
  float* w_out;
  int64_t ws[2];
  float2* stats;           // [heads][rows]: maximum and sum of a row's softmax
};

struct Shared {
  HeadMeta m;
  float cb[kLutEntries + 2];
  float q[kRows][kD];
  float k[kTile][kD + 1];
  float v[kTile][kD];
  float s[kRows][kTile + 1];
  float o[kRows][kD];
  float mx[kRows], sum[kRows], fac[kRows];
};

__device__ int64_t chunk_len(const ChunkArgs& a, int b) {
  if (!a.chunk_lens) return a.n;
  const int64_t c = a.chunk_lens[b];
  return c < 0 ? 0 : (c < a.n ? c : a.n);
}

__device__ void load_head(const ChunkArgs& a, int head, Shared& sh) {
  for (int i = threadIdx.x; i < (int)(sizeof(HeadMeta) / 4); i += kThreadsC)
    reinterpret_cast<uint32_t*>(&sh.m)[i] = reinterpret_cast<const uint32_t*>(a.meta + head)[i];
  for (int w = 1; w <= 8; ++w)
    for (int i = threadIdx.x; i < (1 << w); i += kThreadsC) {
      const __half2 e = *reinterpret_cast<const __half2*>(a.singles + kSingleOff(w) + 4 * i);
      sh.cb[lut_base(w) + i] = __half2float(__low2half(e)) + __half2float(__high2half(e));
    }
  __syncthreads();
}

// rows [r0, r0 + kRows) of the head's queries in the keys' rotated bases
__device__ void load_q(const ChunkArgs& a, int b, int h, int head, int64_t r0, int64_t n_rows, Shared& sh) {
  for (int i = threadIdx.x; i < kRows * kD; i += kThreadsC) {
    const int r = i / kD, pos = i % kD;
    const int64_t row = r0 + r;
    float x = 0.f;
    if (row < n_rows) {
      const int64_t tok = row / a.gq;
      const __half* q = a.q + b * a.qs[0] + (h * a.gq + row % a.gq) * a.qs[1] + tok * a.qs[2];
      const float* mr = a.mrow + ((size_t)head * kD + pos) * kD;
      for (int d = 0; d < kD; ++d) x = fmaf(mr[d], __half2float(q[d]), x);
    }
    sh.q[r][pos] = x * kScale;
  }
  __syncthreads();
}

__device__ void load_tile(const ChunkArgs& a, int head, int64_t t, Shared& sh, bool values) {
  const uint8_t* tile = a.sm.tile(const_cast<uint8_t*>(a.packed), head, t);
  const int kn = key_norm_offset(a.kb, a.vb);
  for (int i = threadIdx.x; i < kTile * kD; i += kThreadsC) {
    const int j = i / kD, p = i % kD;
    float k = 0.f;
    const int w = (p >> 1) < sh.m.n_slots ? sh.m.slot_width[p >> 1] : 0;
    if (w) {
      const int g = sh.m.slot_group[p >> 1];
      k = sh.cb[lut_base(w) + key_code(tile, sh.m, j, p, w)] * tile_norm(tile, kn + 128 * g, j) *
          sh.m.inv_sqrt_m[g];
    }
    sh.k[j][p] = k;
    if (values)
      sh.v[j][p] = sh.cb[lut_base(a.vb) + value_code(tile, a.kb, a.vb, j, p)] *
                   tile_norm(tile, value_norm_offset(a.kb, a.vb), j) * kScale;
  }
  __syncthreads();
}

// scores of the rows on the tile in sh.k; -inf where a row sees nothing
__device__ void score_tile(const ChunkArgs& a, int64_t t, int64_t r0, int64_t n_rows, int64_t len,
                           int64_t cl, Shared& sh) {
  for (int i = threadIdx.x; i < kRows * kTile; i += kThreadsC) {
    const int r = i / kTile, j = i % kTile;
    float s = 0.f;
    for (int p = 0; p < kD; ++p) s = fmaf(sh.q[r][p], sh.k[j][p], s);
    const int64_t tok = t * kTile + j;
    const int64_t last = a.causal ? len - cl + (r0 + r) / a.gq : len - 1;
    sh.s[r][j] = r0 + r < n_rows && tok < len && tok <= last ? s : -INFINITY;
  }
  __syncthreads();
}

template <bool WEIGHTS>
__global__ void __launch_bounds__(kThreadsC) chunk_kernel(ChunkArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv, tid = threadIdx.x;
  const int64_t len = a.sm.len(b, a.T), cl = chunk_len(a, b), n_rows = cl * a.gq;
  const int64_t r0 = (int64_t)blockIdx.x * kRows;
  if (r0 >= n_rows) return;
  load_head(a, head, sh);
  load_q(a, b, h, head, r0, n_rows, sh);
  for (int i = tid; i < kRows * kD; i += kThreadsC) sh.o[i / kD][i % kD] = 0.f;
  if (tid < kRows) {
    sh.mx[tid] = -INFINITY;
    sh.sum[tid] = 0.f;
  }
  for (int64_t t = 0; t * kTile < len; ++t) {
    load_tile(a, head, t, sh, !WEIGHTS);
    score_tile(a, t, r0, n_rows, len, cl, sh);
    if (tid < kRows) {
      float mx = sh.mx[tid];
      for (int j = 0; j < kTile; ++j) mx = fmaxf(mx, sh.s[tid][j]);
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float fac = expf(sh.mx[tid] - ref);
      float sum = 0.f;  // a tile's own first: a long row's sum loses less that way
      for (int j = 0; j < kTile; ++j) {
        const float p = expf(sh.s[tid][j] - ref);
        sh.s[tid][j] = p;
        sum += p;
      }
      sh.mx[tid] = mx;
      sh.sum[tid] = sh.sum[tid] * fac + sum;
      sh.fac[tid] = fac;
    }
    __syncthreads();
    if (!WEIGHTS)
      for (int i = tid; i < kRows * kD; i += kThreadsC) {
        const int r = i / kD, d = i % kD;
        float o = sh.o[r][d] * sh.fac[r];
        for (int j = 0; j < kTile; ++j) o = fmaf(sh.s[r][j], sh.v[j][d], o);
        sh.o[r][d] = o;
      }
    __syncthreads();
  }
  __syncthreads();
  if (WEIGHTS) {
    if (tid < kRows && r0 + tid < n_rows)
      a.stats[(size_t)head * a.n * a.gq + r0 + tid] = make_float2(sh.mx[tid], sh.sum[tid]);
    return;
  }
  for (int i = tid; i < kRows * kD; i += kThreadsC) {
    const int r = i / kD, d = i % kD;
    const int64_t row = r0 + r;
    if (row >= n_rows) continue;
    float o = 0.f;
    for (int p = 0; p < kD; ++p) o = fmaf(sh.o[r][p], a.rv[p * kD + d], o);
    o = sh.sum[r] > 0.f ? o / sh.sum[r] : 0.f;
    a.out[b * a.os[0] + (h * a.gq + row % a.gq) * a.os[1] + row / a.gq * a.os[2] + d] = __float2half_rn(o);
  }
}

__global__ void __launch_bounds__(kThreadsC) weights_kernel(ChunkArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int head = blockIdx.y, b = head / a.hkv, h = head % a.hkv, tid = threadIdx.x;
  const int64_t len = a.sm.len(b, a.T), cl = chunk_len(a, b), n_rows = cl * a.gq;
  const int64_t t = blockIdx.x;
  if (t * kTile >= len) return;
  load_head(a, head, sh);
  load_tile(a, head, t, sh, false);
  float w = 0.f;
  for (int64_t r0 = 0; r0 < n_rows; r0 += kRows) {
    __syncthreads();
    load_q(a, b, h, head, r0, n_rows, sh);
    score_tile(a, t, r0, n_rows, len, cl, sh);
    if (tid < kTile)
      for (int r = 0; r < kRows && r0 + r < n_rows; ++r) {
        const float2 st = a.stats[(size_t)head * a.n * a.gq + r0 + r];
        if (st.y > 0.f) w += expf(sh.s[r][tid] - st.x) / st.y;
      }
  }
  const int64_t tok = t * kTile + tid;
  if (tid < kTile && tok < len) {
    const int64_t o = b * a.ws[0] + h * a.ws[1] + tok;
    a.w_out[o] = (a.w_in ? a.w_in[o] : 0.f) + w;
  }
}

ChunkArgs chunk_args(const gtq_plan* p, const uint8_t* packed, int64_t T, const SeqMap& sm,
                     const gtq_chunk& c, const __half* q) {
  ChunkArgs a = {};
  a.packed = packed;
  a.sm = sm;
  a.T = T;
  a.q = q;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = c.q_strides[i];
    a.os[i] = c.out_strides[i];
  }
  a.n = c.n_tokens;
  a.chunk_lens = c.chunk_lens_dev;
  a.causal = c.causal;
  a.gq = p->g_q;
  a.hkv = p->cfg.n_kv_heads;
  a.kb = p->cfg.k_bits;
  a.vb = p->cfg.v_bits;
  a.meta = p->d_meta;
  a.mrow = p->d_mrow;
  a.rv = p->tab.rot_v;
  a.singles = reinterpret_cast<const uint8_t*>(p->tab.dec_image) + kTabSS;
  return a;
}

}  // namespace

size_t weights_workspace(const gtq_plan* p, int64_t, int64_t n) {
  return (size_t)p->n_heads * n * p->g_q * sizeof(float2);
}

cudaError_t launch_weights(const gtq_plan* p, const uint8_t* packed, int64_t T, const SeqMap& sm,
                           const gtq_chunk& c, const __half* q, const float* w_in, float* w_out,
                           const int64_t* ws, uint8_t* workspace, cudaStream_t s) {
  ChunkArgs a = chunk_args(p, packed, T, sm, c, q);
  a.w_in = w_in;
  a.w_out = w_out;
  a.ws[0] = ws[0];
  a.ws[1] = ws[1];
  a.stats = reinterpret_cast<float2*>(workspace);
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(Shared));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  if (e != cudaSuccess) return e;
  const int64_t rows = c.n_tokens * p->g_q;
  chunk_kernel<true><<<dim3((unsigned)((rows + kRows - 1) / kRows), (unsigned)p->n_heads), kThreadsC,
                       sizeof(Shared), s>>>(a);
  weights_kernel<<<dim3((unsigned)((T + kTile - 1) / kTile), (unsigned)p->n_heads), kThreadsC,
                   sizeof(Shared), s>>>(a);
  return cudaGetLastError();
}

}  // namespace gtq
