// Rotary positions of queries and keys (include/gtq.h, gtq_rope): pair i of a
// row at position p turns by a = p f_i,
//     y0 = m (x0 cos a - x1 sin a),   y1 = m (x1 cos a + x0 sin a).
//
// The floor is memory: every element is read once and written once.  A block
// takes kTok positions of one sequence and all heads of q and k, so an angle's
// sine and cosine are formed once per (position, pair) and used by every head.
//   * Angles in turns: u = p (f_i / 2 pi) in fp64, reduced by u - rint(u) (exact),
//     then sincospif of the fp32 rest, off by 2^-25 of a half turn.  The frequency and
//     the product are off by a few 2^-53, relatively: p f_i 2^-50 of angle at most,
//     2^-25 of a half turn at positions of about 2^27.
//   * An item is two vectors of V elements, the halves of V pairs (HALF: V dims
//     and the V dims rotary_dim / 2 further; INTERLEAVED: 2 V neighbours) or, past
//     rotary_dim, one vector that is copied.  An item reads all it needs before it
//     writes, which makes y = x safe.
//   * V is the widest vector (16 bytes at most) that divides rotary_dim / 2, the
//     copied rest, every stride and both addresses.
//   * Loads in flight come from many threads (2048 an SM): two items at a time a thread
//     measured 1.07 times slower than one, four 1.4 times.  32768 positions of 40 heads,
//     fp16, 0.67 GB: 110 to 121 us, the rate of a copy being 104; 8198 of 18 heads, fp32, half
//     of each turned, 0.15 GB: 35 us.
#include <algorithm>
#include <cmath>

#include "gtq_internal.h"

namespace gtq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 128;

// Division by a number known at launch: one multiplication where that is exact (dividends up to
// `most` with most * d below 2^32), else a division.
struct Divisor {
  uint32_t d, m;
  void set(uint32_t by, uint64_t most) {
    d = by;
    m = by > 1 && most * by < (1ull << 32) ? (uint32_t)((1ull << 32) / by + 1) : 0;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return m ? __umulhi(n, m) : n / d; }
};

struct RopeSide {
  const uint8_t* x;
  uint8_t* y;
  int heads;
  int64_t xs[3], ys[3];  // bytes: sequence, head, token
};

struct RopeArgs {
  RopeSide t[2];
  const int64_t* pos;
  int64_t pos_stride, pos0;
  int64_t n_rows;  // batch * tokens
  int64_t tokens;
  int pairs;       // rotary_dim / 2
  int rot_items;   // pairs / V
  int items;       // rot_items + copied vectors
  int per_tok;     // items of a position: all heads'
  Divisor by_tok, by_items;
  float magnitude;
  int backward;
  double turns[kMaxPairs];  // f_i / (2 pi)
};

template <typename E, int V>
struct alignas(sizeof(E) * V) Vec {
  E e[V];
};

__device__ __forceinline__ float to_f(__half h) { return __half2float(h); }
__device__ __forceinline__ float to_f(float f) { return f; }
__device__ __forceinline__ void from_f(__half& o, float f) { o = __float2half_rn(f); }
__device__ __forceinline__ void from_f(float& o, float f) { o = f; }

template <typename E, int V, bool HALF, int TOK>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs[TOK][kMaxPairs];
  __shared__ int64_t seq[TOK];  // sequence of each position
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * TOK;
  const int n_tok = (int)(a.n_rows - row0 < TOK ? a.n_rows - row0 : TOK);
  if (tid < n_tok) seq[tid] = (row0 + tid) / a.tokens;
  for (int i = tid; i < n_tok * a.pairs; i += kRopeThreads) {
    const int r = i / a.pairs, j = i - r * a.pairs;
    const int64_t row = row0 + r, b = row / a.tokens, t = row - b * a.tokens;
    const int64_t p = a.pos ? a.pos[b * a.pos_stride + t] : a.pos0 + t;
    const double u = (double)p * a.turns[j];
    float s, c;
    sincospif(2.f * (float)(u - rint(u)), &s, &c);
    cs[r][j] = make_float2(c * a.magnitude, (a.backward ? -s : s) * a.magnitude);
  }
  __syncthreads();
  const int total = n_tok * a.per_tok;
  using W = Vec<E, V>;
  for (int i = tid; i < total; i += kRopeThreads) {
    const int r = TOK == 1 ? 0 : (int)a.by_tok.div((uint32_t)i), in_tok = i - r * a.per_tok;
    int h = (int)a.by_items.div((uint32_t)in_tok);
    const int item = in_tok - h * a.items;
    const bool second = h >= a.t[0].heads;
    const RopeSide& sd = a.t[second ? 1 : 0];
    if (second) h -= a.t[0].heads;
    const int64_t b = seq[r], t = row0 + r - b * a.tokens;
    const E* x = reinterpret_cast<const E*>(sd.x + b * sd.xs[0] + h * sd.xs[1] + t * sd.xs[2]);
    E* y = reinterpret_cast<E*>(sd.y + b * sd.ys[0] + h * sd.ys[1] + t * sd.ys[2]);
    if (item < a.rot_items) {
      const int o0 = HALF ? item * V : 2 * item * V;
      const int o1 = HALF ? o0 + a.pairs : o0 + V;
      const W u0 = *reinterpret_cast<const W*>(x + o0), u1 = *reinterpret_cast<const W*>(x + o1);
      W v0, v1;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 w = cs[r][item * V + e];
        if (HALF) {
          const float p = to_f(u0.e[e]), q = to_f(u1.e[e]);
          from_f(v0.e[e], p * w.x - q * w.y);
          from_f(v1.e[e], q * w.x + p * w.y);
        } else {  // pair e: elements 2e, 2e + 1 of the two vectors side by side
          const int e0 = (2 * e) % V, e1 = (2 * e + 1) % V;
          const float p = to_f(2 * e < V ? u0.e[e0] : u1.e[e0]);
          const float q = to_f(2 * e + 1 < V ? u0.e[e1] : u1.e[e1]);
          from_f(2 * e < V ? v0.e[e0] : v1.e[e0], p * w.x - q * w.y);
          from_f(2 * e + 1 < V ? v0.e[e1] : v1.e[e1], q * w.x + p * w.y);
        }
      }
      *reinterpret_cast<W*>(y + o0) = v0;
      *reinterpret_cast<W*>(y + o1) = v1;
    } else {
      const int o = 2 * a.pairs + (item - a.rot_items) * V;
      *reinterpret_cast<W*>(y + o) = *reinterpret_cast<const W*>(x + o);
    }
  }
}

template <typename E, int V>
cudaError_t launch_v(const RopeArgs& a, bool half, cudaStream_t s) {
  // one position a block while that fills the GPU's SMs a few times over at most
  // (a decode step: 16 positions are 16 blocks); four beyond, where an angle's cost
  // and a block's start spread over more rows
  const bool few = a.n_rows < 1024;
  const unsigned grid = (unsigned)(few ? a.n_rows : (a.n_rows + 3) / 4);
  if (few) {
    if (half) rope_kernel<E, V, true, 1><<<grid, kRopeThreads, 0, s>>>(a);
    else rope_kernel<E, V, false, 1><<<grid, kRopeThreads, 0, s>>>(a);
  } else {
    if (half) rope_kernel<E, V, true, 4><<<grid, kRopeThreads, 0, s>>>(a);
    else rope_kernel<E, V, false, 4><<<grid, kRopeThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

// Frequencies of a config, in turns per position.
void frequencies(const gtq_rope_config& c, double* turns) {
  const double two_pi = 6.283185307179586476925286766559;
  const int r = c.rotary_dim;
  double lo = 0, hi = 0;
  if (c.scaling == GTQ_ROPE_YARN) {
    auto at = [&](double n) {
      return r * std::log(c.original_context / (n * two_pi)) / (2 * std::log(c.theta));
    };
    lo = std::max(std::floor(at(c.high_freq)), 0.0);
    hi = std::min(std::ceil(at(c.low_freq)), (double)r - 1);
  }
  for (int i = 0; i < r / 2; ++i) {
    double f = std::pow(c.theta, -2.0 * i / r);
    if (c.scaling == GTQ_ROPE_LINEAR) {
      f /= c.factor;
    } else if (c.scaling == GTQ_ROPE_LLAMA3) {
      const double n = c.original_context * f / two_pi;
      const double s = std::min(1.0, std::max(0.0, (n - c.low_freq) / (c.high_freq - c.low_freq)));
      f = (1 - s) * f / c.factor + s * f;
    } else if (c.scaling == GTQ_ROPE_YARN) {
      const double s = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      f = s * f / c.factor + (1 - s) * f;
    }
    turns[i] = f / two_pi;
  }
}

}  // namespace

cudaError_t launch_rope(const gtq_rope_config& c, int64_t batch, int64_t tokens, const int64_t* pos,
                        int64_t pos_stride, int64_t pos0, const gtq_rope_tensor* q,
                        const gtq_rope_tensor* k, cudaStream_t s) {
  const int es = c.dtype == GTQ_DTYPE_FP16 ? 2 : 4;
  RopeArgs a = {};
  uint64_t align = 0;  // or of everything that the vector width has to divide (bytes)
  const gtq_rope_tensor* in[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    a.t[i].x = (const uint8_t*)in[i]->x;
    a.t[i].y = (uint8_t*)in[i]->y;
    a.t[i].heads = in[i]->heads;
    align |= (uintptr_t)in[i]->x | (uintptr_t)in[i]->y;
    const int64_t extent[3] = {batch, in[i]->heads, tokens};
    for (int d = 0; d < 3; ++d) {
      a.t[i].xs[d] = in[i]->x_strides[d] * es;
      a.t[i].ys[d] = in[i]->y_strides[d] * es;
      if (extent[d] > 1) align |= (uint64_t)a.t[i].xs[d] | (uint64_t)a.t[i].ys[d];
    }
  }
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.pos0 = pos0;
  a.n_rows = batch * tokens;
  a.tokens = tokens;
  a.pairs = c.rotary_dim / 2;
  a.magnitude = (float)c.magnitude;
  a.backward = c.backward;
  frequencies(c, a.turns);
  align |= (uint64_t)(a.pairs * es) | (uint64_t)((c.head_dim - c.rotary_dim) * es);
  int v = 16 / es;
  while (v > 1 && align % (uint64_t)(v * es)) v /= 2;
  a.rot_items = a.pairs / v;
  a.items = a.rot_items + (c.head_dim - c.rotary_dim) / v;
  a.per_tok = (a.t[0].heads + a.t[1].heads) * a.items;
  a.by_tok.set((uint32_t)a.per_tok, 4ull * a.per_tok);
  a.by_items.set((uint32_t)a.items, (uint64_t)a.per_tok);
  const bool half = c.rope_pairing == GTQ_PAIRING_HALF;
  if (es == 2) {
    switch (v) {
      case 8: return launch_v<__half, 8>(a, half, s);
      case 4: return launch_v<__half, 4>(a, half, s);
      case 2: return launch_v<__half, 2>(a, half, s);
      default: return launch_v<__half, 1>(a, half, s);
    }
  }
  switch (v) {
    case 4: return launch_v<float, 4>(a, half, s);
    case 2: return launch_v<float, 2>(a, half, s);
    default: return launch_v<float, 1>(a, half, s);
  }
}

}  // namespace gtq
