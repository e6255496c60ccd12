// Rotary positions over one or several axes, and their gradient (the same rotation, backwards).
//
// Bound by memory: every element is read once and written once, with three operations on it. A thread holds the cosines
// and sines of kVec pairs of one token and turns those pairs in head after head, so that an angle (float64: the product, its
// reduction to a quarter turn; float32: the series) is formed once for many heads.
#include "attn.h"
#include "moe_device.h"

namespace awq {
namespace {

constexpr int kThreads = 256;

// cos and sin of position * freq. The quarter turns are taken off in float64 (pi / 2 in two parts), so that far positions lose
// nothing; what is left, at most pi / 4, goes through the Taylor series in float32: the first terms left out are
// below 2^-28 of the result.
__device__ __forceinline__ void cos_sin(int64_t position, float freq, float& c, float& s) {
  constexpr double kTwoOverPi = 0.63661977236758134308;
  constexpr double kHi = 1.57079632679489655800, kLo = 6.12323399573676603587e-17;
  const double angle = (double)position * (double)freq;
  const double quarters = rint(angle * kTwoOverPi);
  const float r = (float)fma(-quarters, kLo, fma(-quarters, kHi, angle));
  const float z = r * r;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(z, sn, 1.f / 120.f);
  sn = fmaf(z, sn, -1.f / 6.f);
  sn = fmaf(r * z, sn, r);
  float cs = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  cs = fmaf(z, cs, -1.f / 720.f);
  cs = fmaf(z, cs, 1.f / 24.f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.f);
  const int q = (int)(long long)quarters;
  const float a = q & 1 ? sn : cs, b = q & 1 ? cs : sn;
  c = (q + 1) & 2 ? -a : a;
  s = q & 2 ? -b : b;
}

// Block (x: token, y: part of the heads). Threads: items of a head (chunks of kVec pairs, then chunks of the channels that are
// only copied) times heads.
template <typename T, bool PAIRS>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int pair_items, int items, int heads_at_once) {
  constexpr int V = kVec<T>;
  const int item = (int)threadIdx.x % items;
  int head = (int)threadIdx.x / items + (int)blockIdx.y * heads_at_once;
  if ((int)threadIdx.x >= items * heads_at_once) return;
  const int64_t t = blockIdx.x;
  const T* x = (const T*)a.x.p + t * a.x.ld + head * a.x.ld_head;
  T* out = (T*)a.out.p + t * a.out.ld + head * a.out.ld_head;
  const int step = heads_at_once * (int)gridDim.y;
  const int64_t x_step = step * a.x.ld_head, out_step = step * a.out.ld_head;
  if (item >= pair_items) {
    const int i = a.rot_dim + (item - pair_items) * V;
    for (; head < a.n_heads; head += step, x += x_step, out += out_step) {
      float v[V];
      load_chunk(x, i, a.head_dim, v);
      store_chunk(out, i, a.head_dim, v);
    }
    return;
  }
  const int half = a.rot_dim / 2, first = item * V;
  float c[V], s[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int i = min(first + k, half - 1);
    const int axis = a.axis ? a.axis[i] : 0;
    int64_t p = 0;
    if (axis >= 0 && axis < a.n_axes)
      p = a.pos64 ? ((const int64_t*)a.positions)[axis * a.ld_positions + t]
                  : (int64_t)((const int32_t*)a.positions)[axis * a.ld_positions + t];
    cos_sin(p, a.inv_freq[i], c[k], s[k]);
    c[k] *= a.cos_scale;
    s[k] *= a.sin_scale;
  }
  // two chunks: the pairs' first and second channels, or the channels 2 first .. of adjacent pairs
  const int at = PAIRS ? 2 * first : first, end = PAIRS ? a.rot_dim : half;
  const int at2 = PAIRS ? at + V : half + first, end2 = a.rot_dim;
#pragma unroll 2
  for (; head < a.n_heads; head += step, x += x_step, out += out_step) {
    float u[V], w[V], p[V], q[V];
    load_chunk(x, at, end, u);
    load_chunk(x, at2, end2, w);
    if constexpr (PAIRS) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float lo = 2 * k < V ? u[(2 * k) % V] : w[(2 * k) % V];
        const float hi = 2 * k < V ? u[(2 * k + 1) % V] : w[(2 * k + 1) % V];
        const float lo2 = fmaf(lo, c[k], -(hi * s[k])), hi2 = fmaf(hi, c[k], lo * s[k]);
        if (2 * k < V) p[(2 * k) % V] = lo2, p[(2 * k + 1) % V] = hi2;
        else q[(2 * k) % V] = lo2, q[(2 * k + 1) % V] = hi2;
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        p[k] = fmaf(u[k], c[k], -(w[k] * s[k]));
        q[k] = fmaf(w[k], c[k], u[k] * s[k]);
      }
    }
    store_chunk(out, at, end, p);
    store_chunk(out, at2, end2, q);
  }
}

template <typename T>
hipError_t launch(const RopeArgs& a, bool pairs, hipStream_t stream) {
  constexpr int V = kVec<T>;
  const int pair_items = (a.rot_dim / 2 + V - 1) / V;
  const int copies = a.in_place ? 0 : (a.head_dim - a.rot_dim + V - 1) / V;
  const int items = pair_items + copies;  // at most 128 (512 float32 channels that are copied)
  const int at_once = min(kThreads / items, a.n_heads);
  const dim3 grid((unsigned)a.n_tokens, 1);
  if (pairs) rope_kernel<T, true><<<grid, kThreads, 0, stream>>>(a, pair_items, items, at_once);
  else rope_kernel<T, false><<<grid, kThreads, 0, stream>>>(a, pair_items, items, at_once);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int dtype, bool pairs, hipStream_t stream) {
  return dtype == 0 ? launch<float>(a, pairs, stream) : dtype == 1 ? launch<Bf16>(a, pairs, stream) : launch<F16>(a, pairs, stream);
}

}  // namespace awq
