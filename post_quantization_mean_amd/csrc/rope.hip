// Rotary positions over one or several axes, and their gradient (the same rotation, backwards).
//
// Bound by memory: every element is read once and written once, with three operations on it. An angle costs some forty
// operations (float64: the product, its reduction to a quarter turn; float32: the series) and serves all heads of a token:
// a block's threads form the cosines and sines of its tokens once, into LDS, and then turn the heads' pairs, kVec
// a thread, with the loads of kRows heads on their way. 16384 tokens of 72 heads of 128 bf16: 114 us (5.3 TB/s, a large copy's
// rate; one head's load at a time with its own cosines 170). One token of 40 heads: 2.5 us. Channels that are only copied go a
// row at a time: 136 us with 64 of 128 channels turned, 202 with 32.
#include "attn.h"
#include "moe_device.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

// cos and sin of position * freq. The product is a float64 (rounded where both factors are long: 2^-53 of the angle, 2^-22
// at angles of 2^31); its quarter turns are taken off in float64 (pi / 2 in two parts), which loses nothing more; what is left, at most pi / 4, goes through the Taylor series in float32: the first terms left out are
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

// Tokens of a block: as many as its threads have angles.
inline int tokens_of(int rot_dim) { return min(max(kThreads / (rot_dim / 2), 1), 16); }
constexpr int kAngles = 256;  // of a block, at most: AWQ_MAX_ROPE_DIM / 2
constexpr int kRows = 4;

// Block (x: tokens, y: part of their rows; a row: one head of one token). Threads: items of a row (chunks of kVec pairs, then
// chunks of the channels that are only copied) times rows.
template <typename T, bool PAIRS, bool STREAM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, int tokens, int pair_items, int items, int rows_at_once) {
  constexpr int V = kVec<T>;
  __shared__ float2 turn[kAngles];
  const int half = a.rot_dim / 2;
  const int64_t first_token = (int64_t)blockIdx.x * tokens;
  const int n = (int)min((int64_t)tokens, a.n_tokens - first_token);
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, pair = i - t * half;
    const int axis = a.axis ? a.axis[pair] : 0;
    int64_t p = 0;
    if (axis >= 0 && axis < a.n_axes) {
      const int64_t at = axis * a.ld_positions + first_token + t;
      p = a.pos64 ? ((const int64_t*)a.positions)[at] : (int64_t)((const int32_t*)a.positions)[at];
    }
    float c, s;
    cos_sin(p, a.inv_freq[pair], c, s);
    turn[i] = make_float2(c * a.cos_scale, s * a.sin_scale);
  }
  __syncthreads();
  const int item = (int)threadIdx.x % items, step = rows_at_once * (int)gridDim.y;
  int row = (int)threadIdx.x / items + (int)blockIdx.y * rows_at_once;
  if ((int)threadIdx.x >= items * rows_at_once) return;
  const int rows = n * a.n_heads;
  const T* const x = (const T*)a.x.p + first_token * a.x.ld;
  T* const out = (T*)a.out.p + first_token * a.out.ld;
  if (item >= pair_items) {
    const int i = a.rot_dim + (item - pair_items) * V;
    for (; row < rows; row += step) {
      const int t = a.by_heads.of(row), head = row - t * a.n_heads;
      float v[V];
      load_chunk(x + t * a.x.ld + head * a.x.ld_head, i, a.head_dim, v);
      store_chunk(out + t * a.out.ld + head * a.out.ld_head, i, a.head_dim, v);
    }
    return;
  }
  // two chunks: the pairs' first and second channels, or the channels 2 first .. of adjacent pairs
  const int first = item * V;
  const int at = PAIRS ? 2 * first : first, end = PAIRS ? a.rot_dim : half;
  const int at2 = PAIRS ? at + V : half + first, end2 = a.rot_dim;
  const bool whole = first + V <= half;  // both chunks
  const auto place = [&](int r, int64_t ld, int64_t ld_head) {
    const int t = a.by_heads.of(r);
    return t * ld + (r - t * a.n_heads) * ld_head;
  };
  const auto rotate = [&](int r, const float (&u)[V], const float (&w)[V], float (&p)[V], float (&q)[V]) {
    const float2* cs = turn + a.by_heads.of(r) * half;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float2 z = cs[min(first + k, half - 1)];
      if constexpr (PAIRS) {
        const float lo = 2 * k < V ? u[(2 * k) % V] : w[(2 * k) % V];
        const float hi = 2 * k < V ? u[(2 * k + 1) % V] : w[(2 * k + 1) % V];
        const float lo2 = fmaf(lo, z.x, -(hi * z.y)), hi2 = fmaf(hi, z.x, lo * z.y);
        if (2 * k < V) p[(2 * k) % V] = lo2, p[(2 * k + 1) % V] = hi2;
        else q[(2 * k) % V] = lo2, q[(2 * k + 1) % V] = hi2;
      } else {
        p[k] = fmaf(u[k], z.x, -(w[k] * z.y));
        q[k] = fmaf(w[k], z.x, u[k] * z.y);
      }
    }
  };
  if (whole) {
    for (; row < rows; row += kRows * step) {
      Chunk<T> raw[kRows][2];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {  // (past the last row: the first one again, not stored)
        const T* from = x + place(row + k * step < rows ? row + k * step : row, a.x.ld, a.x.ld_head);
        raw[k][0] = *reinterpret_cast<const Chunk<T>*>(from + at);
        raw[k][1] = *reinterpret_cast<const Chunk<T>*>(from + at2);
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int r = row + k * step;
        if (r >= rows) break;
        float u[V], w[V], p[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) u[j] = to_f32(raw[k][0].v[j]), w[j] = to_f32(raw[k][1].v[j]);
        rotate(r, u, w, p, q);
        T* to = out + place(r, a.out.ld, a.out.ld_head);
        store_own<T, STREAM>(to, Place<T>(at, end + V), p);
        store_own<T, STREAM>(to, Place<T>(at2, end2 + V), q);
      }
    }
    return;
  }
  for (; row < rows; row += step) {
    float u[V], w[V], p[V], q[V];
    const T* from = x + place(row, a.x.ld, a.x.ld_head);
    load_chunk(from, at, end, u);
    load_chunk(from, at2, end2, w);
    rotate(row, u, w, p, q);
    T* to = out + place(row, a.out.ld, a.out.ld_head);
    store_chunk(to, at, end, p);
    store_chunk(to, at2, end2, q);
  }
}

template <typename T>
hipError_t launch(const RopeArgs& a, bool pairs, hipStream_t stream) {
  constexpr int V = kVec<T>;
  const int pair_items = (a.rot_dim / 2 + V - 1) / V;
  const int copies = a.in_place ? 0 : (a.head_dim - a.rot_dim + V - 1) / V;
  const int items = pair_items + copies;  // at most 129 (float32, two of 512 channels turned)
  // few tokens: one a block, and its rows over several blocks, so that each thread has one or two
  int tokens = tokens_of(a.rot_dim);
  if (a.n_tokens < 256 * tokens) tokens = 1;
  const int rows_at_once = kThreads / items;
  const int rows = min((int64_t)tokens, a.n_tokens) * a.n_heads;
  const int parts = a.n_tokens <= 64 ? min((rows + rows_at_once - 1) / rows_at_once, 64) : 1;
  const dim3 grid((unsigned)((a.n_tokens + tokens - 1) / tokens), (unsigned)parts);
  // an output that the second-level caches do not hold goes past them
  const bool past = a.n_tokens * a.n_heads * a.rot_dim * (int64_t)sizeof(T) >= kStreamBytes;
#define ROPE(P, S) rope_kernel<T, P, S><<<grid, kThreads, 0, stream>>>(a, tokens, pair_items, items, rows_at_once)
  if (pairs) past ? ROPE(true, true) : ROPE(true, false);
  else past ? ROPE(false, true) : ROPE(false, false);
#undef ROPE
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int dtype, bool pairs, hipStream_t stream) {
  return dtype == 0 ? launch<float>(a, pairs, stream) : dtype == 1 ? launch<Bf16>(a, pairs, stream) : launch<F16>(a, pairs, stream);
}

}  // namespace awq
