// The paged cache of 4-bit keys and values: quantizing new tokens into their slots, and reading slots back.
//
// Both are bound by memory: a head's row of 128 16-bit channels is 256 bytes outside and 68 bytes in the cache. A group (up
// to 128 consecutive channels) belongs to kLanes = 4, 8 or 16 neighbouring lanes of 8 channels each, which find its minimum
// and maximum by lane exchanges. A block takes a head of kTile consecutive tokens, keys or values, so that the 64-byte
// rows of codes and the 4-byte parameters of tokens in consecutive slots are written as whole lines by one compute die.
#include "attn.h"
#include "moe_device.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr float kLargest = 65024.f;
constexpr uint32_t kNanParams = 0x7E007E00u;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

template <int LANES, typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  v = f(v, dpp<kDppXor1>(v));
  v = f(v, dpp<kDppXor2>(v));
  if constexpr (LANES > 4) v = f(v, dpp<kDppHalfMirror>(v));
  if constexpr (LANES > 8) v = f(v, dpp<kDppRowMirror>(v));
  return v;
}

__device__ __forceinline__ int64_t slot_of(const Kv4MoveArgs& a, int64_t t) {
  const int64_t s = a.slots64 ? ((const int64_t*)a.slots)[t] : (int64_t)((const int32_t*)a.slots)[t];
  return s >= 0 && s < a.c.n_pages << a.c.page_log2 ? s : -1;
}

// 8 consecutive channels i .. i + 7 of a row; i is a multiple of 8 and so is the row's width.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int i, float (&x)[8]) {
  constexpr int V = kVec<T>;
#pragma unroll
  for (int c = 0; c < 8 / V; ++c) {
    const Chunk<T> u = *reinterpret_cast<const Chunk<T>*>(row + i + c * V);
#pragma unroll
    for (int k = 0; k < V; ++k) x[c * V + k] = to_f32(u.v[k]);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int i, const float (&x)[8]) {
  constexpr int V = kVec<T>;
#pragma unroll
  for (int c = 0; c < 8 / V; ++c) {
    Chunk<T> u;
#pragma unroll
    for (int k = 0; k < V; ++k) u.v[k] = from_f32<T>(x[c * V + k]);
    *reinterpret_cast<Chunk<T>*>(row + i + c * V) = u;
  }
}

// float16 bits of v >= 0, rounded once: to float32 towards zero with the lost bits' presence kept in the lowest one, then
// to nearest even.
__device__ __forceinline__ uint32_t f16_of(double v) {
  float f = (float)v;
  if ((double)f > v) f = __uint_as_float(__float_as_uint(f) - 1);
  if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1);
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
}

// The code of x. float32 decides unless the quotient lies next to a border of two codes: its error there is below 2^-18
// (three roundings of a quotient below 16), and within 2^-16 of a border float64 decides.
__device__ __forceinline__ uint32_t code_of(float x, float step, float inv, float offset) {
  const float q = (x - offset) * inv;
  float n = rintf(q);
  if (fabsf(fabsf(q - n) - 0.5f) < 0x1p-16f) n = (float)rint(((double)x - (double)offset) / (double)step);
  return (uint32_t)fminf(fmaxf(n, 0.f), 15.f);
}

template <typename T, int LANES>
__global__ __launch_bounds__(kThreads) void write_kernel(Kv4MoveArgs a, CHeads k, CHeads v, int tile) {
  constexpr int kAtOnce = kThreads / LANES;
  const int which = (int)blockIdx.y & 1, group = ((int)blockIdx.y >> 1) % a.c.n_groups, head = ((int)blockIdx.y >> 1) / a.c.n_groups;
  const CHeads from = which ? v : k;
  const int lane = (int)threadIdx.x % LANES;
  const int channel = group * 128 + lane * 8;
  const bool there = channel < a.c.head_dim;
  const int page = 1 << a.c.page_log2, row_bytes = a.c.head_dim / 2;
  const int64_t in_head = which * a.c.n_kv + head;
  const int64_t first = (int64_t)blockIdx.x * tile, last = min(first + tile, a.n_tokens);
  for (int64_t t = first + (int)threadIdx.x / LANES; t < last; t += kAtOnce) {
    const int64_t slot = slot_of(a, t);
    if (slot < 0) continue;  // the lanes of a group agree
    float x[8];
    if (there) load8((const T*)from.p + t * from.ld + head * from.ld_head, channel, x);
    // lanes past the head's last channel repeat nothing: their bounds do not count
    float lo = __builtin_inff(), hi = -__builtin_inff(), nan = 0.f;
    if (there) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        nan = fmaf(x[i], 0.f, nan);  // NaN for a NaN or an infinity
        x[i] = fminf(fmaxf(x[i], -kLargest), kLargest);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
      }
    }
    lo = over_lanes<LANES>(lo, [](float p, float q) { return fminf(p, q); });
    hi = over_lanes<LANES>(hi, [](float p, float q) { return fmaxf(p, q); });
    nan = over_lanes<LANES>(nan, [](float p, float q) { return p + q; });
    const uint32_t step16 = f16_of(((double)hi - (double)lo) / 15.0);
    const uint32_t offset16 = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo);
    const bool fine = nan == 0.f;
    const float step = (float)__builtin_bit_cast(_Float16, (uint16_t)step16);
    const float offset = (float)__builtin_bit_cast(_Float16, (uint16_t)offset16);
    const float inv = 1.f / step;
    const int at = (int)(slot & (page - 1));
    if (there) {
      uint32_t word = 0;
      if (fine && step > 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) word |= code_of(x[i], step, inv, offset) << (4 * i);
      }
      uint8_t* to = a.c.codes + (slot >> a.c.page_log2) * a.c.page_codes + (in_head * page + at) * row_bytes + channel / 2;
      *reinterpret_cast<uint32_t*>(to) = word;
    }
    if (lane == 0)
      a.c.params[(slot >> a.c.page_log2) * a.c.page_params + (in_head * a.c.n_groups + group) * page + at] =
          fine ? step16 | offset16 << 16 : kNanParams;
  }
}

template <typename T, int LANES>
__global__ __launch_bounds__(kThreads) void read_kernel(Kv4MoveArgs a, Heads k, Heads v, int tile) {
  constexpr int kAtOnce = kThreads / LANES;
  const int which = (int)blockIdx.y & 1, group = ((int)blockIdx.y >> 1) % a.c.n_groups, head = ((int)blockIdx.y >> 1) / a.c.n_groups;
  const Heads to = which ? v : k;
  if (!to.p) return;
  const int channel = group * 128 + (int)threadIdx.x % LANES * 8;
  if (channel >= a.c.head_dim) return;
  const int page = 1 << a.c.page_log2, row_bytes = a.c.head_dim / 2;
  const int64_t in_head = which * a.c.n_kv + head;
  const int64_t first = (int64_t)blockIdx.x * tile, last = min(first + tile, a.n_tokens);
  for (int64_t t = first + (int)threadIdx.x / LANES; t < last; t += kAtOnce) {
    const int64_t slot = slot_of(a, t);
    if (slot < 0) continue;
    const int at = (int)(slot & (page - 1));
    const uint32_t word = *reinterpret_cast<const uint32_t*>(
        a.c.codes + (slot >> a.c.page_log2) * a.c.page_codes + (in_head * page + at) * row_bytes + channel / 2);
    const uint32_t p = a.c.params[(slot >> a.c.page_log2) * a.c.page_params + (in_head * a.c.n_groups + group) * page + at];
    float step = (float)__builtin_bit_cast(_Float16, (uint16_t)p), offset = (float)__builtin_bit_cast(_Float16, (uint16_t)(p >> 16));
    const float nan = fmaf(step, 0.f, offset * 0.f);  // NaN where one of them is not finite
    step += nan;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf((float)(word >> (4 * i) & 15u), step, offset);
    store8((T*)to.p + t * to.ld + head * to.ld_head, channel, x);
  }
}

// Tokens of a block: as many as its threads take at once, and four times that where the blocks are many anyway.
struct Split {
  dim3 grid;
  int tile;
};
Split split(const Kv4MoveArgs& a, int lanes) {
  const int64_t rows = (int64_t)a.c.n_kv * a.c.n_groups * 2;
  int tile = kThreads / lanes;
  if ((a.n_tokens + 4 * tile - 1) / (4 * tile) * rows >= 4096) tile *= 4;
  return {dim3((unsigned)((a.n_tokens + tile - 1) / tile), (unsigned)rows), tile};
}

template <typename F>
hipError_t with_type(int dtype, F f) {
  if (dtype == 0) f(float{});
  else if (dtype == 1) f(Bf16{});
  else f(F16{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_write(const Kv4MoveArgs& a, int dtype, CHeads k, CHeads v, hipStream_t stream) {
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const int lanes = a.c.head_dim <= 32 ? 4 : a.c.head_dim <= 64 ? 8 : 16;
    const Split s = split(a, lanes);
    if (lanes == 4) write_kernel<T, 4><<<s.grid, kThreads, 0, stream>>>(a, k, v, s.tile);
    else if (lanes == 8) write_kernel<T, 8><<<s.grid, kThreads, 0, stream>>>(a, k, v, s.tile);
    else write_kernel<T, 16><<<s.grid, kThreads, 0, stream>>>(a, k, v, s.tile);
  });
}

hipError_t launch_kv4_read(const Kv4MoveArgs& a, int dtype, Heads k, Heads v, hipStream_t stream) {
  return with_type(dtype, [&](auto t) {
    using T = decltype(t);
    const int lanes = a.c.head_dim <= 32 ? 4 : a.c.head_dim <= 64 ? 8 : 16;
    const Split s = split(a, lanes);
    if (lanes == 4) read_kernel<T, 4><<<s.grid, kThreads, 0, stream>>>(a, k, v, s.tile);
    else if (lanes == 8) read_kernel<T, 8><<<s.grid, kThreads, 0, stream>>>(a, k, v, s.tile);
    else read_kernel<T, 16><<<s.grid, kThreads, 0, stream>>>(a, k, v, s.tile);
  });
}

}  // namespace awq
