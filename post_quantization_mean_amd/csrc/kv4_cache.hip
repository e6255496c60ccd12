// The paged cache of 4-bit keys and values: quantizing new tokens into their slots, and reading slots back.
//
// A head's row of 128 16-bit channels is 256 bytes outside and 68 bytes in the cache. Reading back is bound by memory; writing by the latency
// of blocks that load, work and store once (neither memory nor the vector units are full). To write, a group
// (up to 128 consecutive channels) belongs to kLanes = 2, 4 or 8 neighbouring lanes of 16 channels each, which find its minimum
// and maximum by lane exchanges; to read, to 4, 8 or 16 lanes of 8 channels. A block takes a head of 16 to 256 consecutive
// tokens, keys or values, so that the 64-byte rows of codes and the 4-byte parameters of tokens in consecutive slots are
// written as whole lines by one compute die. 32768 tokens of 8 heads of 128 bf16, keys and values: written in 44 us (3.9 TB/s,
// the vector units half busy; with float64 steps and codes, 8 channels a lane, 56), read back in 27 (6.3 TB/s).
#include <algorithm>
#include <type_traits>

#include "attn.h"
#include "moe_device.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kGridTokens = 32768;  // blocks of tokens: y + kGridTokens z
constexpr float kLargest = 65024.f;
constexpr uint32_t kNanParams = 0x7E007E00u;

template <int LANES, typename F>
__device__ __forceinline__ int over_lanes(int v, F f) {
  v = f(v, __builtin_amdgcn_mov_dpp(v, kDppXor1, 0xF, 0xF, true));
  if constexpr (LANES > 2) v = f(v, __builtin_amdgcn_mov_dpp(v, kDppXor2, 0xF, 0xF, true));
  if constexpr (LANES > 4) v = f(v, __builtin_amdgcn_mov_dpp(v, kDppHalfMirror, 0xF, 0xF, true));
  return v;
}

// Integers in the order of the numbers whose bits they are, a NaN past the infinity of its sign, and back.
__device__ __forceinline__ int ordered(int bits) { return bits ^ ((bits >> 31) & 0x7FFFFFFF); }

__device__ __forceinline__ int64_t slot_of(const Kv4MoveArgs& a, int64_t t) {
  const int64_t s = a.slots64 ? ((const int64_t*)a.slots)[t] : (int64_t)((const int32_t*)a.slots)[t];
  return s >= 0 && s < a.c.n_pages << a.c.page_log2 ? s : -1;
}

// 16 consecutive channels of a row, as they are stored.
template <typename T>
struct Sixteen {
  uint4 u[16 / kVec<T>];
  __device__ __forceinline__ void load(const T* from) {
#pragma unroll
    for (int c = 0; c < 16 / kVec<T>; ++c) u[c] = __builtin_bit_cast(uint4, *reinterpret_cast<const Chunk<T>*>(from + c * kVec<T>));
  }
  __device__ __forceinline__ float at(int i) const { return raw_f32<T>(u[i / kVec<T>], i % kVec<T>); }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& v = u[i / 4];
    return i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
  }
  // The least and the largest, as ordered integers of T's width. (Comparing as integers keeps NaNs in sight, and needs no
  // operation that makes a loaded number canonical first.)
  __device__ __forceinline__ void bounds(int& lo, int& hi) const {
    if constexpr (sizeof(T) == 4) {
      lo = hi = ordered((int)word(0));
#pragma unroll
      for (int i = 1; i < 16; ++i) {
        const int k = ordered((int)word(i));
        lo = min(lo, k);
        hi = max(hi, k);
      }
    } else {
      typedef short s2 __attribute__((ext_vector_type(2)));
      s2 l, h;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const s2 w = __builtin_bit_cast(s2, word(i));
        const s2 k = w ^ ((w >> 15) & s2{0x7FFF, 0x7FFF});
        l = i ? __builtin_elementwise_min(l, k) : k;
        h = i ? __builtin_elementwise_max(h, k) : k;
      }
      lo = min((int)l.x, (int)l.y);
      hi = max((int)h.x, (int)h.y);
    }
  }
};

// The number of an ordered integer of T's width.
template <typename T>
__device__ __forceinline__ float unordered(int k) {
  if constexpr (sizeof(T) == 4) return __uint_as_float((uint32_t)ordered(k));
  else return to_f32(T{(uint16_t)(k ^ ((k >> 31) & 0x7FFF))});
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

// float32 of v towards zero with the lost bits' presence kept in the lowest one: what rounds it to 16 bits rounds v.
__device__ __forceinline__ float odd_f32(double v) {
  float f = (float)v;
  if (fabs((double)f) > fabs(v)) f = __uint_as_float(__float_as_uint(f) - 1);
  if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1);
  return f;
}

// float16 bits of v >= 0, rounded once.
__device__ __forceinline__ uint32_t f16_of(double v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)odd_f32(v));
}

// Is offset + c * step a float32 for every code c? A product has 15 bits, so it is where the exponents do not lie far apart: then the sum's
// highest bit is at most 2^max(o, s + 4) * 2 and its lowest at least 2^(min(o, s) - 10). (The exponents: of float16, that of subnormal numbers
// and zero as 1 is the one of their lowest bit's place. An offset of zero adds nothing.)
__device__ __forceinline__ bool sums_are_exact(uint32_t params) {
  const int s = max((int)(params >> 10 & 31), 1), o = max((int)(params >> 26 & 31), 1);
  return (params & 0x7FFF0000u) == 0 || max(o, s + 4) - min(o, s) <= 12;
}

// float16 bits of (hi - lo) / 15, rounded once. float32's quotient is within 3 of its steps of the true one (the difference,
// 1 / 15 and the product are rounded once each): it decides unless it lies within 8 steps of the middle of two float16
// numbers (its low 13 bits at 0x1000) or below float16's normal numbers; then float64 decides.
__device__ __forceinline__ uint32_t step_of(float lo, float hi) {
  const float s = (hi - lo) * (1.f / 15.f);
  const uint32_t from_middle = (__float_as_uint(s) + 8u - 0x1000u) & 0x1FFFu;
  if (from_middle <= 16u || s < 0x1p-13f) return f16_of(((double)hi - (double)lo) / 15.0);
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)s);
}

// Eight codes. float32 decides unless a quotient lies next to a border of two codes: its error there is at most 2^-18 (a difference,
// a reciprocal of one step and a product, of a quotient below 16), and within 2^-16 of a border float64 decides. 16-bit
// numbers lie on a border now and then (about one in 1500), so each has a branch of its own.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float step, float inv, float offset) {
  float n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = (x[i] - offset) * inv;
    float r = rintf(q);
    if (__builtin_expect(fabsf(q - r) > 0.5f - 0x1p-16f, 0)) r = (float)rint(((double)x[i] - (double)offset) / (double)step);
    n[i] = __builtin_amdgcn_fmed3f(r, 0.f, 15.f);
  }
  const uint32_t lo = (uint32_t)fmaf(fmaf(fmaf(n[3], 16.f, n[2]), 16.f, n[1]), 16.f, n[0]);
  const uint32_t hi = (uint32_t)fmaf(fmaf(fmaf(n[7], 16.f, n[6]), 16.f, n[5]), 16.f, n[4]);
  return lo | hi << 16;
}

// Near memory's rate only while an element costs no more than some 15 vector operations: hence the decisions in float32, the bounds
// as packed integers, and 16 elements a lane beside what a group costs once.
template <typename T, int LANES, int TOKENS>
__global__ __launch_bounds__(kThreads) void write_kernel(Kv4MoveArgs a, CHeads k, CHeads v) {
  constexpr int kAtOnce = kThreads / LANES;
  const int which = (int)blockIdx.x & 1, group = ((int)blockIdx.x >> 1) % a.c.n_groups, head = ((int)blockIdx.x >> 1) / a.c.n_groups;
  const CHeads from = which ? v : k;
  const int lane = (int)threadIdx.x % LANES;
  const int channel = group * 128 + lane * 16;
  const bool there = channel < a.c.head_dim;
  const int page = 1 << a.c.page_log2, row_bytes = a.c.head_dim / 2;
  const int64_t in_head = which * a.c.n_kv + head;
  const int64_t first = (int64_t)(blockIdx.z * kGridTokens + blockIdx.y) * (TOKENS * kAtOnce) + (int)threadIdx.x / LANES;
  if (first - (int)threadIdx.x / LANES >= a.n_tokens) return;
  Sixteen<T> raw[TOKENS];
  int64_t slots[TOKENS];
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    const int64_t t = min(first + i * kAtOnce, a.n_tokens - 1);
    // lanes past the head's last channel repeat the group's first ones, and store nothing
    raw[i].load((const T*)from.p + t * from.ld + head * from.ld_head + (there ? channel : group * 128));
    slots[i] = first + i * kAtOnce < a.n_tokens ? slot_of(a, t) : -1;
  }
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    const int64_t slot = slots[i];
    if (slot < 0) continue;  // the lanes of a group agree
    int least, most;
    raw[i].bounds(least, most);
    float lo = unordered<T>(over_lanes<LANES>(least, [](int p, int q) { return min(p, q); }));
    float hi = unordered<T>(over_lanes<LANES>(most, [](int p, int q) { return max(p, q); }));
    float x[2][8];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j / 8][j % 8] = raw[i].at(j);
    bool fine = true;
    if (!(lo >= -kLargest && hi <= kLargest)) {  // also where one of them is NaN
      fine = fabsf(lo) < __builtin_inff() && fabsf(hi) < __builtin_inff();
      lo = fminf(fmaxf(lo, -kLargest), kLargest);
      hi = fminf(fmaxf(hi, -kLargest), kLargest);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j / 8][j % 8] = fminf(fmaxf(x[j / 8][j % 8], -kLargest), kLargest);
    }
    const uint32_t step16 = step_of(lo, hi);
    const _Float16 offset16 = (_Float16)lo;
    const float step = (float)__builtin_bit_cast(_Float16, (uint16_t)step16), offset = (float)offset16;
    const int at = (int)(slot & (page - 1));
    const int64_t in_cache = slot >> a.c.page_log2;
    if (there) {
      const float inv = __builtin_amdgcn_rcpf(step);
      uint2 words = make_uint2(0, 0);
      if (fine && step > 0.f) words = make_uint2(codes_of(x[0], step, inv, offset), codes_of(x[1], step, inv, offset));
      *reinterpret_cast<uint2*>(a.c.codes + in_cache * a.c.page_codes + (in_head * page + at) * row_bytes + channel / 2) = words;
    }
    if (lane == 0)
      a.c.params[in_cache * a.c.page_params + (in_head * a.c.n_groups + group) * page + at] =
          fine ? step16 | (uint32_t)__builtin_bit_cast(uint16_t, offset16) << 16 : kNanParams;
  }
}

template <typename T, int LANES, int TOKENS>
__global__ __launch_bounds__(kThreads) void read_kernel(Kv4MoveArgs a, Heads k, Heads v) {
  constexpr int kAtOnce = kThreads / LANES;
  const int which = (int)blockIdx.x & 1, group = ((int)blockIdx.x >> 1) % a.c.n_groups, head = ((int)blockIdx.x >> 1) / a.c.n_groups;
  const Heads to = which ? v : k;
  if (!to.p) return;
  const int channel = group * 128 + (int)threadIdx.x % LANES * 8;
  if (channel >= a.c.head_dim) return;
  const int page = 1 << a.c.page_log2, row_bytes = a.c.head_dim / 2;
  const int64_t in_head = which * a.c.n_kv + head;
  const int64_t first = (int64_t)(blockIdx.z * kGridTokens + blockIdx.y) * (TOKENS * kAtOnce) + (int)threadIdx.x / LANES;
  if (first - (int)threadIdx.x / LANES >= a.n_tokens) return;
  uint32_t words[TOKENS], params[TOKENS];
  int64_t slots[TOKENS];
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    slots[i] = slot_of(a, min(first + i * kAtOnce, a.n_tokens - 1));
    const int64_t slot = max(slots[i], (int64_t)0);
    const int at = (int)(slot & (page - 1));
    words[i] = *reinterpret_cast<const uint32_t*>(a.c.codes + (slot >> a.c.page_log2) * a.c.page_codes + (in_head * page + at) * row_bytes +
                                                  channel / 2);
    params[i] = a.c.params[(slot >> a.c.page_log2) * a.c.page_params + (in_head * a.c.n_groups + group) * page + at];
  }
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    const int64_t t = first + i * kAtOnce;
    if (t >= a.n_tokens || slots[i] < 0) continue;
    const uint32_t word = words[i], p = params[i];
    float step = (float)__builtin_bit_cast(_Float16, (uint16_t)p), offset = (float)__builtin_bit_cast(_Float16, (uint16_t)(p >> 16));
    const float nan = fmaf(step, 0.f, offset * 0.f);  // NaN where one of them is not finite
    step += nan;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf((float)(word >> (4 * j) & 15u), step, offset);
    // 16 bits: not by way of a rounded float32
    if (sizeof(T) == 2 && __builtin_expect(!sums_are_exact(p), 0)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = odd_f32((double)(word >> (4 * j) & 15u) * (double)step + (double)offset);
    }
    store8((T*)to.p + t * to.ld + head * to.ld_head, channel, x);
  }
}

template <typename F>
hipError_t with_type(int dtype, F f) {
  if (dtype == 0) f(float{});
  else if (dtype == 1) f(Bf16{});
  else f(F16{});
  return hipGetLastError();
}

// f(lanes of a group, tokens of a thread): MANY tokens where the blocks are many anyway; 128 / LANES channels a lane.
template <int LANES, int MANY, typename F>
void with_split(const Kv4MoveArgs& a, F f) {
  const int lanes = a.c.head_dim <= 32 ? LANES / 4 : a.c.head_dim <= 64 ? LANES / 2 : LANES, at_once = kThreads / lanes;
  const int64_t rows = (int64_t)a.c.n_kv * a.c.n_groups * 2, blocks = (a.n_tokens + MANY * at_once - 1) / (MANY * at_once);
  const bool many = blocks * rows >= 1024;
  const int64_t n = many ? blocks : (a.n_tokens + at_once - 1) / at_once;
  // heads first: what runs at once reads whole rows of tokens
  const dim3 grid((unsigned)rows, (unsigned)std::min(n, (int64_t)kGridTokens), (unsigned)((n - 1) / kGridTokens + 1));
  const auto run = [&](auto l) {
    if (many) f(l, std::integral_constant<int, MANY>{}, grid);
    else f(l, std::integral_constant<int, 1>{}, grid);
  };
  if (lanes == LANES / 4) run(std::integral_constant<int, LANES / 4>{});
  else if (lanes == LANES / 2) run(std::integral_constant<int, LANES / 2>{});
  else run(std::integral_constant<int, LANES>{});
}

}  // namespace

hipError_t launch_kv4_write(const Kv4MoveArgs& a, int dtype, CHeads k, CHeads v, hipStream_t stream) {
  return with_type(dtype, [&](auto t) {
    with_split<8, 2>(a, [&](auto lanes, auto tokens, dim3 grid) {
      write_kernel<decltype(t), decltype(lanes)::value, decltype(tokens)::value><<<grid, kThreads, 0, stream>>>(a, k, v);
    });
  });
}

hipError_t launch_kv4_read(const Kv4MoveArgs& a, int dtype, Heads k, Heads v, hipStream_t stream) {
  return with_type(dtype, [&](auto t) {
    with_split<16, 4>(a, [&](auto lanes, auto tokens, dim3 grid) {
      read_kernel<decltype(t), decltype(lanes)::value, decltype(tokens)::value><<<grid, kThreads, 0, stream>>>(a, k, v);
    });
  });
}

}  // namespace awq
