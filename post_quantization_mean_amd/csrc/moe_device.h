// Device helpers of the mixture-of-experts block's element-wise kernels: storage types and chunks of
// 16 bytes of a row at any alignment.
#pragma once

#include "device_common.h"

namespace awq {

struct Bf16 {
  uint16_t v;
};
struct F16 {
  uint16_t v;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (__is_same(T, Bf16)) return bf16_to_f32(v.v);
  else return (float)__builtin_bit_cast(_Float16, v.v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float f) {
  if constexpr (sizeof(T) == 4) return f;
  else if constexpr (__is_same(T, Bf16)) return Bf16{(uint16_t)(pack_bf16x2(f, 0.f) & 0xFFFFu)};
  else return F16{__builtin_bit_cast(uint16_t, (_Float16)f)};
}

// Elements of a 16-byte chunk.
template <typename T>
inline constexpr int kVec = 16 / (int)sizeof(T);

// 16 bytes at the alignment of one element: the memory path takes 16-byte accesses at any address, so a
// row that starts anywhere is moved in whole chunks.
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Chunk {
  T v[kVec<T>];
};

// Elements i .. i + kVec - 1 of a row of width d; elements past its end are not touched (loaded as zero).
template <typename T>
__device__ __forceinline__ void load_chunk(const T* row, int i, int d, float (&v)[kVec<T>]) {
  constexpr int N = kVec<T>;
  if (i + N <= d) {
    const Chunk<T> c = *reinterpret_cast<const Chunk<T>*>(row + i);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = to_f32(c.v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = i + k < d ? to_f32(row[i + k]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int i, int d, const float (&v)[kVec<T>]) {
  constexpr int N = kVec<T>;
  if (i + N <= d) {
    Chunk<T> c;
#pragma unroll
    for (int k = 0; k < N; ++k) c.v[k] = from_f32<T>(v[k]);
    *reinterpret_cast<Chunk<T>*>(row + i) = c;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (i + k < d) row[i + k] = from_f32<T>(v[k]);
  }
}

// A thread's chunk of a row of width d >= kVec as whole loads without a branch: the chunk at element i, moved back
// to end with the row where it would pass its end. `skip` counts its leading elements that belong to the chunk
// before (kVec or more: all of it).
template <typename T>
struct Place {
  int at, skip;
  __device__ __forceinline__ Place(int i, int d) : at(min(i, d - kVec<T>)), skip(i - min(i, d - kVec<T>)) {}
};

template <typename T>
__device__ __forceinline__ uint4 load_raw(const T* row, const Place<T>& p) {
  return __builtin_bit_cast(uint4, *reinterpret_cast<const Chunk<T>*>(row + p.at));
}

// The chunk with the skipped elements zero.
template <typename T>
__device__ __forceinline__ uint4 own_raw(uint4 u, int skip) {
  constexpr int per = 4 / (int)sizeof(T);
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = skip - j * per;  // skipped elements of this word
    w[j] = n <= 0 ? w[j] : n >= per ? 0u : w[j] & 0xFFFF0000u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// STREAM: past the second-level caches.
template <typename T, bool STREAM = false>
__device__ __forceinline__ void store_own(T* row, const Place<T>& p, const float (&v)[kVec<T>]) {
  typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));  // at any element
  Chunk<T> c;
#pragma unroll
  for (int k = 0; k < kVec<T>; ++k) c.v[k] = from_f32<T>(v[k]);
  if (p.skip == 0) {
    Words* to = reinterpret_cast<Words*>(row + p.at);
    if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(Words, c), to);
    else *to = __builtin_bit_cast(Words, c);
  } else {
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k)
      if (k >= p.skip) row[p.at + k] = c.v[k];
  }
}

// Element k of a chunk's bits.
template <typename T>
__device__ __forceinline__ float raw_f32(const uint4& u, int k) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[k]);
  else if constexpr (__is_same(T, Bf16)) return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)(k & 1 ? w[k >> 1] >> 16 : w[k >> 1]));
}

// A chunk of ones.
template <typename T>
__device__ __forceinline__ uint4 raw_ones() {
  const uint32_t one = sizeof(T) == 4 ? 0x3F800000u : __is_same(T, Bf16) ? 0x3F803F80u : 0x3C003C00u;
  return make_uint4(one, one, one, one);
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(
                 float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}

// Sum over each row of 16 lanes, in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  return dpp_add<kDppRowMirror>(dpp_add<kDppHalfMirror>(dpp_add<kDppXor2>(dpp_add<kDppXor1>(v))));
}

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// Sums of N values over a block of up to 16 waves, in every thread, in a fixed order. `red` holds 16 N
// floats used by this call alone between two barriers of other calls.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 16 + (threadIdx.x >> 6)] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = row16_sum((lane & 15) < waves ? red[k * 16 + (lane & 15)] : 0.f);
}

}  // namespace awq
