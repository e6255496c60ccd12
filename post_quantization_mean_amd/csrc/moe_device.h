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

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// Sums of N values over the block's THREADS threads, in every thread. `red` holds THREADS / 64 * N floats
// used by this call alone between two barriers of other calls.
template <int THREADS, int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if constexpr (THREADS > 64) {
    constexpr int W = THREADS / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[wave * N + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[w * N + k];
      v[k] = s;
    }
  }
}

}  // namespace awq
