// Device helpers of the W4A16 kernels (one weight matrix: w4a16.hip; one per expert: w4a16_grouped.hip):
// dequantization of packed 4-bit codes to 16-bit operands, the matrix instructions, and the stores.
// A code q of group g gives (q - zero) * step, exact in float32 (a 5-bit integer times an 11-bit mantissa)
// and rounded once, to nearest even, to the operands' type (KIND 0: bfloat16, 1: float16).
#pragma once

#include "device_common.h"
#include "lds_dma.h"

namespace awq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float a, float b, int kind) {
  if (kind == 0) return pack_bf16x2(a, b);
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

// 8 codes (one dword, element e in bits 4e..4e+3) -> 8 operands, two per register.
template <int KIND>
__device__ __forceinline__ uint4 dequant8(uint32_t w, float st, float nzs) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf((float)((w >> (4 * e)) & 15u), st, nzs);
  return make_uint4(pack2(v[0], v[1], KIND), pack2(v[2], v[3], KIND), pack2(v[4], v[5], KIND),
                    pack2(v[6], v[7], KIND));
}

template <int KIND>
__device__ __forceinline__ f32x4 mma(const uint4& a, const uint4& b, const f32x4& c) {
  if constexpr (KIND == 0)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

template <typename OutT>
__device__ __forceinline__ OutT to_out(float v, int kind);
template <>
__device__ __forceinline__ float to_out<float>(float v, int) { return v; }
template <>
__device__ __forceinline__ uint16_t to_out<uint16_t>(float v, int kind) {
  return (uint16_t)(pack2(v, 0.f, kind) & 0xFFFFu);
}

// The step and the negated offset of a group from its raw float16 step and zero-point byte.
__device__ __forceinline__ void group_params(uint32_t step_bits, uint32_t zbyte, int g, float& st, float& nzs) {
  const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)step_bits);
  const int z = (zbyte >> ((g & 1) * 4)) & 15;
  st = s;
  nzs = -(float)z * s;  // exact: 4-bit integer times an 11-bit mantissa
}

// (h & mask) | magic in one instruction: VOP3 takes no literal operand on this architecture, so the
// mask comes in a scalar register and the float16 exponent pattern in a vector register.
__device__ __forceinline__ uint32_t and_or(uint32_t h, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(h), "s"(mask), "v"(magic));
  return r;
}

// Per-lane constants of a group: fma(1024 + q, st, c0) and fma(1024 + 16 q, st16, c16) both give
// (q - zero) * step exactly.
struct MixParams {
  float st, c0, st16, c16;
};

template <int KIND>
__device__ __forceinline__ uint4 dequant8_mix(uint32_t w, const MixParams& p, uint32_t magic) {
  const uint32_t w8 = w >> 8;
  const f16x2_t h0 = __builtin_bit_cast(f16x2_t, and_or(w, 0x000F000Fu, magic));   // nibbles 0, 4
  const f16x2_t h1 = __builtin_bit_cast(f16x2_t, and_or(w, 0x00F000F0u, magic));   // 1, 5 (times 16)
  const f16x2_t h2 = __builtin_bit_cast(f16x2_t, and_or(w8, 0x000F000Fu, magic));  // 2, 6
  const f16x2_t h3 = __builtin_bit_cast(f16x2_t, and_or(w8, 0x00F000F0u, magic));  // 3, 7 (times 16)
  const float v0 = fmaf((float)h0.x, p.st, p.c0), v4 = fmaf((float)h0.y, p.st, p.c0);
  const float v1 = fmaf((float)h1.x, p.st16, p.c16), v5 = fmaf((float)h1.y, p.st16, p.c16);
  const float v2 = fmaf((float)h2.x, p.st, p.c0), v6 = fmaf((float)h2.y, p.st, p.c0);
  const float v3 = fmaf((float)h3.x, p.st16, p.c16), v7 = fmaf((float)h3.y, p.st16, p.c16);
  return make_uint4(pack2(v0, v1, KIND), pack2(v2, v3, KIND), pack2(v4, v5, KIND), pack2(v6, v7, KIND));
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int KIND, bool ZC>
__device__ __forceinline__ void mma32(const uint4& a, const uint4& b, f32x16& c) {
  const f32x16 zero = {};
  if constexpr (KIND == 0)
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                ZC ? zero : c, 0, 0, 0);
  else
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                               ZC ? zero : c, 0, 0, 0);
}

// Byte j of a word as a float (v_cvt_f32_ubyte{j}: one instruction; written out because the compiler
// otherwise extracts the byte with a bit-field instruction first when it knows the upper bits are zero).
template <int J>
__device__ __forceinline__ float ubyte_f32(uint32_t w) {
  float f;
  if constexpr (J == 0) asm("v_cvt_f32_ubyte0 %0, %1" : "=v"(f) : "v"(w));
  else if constexpr (J == 1) asm("v_cvt_f32_ubyte1 %0, %1" : "=v"(f) : "v"(w));
  else if constexpr (J == 2) asm("v_cvt_f32_ubyte2 %0, %1" : "=v"(f) : "v"(w));
  else asm("v_cvt_f32_ubyte3 %0, %1" : "=v"(f) : "v"(w));
  return f;
}

// 8 codes (one word: element 2j in the low nibble of byte j, 2j+1 in the high one) -> 8 operands,
// (q - zero) * step rounded once to the 16-bit type; the low and high nibbles are masked four at a
// time and each byte converted directly.
template <int KIND>
__device__ __forceinline__ uint4 dequant8_bytes(uint32_t w, float st, float nzs) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const float v[8] = {fmaf(ubyte_f32<0>(lo), st, nzs), fmaf(ubyte_f32<0>(hi), st, nzs),
                      fmaf(ubyte_f32<1>(lo), st, nzs), fmaf(ubyte_f32<1>(hi), st, nzs),
                      fmaf(ubyte_f32<2>(lo), st, nzs), fmaf(ubyte_f32<2>(hi), st, nzs),
                      fmaf(ubyte_f32<3>(lo), st, nzs), fmaf(ubyte_f32<3>(hi), st, nzs)};
  return make_uint4(pack2(v[0], v[1], KIND), pack2(v[2], v[3], KIND), pack2(v[4], v[5], KIND),
                    pack2(v[6], v[7], KIND));
}

// group_params reading only the zero-point byte's low 8 bits (one byte-to-float conversion, the nibble
// then split off in exact float arithmetic): a byte loaded in one loop iteration and used in the next
// then needs no zero extension, which the compiler would otherwise place at the loop head and wait
// there for the load in flight
__device__ __forceinline__ void tile_group_params(uint32_t step_bits, uint32_t zbyte, int g, float& st, float& nzs) {
  const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)step_bits);
  const float zb = (float)(zbyte & 0xFFu);           // 0 .. 255
  const float zhi = __builtin_floorf(zb * 0.0625f);  // high nibble (exact)
  const float z = (g & 1) ? zhi : __builtin_fmaf(-16.f, zhi, zb);
  st = s;
  nzs = -z * s;  // exact: 4-bit integer times an 11-bit mantissa
}

}  // namespace awq
