// Device helpers of attention over the 4-bit cache: which rows and which cached tokens a block takes, codes to float16 at the
// matrix units' operand layouts, and the softmax's lane exchanges.
#pragma once

#include "attn.h"
#include "moe_device.h"

namespace awq {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float kNothing = -1e30f;  // the running maximum (of base-2 exponents) of a row that has seen nothing
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kAlign = 32;  // cached tokens are taken in aligned runs of this many

// Rows of one key head: row r of a sequence is its new token r / group and query head r % group of the key head's.
struct RowTile {
  int seq, row0, rows;      // first row of the tile, rows of the sequence (rows <= row0: nothing to do)
  int64_t token0;           // the sequence's first new token
  int kv_len, shift;        // new token i stands at i + shift
};

// Tiles of `tile_rows` rows are dealt to the sequences without knowing their lengths on the host: sequence s starts at
// floor(its first row over all sequences / tile_rows) + s, which leaves it enough tiles, at most one of them empty.
__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, int tile) {
  RowTile r;
  int q_len, local;
  if (a.q_offsets) {
    int lo = 0, hi = a.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)a.q_offsets[mid] * a.group / a.tile_rows + mid <= tile) lo = mid;
      else hi = mid - 1;
    }
    r.seq = lo;
    const int64_t begin = min(max((int64_t)a.q_offsets[lo], (int64_t)0), a.n_tokens);
    const int64_t end = min(max((int64_t)a.q_offsets[lo + 1], begin), a.n_tokens);
    r.token0 = begin;
    q_len = (int)(end - begin);
    const int64_t first = (int64_t)a.q_offsets[lo] * a.group / a.tile_rows + lo;
    local = first <= tile && tile - first <= 0x7FFFFFFF / a.tile_rows ? (int)(tile - first) : -1;
  } else {
    const int tiles = (a.each * a.group + a.tile_rows - 1) / a.tile_rows;
    r.seq = tile / tiles;
    local = tile - r.seq * tiles;
    r.token0 = (int64_t)r.seq * a.each;
    q_len = a.each;
  }
  r.rows = local < 0 ? 0 : q_len * a.group;  // a tile before the first sequence's rows has none
  r.row0 = max(local, 0) * a.tile_rows;
  r.kv_len = min(max(a.kv_len[r.seq], 0), a.table_width << a.c.page_log2);
  r.shift = r.kv_len - q_len;
  return r;
}

// The cached tokens that row r sees: [lo, hi).
__device__ __forceinline__ void row_range(const AttnArgs& a, const RowTile& t, int r, int& lo, int& hi) {
  const int p = t.shift + r / a.group;
  hi = r < t.rows ? (a.causal ? min(t.kv_len, p + 1) : t.kv_len) : 0;
  lo = a.window ? max(0, p - a.window + 1) : 0;
}

// The cached tokens that a tile's rows see together, and their blocks' share: at least a.chunk, and more where the caller's
// idea of the longest sequence was too short for a.n_chunks blocks.
struct KvSpan {
  int begin, end, chunk, parts;
};
__device__ __forceinline__ KvSpan kv_span(const AttnArgs& a, const RowTile& t) {
  KvSpan s;
  const int last = min(t.row0 + a.tile_rows, t.rows) - 1;
  int unused;
  row_range(a, t, t.row0, s.begin, unused);
  row_range(a, t, last, unused, s.end);
  s.begin = s.begin / kAlign * kAlign;
  const int n = max(0, s.end - s.begin);
  s.chunk = max(a.chunk, ((n + a.n_chunks - 1) / a.n_chunks + kAlign - 1) / kAlign * kAlign);
  s.parts = (n + s.chunk - 1) / s.chunk;
  return s;
}

__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }
__device__ __forceinline__ uint32_t as_u32(h2 v) { return __builtin_bit_cast(uint32_t, v); }

// A pair of params whose step or offset is not finite, as NaNs.
__device__ __forceinline__ uint32_t finite_or_nan(uint32_t w) {
  return (((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) ? 0x7E007E00u : w;
}
__device__ __forceinline__ bool not_finite(uint32_t w) { return (((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) != 0; }

// Codes of bits 0 - 3 and 4 - 7 of both halves of u as offset + code * step, one rounding. A code under the exponent of
// 1024 is 1024 + code (bits 0 - 3) or 1024 + 16 code (bits 4 - 7), from which the code itself comes back exactly.
__device__ __forceinline__ h2 low_codes(uint32_t u, h2 step, h2 offset) {
  const h2 c = as_h2((u & 0x000F000Fu) | 0x64006400u) + h2{(_Float16)-1024.f, (_Float16)-1024.f};
  return __builtin_elementwise_fma(c, step, offset);
}
__device__ __forceinline__ h2 high_codes(uint32_t u, h2 step, h2 offset) {
  const h2 c = __builtin_elementwise_fma(as_h2((u & 0x00F000F0u) | 0x64006400u), h2{(_Float16)0.0625f, (_Float16)0.0625f},
                                         h2{(_Float16)-64.f, (_Float16)-64.f});
  return __builtin_elementwise_fma(c, step, offset);
}

// Eight consecutive channels of one token: a word of codes, in the order of channels 0, 4, 1, 5, 2, 6, 3, 7 (the queries' operand is
// brought into the same order).
__device__ __forceinline__ h8 token_codes(uint32_t w, h2 step, h2 offset) {
  const uint32_t v = w >> 8;
  const h2 a = low_codes(w, step, offset), b = high_codes(w, step, offset);
  const h2 c = low_codes(v, step, offset), d = high_codes(v, step, offset);
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// bfloat16 queries reach past float16: each row is brought to a largest magnitude in [1, 2) by a power of two (`up`), which the
// scale of its scores takes back (`down`). What then lies below float16's normal numbers is below 2^-14 of the row's
// largest. Negative scales are moved into the queries, so that the largest product is the largest score.
template <bool BF16>
__device__ __forceinline__ void query_range(float largest, float scale, float& up, float& down) {
  up = down = 1.f;
  if constexpr (BF16) {
    const int e = min(max((int)(__float_as_uint(largest) >> 23) - 127, -126), 126);
    up = __uint_as_float((uint32_t)(127 - e) << 23);
    down = __uint_as_float((uint32_t)(127 + e) << 23);
  }
  if (scale < 0.f) up = -up;
}

// Four consecutive channels of the output, element `to` on.
template <bool BF16>
__device__ __forceinline__ void store4(const AttnArgs& a, int64_t to, const float (&y)[4]) {
  if (a.out_f32) {
    struct __attribute__((packed, aligned(4))) Four { float v[4]; };
    *reinterpret_cast<Four*>((float*)a.out.p + to) = Four{{y[0], y[1], y[2], y[3]}};
  } else {
    struct __attribute__((packed, aligned(2))) Four { uint16_t v[4]; } u;
#pragma unroll
    for (int k = 0; k < 4; ++k) u.v[k] = BF16 ? from_f32<Bf16>(y[k]).v : from_f32<F16>(y[k]).v;
    *reinterpret_cast<Four*>((uint16_t*)a.out.p + to) = u;
  }
}

// max or sum over the four rows of 16 lanes, in every lane
__device__ __forceinline__ float max_over_rows(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ uint32_t or_over_rows(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = a[0] | a[1];
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return b[0] | b[1];
}

}  // namespace awq
