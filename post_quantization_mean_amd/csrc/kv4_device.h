// Device helpers of attention over the 4-bit cache: which rows and which cached tokens a block takes, codes to float16 at the
// matrix units' operand layouts, and the softmax's lane exchanges.
#pragma once

#include "attn.h"
#include "moe_device.h"

namespace awq {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

constexpr float kLargestFloat = 3.402823466e38f;
constexpr float kNothing = -kLargestFloat;  // the reference of a row that has seen nothing
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kAlign = 32;  // cached tokens are taken in aligned runs of this many

// Rows of one key head: row r of a sequence is its new token r / group and query head r % group of the key head's.
struct RowTile {
  int seq, row0, rows;      // first row of the tile, rows of the sequence (rows <= row0: nothing to do)
  int token0;               // the sequence's first new token
  int kv_len, shift;        // new token i stands at i + shift
};

// Tiles of `tile_rows` rows are dealt to the sequences without knowing their lengths on the host: sequence s starts at
// floor(its first row over all sequences / tile_rows) + s, which leaves it enough tiles, at most one of them empty.
__device__ __forceinline__ RowTile row_tile(const AttnArgs& a, int tile) {
  RowTile r;
  int q_len, local;
  if (a.q_offsets) {
    const auto offset = [&](int seq) { return min(max(a.q_offsets[seq], 0), (int)a.n_tokens); };
    const auto first_tile = [&](int seq) { return (int)((int64_t)offset(seq) * a.group >> a.tile_log2) + seq; };
    int lo = 0, hi = a.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_tile(mid) <= tile) lo = mid;
      else hi = mid - 1;
    }
    r.seq = lo;
    r.token0 = offset(lo);
    q_len = max(offset(lo + 1) - r.token0, 0);
    local = tile - first_tile(lo);
  } else {
    const int tiles = (a.each * a.group + a.tile_rows - 1) >> a.tile_log2;
    r.seq = a.by_tiles.of(tile);
    local = tile - r.seq * tiles;
    r.token0 = r.seq * a.each;
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
  const int p = t.shift + a.by_group.of(r);
  hi = r < t.rows ? (a.causal ? min(t.kv_len, p + 1) : t.kv_len) : 0;
  lo = a.window ? max(0, p - a.window + 1) : 0;
}

// The cached tokens that a tile's rows see together: [begin, end), in units of kUnit tokens. A tile whose rows see nothing is one
// unit (its results have to be written), one without rows none.
struct KvSpan {
  int begin, end, units;
};
__device__ __forceinline__ KvSpan kv_span(const AttnArgs& a, const RowTile& t) {
  KvSpan s = {0, 0, 0};
  if (t.row0 >= t.rows) return s;
  const int last = min(t.row0 + a.tile_rows, t.rows) - 1;
  int unused;
  row_range(a, t, t.row0, s.begin, unused);
  row_range(a, t, last, unused, s.end);
  s.begin = s.begin / kAlign * kAlign;
  s.units = max(1, (max(0, s.end - s.begin) + kUnit - 1) / kUnit);
  return s;
}

// The even split. The units of all tiles and key heads (tile by tile, a tile's key heads one after the other) are laid end to
// end, and each of n_blocks blocks (fewer where a block would get less than kLeastUnits) takes an equal run of them, whatever
// the sequences' lengths: the end of one tile's tokens, whole tiles, the beginning of another's. What a block has of a
// tile that it does not have whole goes to its part 2 b (the run begins in it) or 2 b + 1 (the run ends in it), and
// join_kernel puts the parts together.
constexpr int kMostTiles = 1024;  // of a split: each block sums up their units
constexpr int kLeastUnits = 2;

struct Split {
  int total, blocks, each, more;  // units; the first `more` blocks have each + 1, the others each
  __device__ __forceinline__ Split(int units, int n_blocks) : total(units) {
    blocks = max(1, min(units / kLeastUnits, n_blocks));
    each = (int)((uint32_t)units / (uint32_t)blocks);
    more = units - each * blocks;
  }
  __device__ __forceinline__ int begin(int block) const { return block * each + min(block, more); }
  __device__ __forceinline__ int of(int unit) const {
    const int edge = more * (each + 1);
    return unit < edge ? (int)((uint32_t)unit / (uint32_t)(each + 1)) : more + (int)((uint32_t)(unit - edge) / (uint32_t)max(each, 1));
  }
};

// lds: [0 .. n_tiles] the units before each tile (one key head's), then room for the waves' sums; by the threads of a block (256 or 512).
constexpr int kPrefixInts = kMostTiles + 1 + 8;
// t, s: the tile of the last one that the thread counted.
__device__ __forceinline__ void unit_prefix(const AttnArgs& a, int* lds, RowTile& t, KvSpan& s) {
  const int tid = threadIdx.x, lane = tid & 63;
  int* const waves = lds + kMostTiles + 1;
  int before = 0;
#pragma unroll 1
  for (int first = 0; first < a.n_tiles; first += blockDim.x) {
    const int tile = first + tid;
    s.units = 0;
    if (tile < a.n_tiles) {
      t = row_tile(a, tile);
      s = kv_span(a, t);
    }
    const int n = s.units;
    int up = n;  // over the lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(up, d);
      if (lane >= d) up += v;
    }
    if (lane == 63) waves[tid >> 6] = up;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < (int)blockDim.x >> 6; ++w) {
      if (w < tid >> 6) up += waves[w];
      all += waves[w];
    }
    if (tile < a.n_tiles) lds[tile] = before + up - n;
    before += all;
    __syncthreads();
  }
  if (tid == 0) lds[a.n_tiles] = before;
  __syncthreads();
}

// Blocks (key head, tile % kGridTiles, tile / kGridTiles), or a row of them that share the work.
constexpr int kGridTiles = 32768;
inline dim3 attention_grid(const AttnArgs& a) {
  if (a.n_blocks) return dim3((unsigned)a.n_blocks);
  return dim3((unsigned)a.c.n_kv, (unsigned)(a.n_tiles < kGridTiles ? a.n_tiles : kGridTiles), (unsigned)((a.n_tiles - 1) / kGridTiles + 1));
}

// Calls take(tile, key head, begin, end, part) for each piece of this block's work; part -1: a tile's whole span.
template <bool SPLIT, typename F>
__device__ __forceinline__ void for_pieces(const AttnArgs& a, int* lds, F take) {
  if constexpr (!SPLIT) {
    const int tile = (int)(blockIdx.z * kGridTiles + blockIdx.y);
    if (tile >= a.n_tiles) return;
    // the last tiles of a causal sequence see the most: they go before its others, of all key heads (sequences in turn, the last one
    // first, whatever their lengths)
    const RowTile t = row_tile(a, a.n_tiles - 1 - tile);
    const KvSpan s = kv_span(a, t);
    if (s.units) take(t, (int)blockIdx.x, s.begin, s.end, -1);
  } else {
    struct Piece {
      RowTile t;
      KvSpan s;
      int tile;
    };
    __shared__ Piece found;
    Piece p;
    unit_prefix(a, lds, p.t, p.s);
    const int block = (int)blockIdx.x;
    if (block == 0)
      for (int i = threadIdx.x; i <= a.n_tiles; i += blockDim.x) a.prefix[i] = lds[i];
    const Split split(__builtin_amdgcn_readfirstlane(lds[a.n_tiles]) * a.c.n_kv, a.n_blocks);
    if (block >= split.blocks) return;
    int u = split.begin(block);
    const int u_end = split.begin(block + 1), of_head = a.by_kv.of(u);
    if (u >= u_end) return;
    // the tile that the first unit is of: its thread writes it down
    for (p.tile = threadIdx.x; p.tile < a.n_tiles; p.tile += blockDim.x)
      if (lds[p.tile] <= of_head && of_head < lds[p.tile + 1]) {
        if (a.n_tiles > (int)blockDim.x) {
          p.t = row_tile(a, p.tile);
          p.s = kv_span(a, p.t);
        }
        found = p;
      }
    __syncthreads();
    const auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    p.tile = uniform(found.tile);
    p.t = {uniform(found.t.seq), uniform(found.t.row0), uniform(found.t.rows), uniform(found.t.token0), uniform(found.t.kv_len),
           uniform(found.t.shift)};
    p.s = {uniform(found.s.begin), uniform(found.s.end), uniform(found.s.units)};
    bool first = true;
    while (true) {
      if (p.s.units) {
        const int at = u - uniform(lds[p.tile]) * a.c.n_kv, units = p.s.units;
        const int head = uniform((int)((uint32_t)at / (uint32_t)units)), k = at - head * units, n = min(units - k, u_end - u);
        if (!first) __syncthreads();  // LDS of the piece before
        take(p.t, head, p.s.begin + k * kUnit, min(p.s.end, p.s.begin + (k + n) * kUnit), n == units ? -1 : 2 * block + (first ? 0 : 1));
        first = false;
        u += n;
        if (u >= u_end) break;
        if (k + n < units || head + 1 < a.c.n_kv) continue;
      }
      ++p.tile;
      const RowTile t = row_tile(a, p.tile);
      p.t = {uniform(t.seq), uniform(t.row0), uniform(t.rows), uniform(t.token0), uniform(t.kv_len), uniform(t.shift)};
      const KvSpan s = kv_span(a, p.t);
      p.s = {uniform(s.begin), uniform(s.end), uniform(s.units)};
    }
  }
}

__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }
__device__ __forceinline__ uint32_t as_u32(h2 v) { return __builtin_bit_cast(uint32_t, v); }

// A pair of params whose step or offset is not finite, as NaNs.
__device__ __forceinline__ uint32_t finite_or_nan(uint32_t w) {
  return (((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) ? 0x7E007E00u : w;
}
__device__ __forceinline__ bool not_finite(uint32_t w) { return (((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) != 0; }

// A branch that is seldom taken: what it needs in other registers is moved there in the branch, not around it.
__device__ __forceinline__ bool rare(bool c) { return __builtin_expect(c, 0); }

// float16 1024 twice, in a register: an instruction takes one constant of 32 bits at most, so that masking codes and setting
// their exponent is one operation with it, two without.
__device__ __forceinline__ uint32_t code_exponent() {
  uint32_t e = 0x64006400u;
  asm("" : "+v"(e));
  return e;
}

// Memory that was never written may hold finite params whose numbers leave float16; as infinities such values would make NaNs of
// the zeros that weigh what a row does not see. Hence values past float16's largest number count as it.
// Sets the wave's mode in which float16 results do so by themselves. The matrix units take infinities and NaN among their float16
// operands as numbers, too, then: a NaN has to come by float32.
__device__ __forceinline__ void saturate_float16(bool on) {
  constexpr int kMode = 1, kBit = 23;  // MODE.FP16_OVFL, one bit
  __builtin_amdgcn_s_setreg(kMode | kBit << 6, on);
}

// Codes of bits 0 - 3 and 4 - 7 of both halves of u as offset + code * step, one rounding. A code under the exponent of
// 1024 is 1024 + code (bits 0 - 3) or 1024 + 16 code (bits 4 - 7), from which the code itself comes back exactly.
__device__ __forceinline__ h2 low_codes(uint32_t u, uint32_t e, h2 step, h2 offset) {
  const h2 c = as_h2((u & 0x000F000Fu) | e) + h2{(_Float16)-1024.f, (_Float16)-1024.f};
  return __builtin_elementwise_fma(c, step, offset);
}
__device__ __forceinline__ h2 high_codes(uint32_t u, uint32_t e, h2 step, h2 offset) {
  const h2 c = __builtin_elementwise_fma(as_h2((u & 0x00F000F0u) | e), h2{(_Float16)0.0625f, (_Float16)0.0625f},
                                         h2{(_Float16)-64.f, (_Float16)-64.f});
  return __builtin_elementwise_fma(c, step, offset);
}

// Eight consecutive channels of one token: a word of codes, in the order of channels 0, 4, 1, 5, 2, 6, 3, 7 (the queries' operand is
// brought into the same order).
__device__ __forceinline__ h8 token_codes(uint32_t w, uint32_t e, h2 step, h2 offset) {
  const uint32_t v = w >> 8;
  const h2 a = low_codes(w, e, step, offset), b = high_codes(w, e, step, offset);
  const h2 c = low_codes(v, e, step, offset), d = high_codes(v, e, step, offset);
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// bfloat16 queries reach past float16: each row is brought to a largest magnitude in [1, 2) by a power of two (`up`), which the
// scale of its scores takes back (`down`). What then lies below float16's normal numbers is below 2^-14 of the row's
// largest. Negative scales are moved into the queries, so that the largest product is the largest score. FIT:
// for such queries, and where they are multiplied by 16.
template <bool FIT>
__device__ __forceinline__ void query_range(float largest, float scale, float& up, float& down) {
  up = down = 1.f;
  if constexpr (FIT) {
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

// What a row's numerators are taken from: a score x (scale not yet applied) has the numerator 2^((x - base) * scale - top). base is 0,
// and top lies kRoom below the largest score's exponent and moves when a numerator would pass 2^kMost, as long as top is below kWide.
// Past it, where the reference's own rounding would count, base is the largest score and top -kRoom: exponents are
// differences of scores then. Bases wait in LDS, and a wave that has one takes the branch that moves references in every step; the
// others have a comparison more (drafts and heads of 256 2 % slower, single tokens and the long prompt alike).
// Where a split's references are kept, NaN in the place of top says that there is a base.
struct Reference {
  float top, base;
};
constexpr float kRoom = 7.f, kMost = 15.f, kWide = 0x1p20f;
__device__ __forceinline__ Reference reference(float top, float base) {
  return __builtin_isnan(top) ? Reference{-kRoom, base} : Reference{top, 0.f};
}

// A scale by which scores, below 2^41 and multiples of 2^-48 (of float16 numbers' products), stay above kNothing. Past it differences of scores
// are 0 or decide alone, as they would anyway.
__device__ __forceinline__ float scale_in_range(float scale) { return fminf(scale, 0x1p86f); }

// The base-2 exponent of numerators of reference a in those of reference b.
__device__ __forceinline__ float between(const Reference& a, const Reference& b, float scale) {
  return fmaf(a.base - b.base, scale, a.top - b.top);
}

// A row has met a score `most` (-infinity: none): moves its reference where it has to be, and gives the factor of the numerators so
// far.
__device__ __forceinline__ float move_reference(Reference& r, float most, float scale) {
  const bool up = (most - r.base) * scale - kRoom > r.top, wide = fabsf(most * scale) > kWide;
  const Reference to = {up ? (wide ? -kRoom : most * scale - kRoom) : r.top, up ? (wide ? most : 0.f) : r.base};
  const float f = __builtin_amdgcn_exp2f(between(r, to, scale));
  r = to;
  return f;
}

// Lane % 16, worked out where it stands: kept from outside a branch, it would cost a register all along.
__device__ __forceinline__ int lane16_here() {
  int zero = 0;
  asm volatile("" : "+v"(zero));
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero)) % 16;
}

// log of a row's sum of exponentials. scale: as it is, but finite
__device__ __forceinline__ float log_of_sum(const Reference& r, float scale, float total) {
  return total == 0.f ? -__builtin_inff() : fmaf(r.base, scale, r.top + __log2f(total)) * kLn2;
}

// The lane, which the compiler takes as new each time: what hangs on it is not kept in registers around a loop over pieces.
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// Two float16 numbers, rounded to the nearest.
__device__ __forceinline__ h2 to_h2(float x, float y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f32x2{x, y}), h2);
}

// The same eight channels as they stand under the exponent: 1024 + code (channels 0, 4, 2, 6), 1024 + 16 code (1, 5, 3, 7).
__device__ __forceinline__ h8 raw_codes(uint32_t w, uint32_t e) {
  const uint32_t v = w >> 8;
  const h2 a = as_h2((w & 0x000F000Fu) | e), b = as_h2((w & 0x00F000F0u) | e);
  const h2 c = as_h2((v & 0x000F000Fu) | e), d = as_h2((v & 0x00F000F0u) | e);
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
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
