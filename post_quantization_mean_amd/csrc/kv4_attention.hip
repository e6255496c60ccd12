// Attention over the 4-bit cache: few rows of a key head (single tokens, drafts), and the joining of split sequences.
//
// A row is one query head of one new token; the rows of a key head (its group of query heads, times the new tokens) share the
// key head's cached tokens, so they go through the matrix units together, 16 rows a tile. Bound by reading the cache: a
// token's keys and values of a head of 128 are 136 bytes.
//
// A block of four waves takes a run of cached tokens, its waves 32 tokens in turn, with v_mfma_f32_16x16x32_f16:
//   S^T = K Q^T   lane (g, m) = (lane / 16, lane % 16): A holds channels g * HD/4 .. of token m, straight from the cache (16
//                 bytes for HD = 128), B the same channels of row m; D: tokens 4 g .. 4 g + 3 of row m.
//   O^T = V^T P^T B holds the numerators of row m for tokens 4 g .. 4 g + 3 of two tiles of 16 tokens: what the first product
//                 left in the lane. A holds the same tokens for channels m * HD/16 .. (4 bytes of each token for HD = 128);
//                 two tokens' bytes beside each other are pairs of the contraction, channel by channel.
// So no operand crosses a lane, and nothing goes through LDS until the waves join. Keys stay codes (0.6 vector operations each):
// step and offset meet the scores, in float32. (Turned into float16 numbers first, as the values are, a float16 draft over 2048
// tokens of heads of 256 was off by 3.3e-4 of its outputs' magnitude instead of 2.6e-4, 2.1e-4 of it the outputs' own rounding,
// and the batch below took 91 us.) Values become float16 numbers offset + code * step with one rounding (2^-11 of the number at
// most; 1.7 operations a code); numerators are rounded to the nearest.
//
// 64 sequences of up to 8192 tokens (ragged), 64 heads on 8 of 128: 84 us (3.6 TB/s), about 10 of them the shares' beginnings and
// ends and 5 the joining kernel; as tiles of whole sequences, the longest ones' blocks alone at the end, 148 us. One token over
// 131071: 41 us (3.5 TB/s).

#include <type_traits>

#include "kv4_device.h"

namespace awq {
namespace {

constexpr int kWaves = 4;
constexpr int kStep = 32;  // tokens of a wave at a time

// What a wave loads for 32 tokens.
template <int HD>
struct Stage {
  static constexpr int KW = HD / 32;   // words of codes of a token in a lane (keys)
  static constexpr int VB = HD / 32;   // bytes of codes of a token in a lane (values)
  static constexpr int G = (HD + 127) / 128;
  uint32_t k[2][KW], kp[2][G];
  uint32_t v[8][(VB + 3) / 4], vp[8];
  bool there[2];
};

template <int HD>
struct Loader {
  const uint8_t* codes;      // the key head's keys in page 0
  const uint32_t* params;
  int64_t page_codes, page_params, v_codes, v_params;  // from keys to values
  const int32_t* table;
  int page_log2, page_mask, row_bytes, lane_pages, lane;
  uint32_t n_pages;
  int group_words;
  // A lane's offsets, unsigned: added to an address that the wave shares, they need no registers of 64 bits.
  uint32_t k_at[(HD + 127) / 128], kp_at, v_at, vp_at;  // bytes of codes, words of params

  // The pages of the wave's next 64 tiles of 16 tokens: lane i has tile i's (-1 past the end).
  __device__ __forceinline__ void pages(int t0, int stride, int end) {
    const int t = t0 + (lane >> 1) * stride + (lane & 1) * 16;
    lane_pages = t < end ? table[t >> page_log2] : -1;
  }
  __device__ __forceinline__ void load(Stage<HD>& s, int i, int t0) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int id = __builtin_amdgcn_readlane(lane_pages, 2 * i + h);
      s.there[h] = (uint32_t)id < n_pages;
      const int64_t page = s.there[h] ? id : 0;
      const int at = (t0 + 16 * h) & page_mask;
      const uint8_t* kc = codes + page * page_codes + at * row_bytes;
      const uint32_t* kp = params + page * page_params + at;
      const uint8_t* vc = kc + v_codes;
      const uint32_t* vp = kp + v_params;
      if constexpr (HD == 64) {
        const uint2 u = *reinterpret_cast<const uint2*>(kc + k_at[0]);
        s.k[h][0] = u.x, s.k[h][1] = u.y;
      } else {
#pragma unroll
        for (int c = 0; c < HD / 128; ++c) {
          const uint4 u = *reinterpret_cast<const uint4*>(kc + k_at[c]);
          s.k[h][4 * c] = u.x, s.k[h][4 * c + 1] = u.y, s.k[h][4 * c + 2] = u.z, s.k[h][4 * c + 3] = u.w;
        }
      }
#pragma unroll
      for (int c = 0; c < Stage<HD>::G; ++c) s.kp[h][c] = (kp + c * group_words)[kp_at];
      const uint4 p = *reinterpret_cast<const uint4*>(vp + vp_at);
      s.vp[4 * h] = p.x, s.vp[4 * h + 1] = p.y, s.vp[4 * h + 2] = p.z, s.vp[4 * h + 3] = p.w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* row = vc + j * row_bytes + v_at;
        if constexpr (HD == 64) s.v[4 * h + j][0] = *reinterpret_cast<const uint16_t*>(row);
        else if constexpr (HD == 128) s.v[4 * h + j][0] = *reinterpret_cast<const uint32_t*>(row);
        else {
          const uint2 u = *reinterpret_cast<const uint2*>(row);
          s.v[4 * h + j][0] = u.x, s.v[4 * h + j][1] = u.y;
        }
      }
    }
  }
};

// First channel of step s of a lane's queries and keys: those of g HD/4 .. in turn, of heads past 128 first the first 128's.
template <int HD>
__device__ __forceinline__ int step_channel(int g, int s) {
  return HD > 128 ? s / 4 * 128 + g * 32 + s % 4 * 8 : g * (HD / 4) + s * 8;
}

// A lane's part of the queries: rows m of NR tiles, channels step_channel .. . Zeros past the last row and channel.
template <int HD, int NR, typename T>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const RowTile& t, int head, int lane, uint4 (&raw)[NR][HD / 32]) {
  const int g = lane >> 4, m = lane & 15;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = min(t.row0 + 16 * n + m, t.rows - 1);
    const int token = a.by_group.of(r), of = r - token * a.group;
    const T* row = (const T*)a.q.p + (int64_t)(t.token0 + token) * a.q.ld + (int64_t)(head * a.group + of) * a.q.ld_head;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) {
      const int c = step_channel<HD>(g, s);
      raw[n][s] = __builtin_bit_cast(uint4, *reinterpret_cast<const Chunk<T>*>(row + (c < a.c.head_dim ? c : 0)));
    }
  }
}

// Their operand for raw_codes, and what their scores are multiplied by (times log2(e)): channels in the order 0, 4, 1, 5, 2, 6,
// 3, 7, the even ones times 16. sum: of a row's queries in each group; less: what the exponents of raw_codes add to their product,
// with the sign turned, from which the product's accumulator starts. A row with a NaN or an infinity has NaN for every score; its
// scale stays a number, so that where it sees nothing it is nothing.
template <int HD, int NR, typename T>
__device__ __forceinline__ void convert_queries(const AttnArgs& a, const RowTile& t, int lane, uint4 (&raw)[NR][HD / 32],
                                                h8 (&q)[NR][HD / 32], float (&scale)[NR], float (&sum)[NR][Stage<HD>::G],
                                                float (&less)[NR][Stage<HD>::G]) {
  const int g = lane >> 4, m = lane & 15;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const bool there = t.row0 + 16 * n + m < t.rows;
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) {
      if (!there || step_channel<HD>(g, s) >= a.c.head_dim) raw[n][s] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(raw_f32<T>(raw[n][s], k)));
    }
    float up, down;
    top = max_over_rows(top);
    query_range<true>(top, a.scale, up, down);
    if (top == __builtin_inff()) up = __builtin_nanf("");  // (an infinity would be saturated)
    scale[n] = fminf(fmaxf(fabsf(a.scale) * (down * 0.0625f), 0x1p-126f), kLargestFloat);
    float even[Stage<HD>::G] = {}, odd[Stage<HD>::G] = {};  // sums of what the operand holds
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) {
      // read again: the numbers of the first pass would not fit the registers
      asm volatile("" : "+v"(raw[n][s].x), "+v"(raw[n][s].y), "+v"(raw[n][s].z), "+v"(raw[n][s].w));
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool of16 = order[k] & 1;
        const _Float16 x = (_Float16)(raw_f32<T>(raw[n][s], order[k]) * up * (of16 ? 1.f : 16.f));
        q[n][s][k] = x;
        if (of16) odd[s / 4 % Stage<HD>::G] += (float)x;
        else even[s / 4 % Stage<HD>::G] += (float)x;
      }
    }
#pragma unroll
    for (int c = 0; c < Stage<HD>::G; ++c) {
      even[c] = sum_over_rows(even[c]);
      odd[c] = sum_over_rows(odd[c]);
      sum[n][c] = fmaf(16.f, odd[c], even[c]);
      less[n][c] = -1024.f * (even[c] + odd[c]);
    }
  }
}

// Waves of a SIMD: what the registers of a variant let live. (Heads of 128 with three: the token over 131071 46 us instead of 41,
// since the work is split over half as many blocks again.)
constexpr int live_waves(int hd_nr) { return hd_nr <= 64 ? 3 : hd_nr <= 256 ? 2 : 1; }

template <int HD, int NR, bool BF16, bool SPLIT>
__global__ __launch_bounds__(kWaves * 64, live_waves(HD * NR)) void rows_kernel(AttnArgs a) {
  constexpr int CT = HD / 16;  // channel tiles; a lane's channels are m * CT .. and, of the result, (4 g + i) * CT ..
  constexpr int kPitch = HD + 4;
  __shared__ __align__(16) float lds_o[kWaves][16][kPitch];
  __shared__ float lds_m[kWaves][16 * NR], lds_l[kWaves][16 * NR];
  __shared__ float lds_base[kWaves][16 * NR], lds_scale[16 * NR];
  __shared__ int lds_prefix[SPLIT ? kPrefixInts : 1];
  saturate_float16(true);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for_pieces<SPLIT>(a, lds_prefix, [&](const RowTile& t, int head, int begin, int end, int part) {
  const int lane = fresh_lane(), g = lane >> 4, m = lane & 15;
  using T = typename std::conditional<BF16, Bf16, F16>::type;
  uint4 raw[NR][HD / 32];
  load_queries<HD, NR, T>(a, t, head, lane, raw);
  int lo[NR], hi[NR], all_lo, all_hi, unused;
#pragma unroll
  for (int n = 0; n < NR; ++n) row_range(a, t, t.row0 + 16 * n + m, lo[n], hi[n]);
  // tokens in [all_lo, all_hi) are seen by every row of the tile
  row_range(a, t, t.row0, unused, all_hi);
  row_range(a, t, min(t.row0 + 16 * NR, t.rows) - 1, all_lo, unused);

  Loader<HD> in;
  in.lane = lane;
  const int page = 1 << a.c.page_log2;
  in.row_bytes = a.c.head_dim / 2;
  in.codes = a.c.codes + (int64_t)head * page * in.row_bytes;
  in.params = a.c.params + (int64_t)head * a.c.n_groups * page;
  in.page_codes = a.c.page_codes;
  in.page_params = a.c.page_params;
  in.v_codes = (int64_t)a.c.n_kv * page * in.row_bytes;
  in.v_params = (int64_t)a.c.n_kv * a.c.n_groups * page;
  in.table = a.table + (int64_t)t.seq * a.ld_table;
  in.page_log2 = a.c.page_log2;
  in.page_mask = page - 1;
  in.n_pages = (uint32_t)a.c.n_pages;
  // channels past the head's last one read others of the row: their queries are zeros, their results are not stored
#pragma unroll
  for (int c = 0; c < (HD + 127) / 128; ++c) {
    const int at = g * (HD > 128 ? 16 : HD / 8) + (HD > 128 ? 64 : 16) * c;
    in.k_at[c] = m * in.row_bytes + (at < in.row_bytes ? at : 0);
  }
  in.group_words = page;
  in.kp_at = m;
  in.v_at = 4 * g * in.row_bytes + (m * (HD / 32) < in.row_bytes ? m * (HD / 32) : 0);
  in.vp_at = min(m * CT / 128, a.c.n_groups - 1) * page + 4 * g;

  constexpr int kStride = kWaves * kStep;
  // Float16 rows: a numerator is two float16 numbers, what the first one's rounding leaves is the second. The outputs' own rounding
  // is no larger than the numerators' (a float16 draft over 2048 tokens of heads of 256: off by 2.6e-4 of its outputs' magnitude
  // with one, 2.3e-4 with two, 2.1e-4 of it their own rounding). The second product costs 0 - 11 % (one token over 131071 40.5 ->
  // 42.7 us, 32 drafts of 4 over 6000 76 -> 84). Bfloat16 rows do without it: in bfloat16 their outputs' own rounding is eight times as
  // large; float32 outputs of bfloat16 queries have the numerators' 2^-11 each, an error of the size of the values' own rounding.
  constexpr bool kRest = !BF16;
  // Steps whose codes are in registers: the one in use and those on their way. (Three: the cases above 92 and 43 us, 64
  // sequences of 8000 tokens of heads of 64 97 instead of 86.)
  constexpr int D = 2;
  const int first = begin + wave * kStep;
  const int steps = first < end ? (end - first + kStride - 1) / kStride : 0;
  Stage<HD> stage[D];
#pragma unroll
  for (int k = 0; k < D - 1; ++k)
    if (k < steps) {
      if (k == 0) in.pages(first, kStride, end);
      in.load(stage[k], k, first + k * kStride);
    }
  constexpr int G = Stage<HD>::G;
  h8 q[NR][HD / 32];
  float scale[NR], q_sum[NR][G], q_less[NR][G];
  convert_queries<HD, NR, T>(a, t, lane, raw, q, scale, q_sum, q_less);

  f32x4 o[NR][CT];
  float top[NR], sum[NR];  // the reference of a row's numerators, and their sum in this lane
  uint64_t based = 0;  // lanes whose reference has a base
  uint32_t poisoned[NR];  // groups (bits) whose values a row has seen a NaN in
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    top[n] = kNothing;
    sum[n] = 0.f;
    lds_base[wave][16 * n + m] = 0.f;
    lds_scale[16 * n + m] = scale[n];  // (the same of every wave)
    scale[n] = scale_in_range(scale[n]);
    poisoned[n] = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) o[n][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // The queries of heads past 128 wait in LDS, in the wave's own part of what the waves join in: the registers hold a second
  // step's codes instead.
  constexpr bool kAside = HD > 128;
  static_assert(NR * HD * 2 <= kPitch * 4);
  uint32_t aside = (uint32_t)lane;
  if constexpr (kAside) {
    h8* to = reinterpret_cast<h8*>(&lds_o[wave][0][0]);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) to[(n * (HD / 32) + i) * 64 + lane] = q[n][i];
  }
  const auto query = [&](int n, int i) {
    if constexpr (kAside) return reinterpret_cast<const h8*>(&lds_o[wave][0][0])[(n * (HD / 32) + i) * 64 + aside];
    else return q[n][i];
  };

  const uint32_t e = code_exponent();
  // 32 tokens from t0 on
  const auto take = [&](Stage<HD>& now, int t0) {
    // ---- scores: step * (q . codes) + offset * (sum of q), the products of codes without rounding
    float x[NR][8];
    if constexpr (kAside) asm volatile("" : "+v"(aside));  // read in every step
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        f32x4 s[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n] = f32x4{q_less[n][c], q_less[n][c], q_less[n][c], q_less[n][c]};
#pragma unroll
        for (int i = 4 * c; i < min(4 * c + 4, HD / 32); ++i) {
          const h8 k = raw_codes(now.k[h][i], e);
#pragma unroll
          for (int n = 0; n < NR; ++n) s[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, query(n, i), s[n], 0, 0, 0);
        }
        // lane m has token m's params; the scores are those of tokens 4 g .. 4 g + 3
        const int w = (int)finite_or_nan(now.kp[h][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const h2 p = as_h2((uint32_t)__builtin_amdgcn_ds_bpermute((4 * g + j) * 4, w));
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float rest = c ? fmaf((float)p.y, q_sum[n][c], x[n][4 * h + j]) : (float)p.y * q_sum[n][c];
            x[n][4 * h + j] = fmaf((float)p.x, s[n][j], rest);
          }
        }
        if constexpr (HD > 128) __builtin_amdgcn_sched_barrier(0);
      }
    }
    const bool whole = t0 >= all_lo && t0 + kStep <= all_hi && t0 + kStep <= end && now.there[0] && now.there[1];
    // ---- values that are not finite: out of the products, noted for the rows that see them
    h2 zeros = as_h2(0);  // stays so where all of them are finite
#pragma unroll
    for (int j = 0; j < 8; ++j) zeros = __builtin_elementwise_fma(as_h2(now.vp[j]), as_h2(0), zeros);
    if (rare(__any((as_u32(zeros) & 0x7FFF7FFFu) != 0))) {
      int mine = 0;  // which of the lane's tokens, in the group of the lane's channels
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (not_finite(now.vp[j])) mine |= 1 << j, now.vp[j] = 0;
#pragma unroll
      for (int c = 0; c < (HD + 127) / 128; ++c) {
        const int in_group = HD > 128 ? __shfl(mine, (lane & 48) + 8 * c) : mine;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = t0 + 16 * (j / 4) + 4 * g + j % 4;
          const bool there = (in_group >> j & 1) && now.there[j / 4];
#pragma unroll
          for (int n = 0; n < NR; ++n)
            if (there && at >= lo[n] && at < min(hi[n], end)) poisoned[n] |= 1u << c;
        }
      }
    }
    // ---- numerators
    h8 p[NR], rest[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float most = -__builtin_inff();
      if (rare(!whole)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = t0 + 16 * h + 4 * g + j;
            if (at < lo[n] || at >= min(hi[n], end) || !now.there[h]) x[n][4 * h + j] = -__builtin_inff();
          }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, x[n][j]);
      // The numerators are powers from a reference that is set 2^7 below the largest score and moves only when they would
      // pass 2^15: float16 holds them, down to 2^-31 of the largest.
      if (rare((based | __ballot(most * scale[n] > top[n] + kMost)) != 0)) {
        float& base = lds_base[wave][16 * n + lane16_here()];
        Reference ref = {top[n], base};
        const float f = move_reference(ref, max_over_rows(most), scale[n]);
        top[n] = ref.top;
        sum[n] *= f;
#pragma unroll
        for (int c = 0; c < CT; ++c) o[n][c] *= f;
        base = ref.base;
        based |= __ballot(ref.base != 0.f);
        if (based) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[n][j] -= ref.base;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float x0 = __builtin_amdgcn_exp2f(fmaf(x[n][j], scale[n], -top[n]));
        const float x1 = __builtin_amdgcn_exp2f(fmaf(x[n][j + 1], scale[n], -top[n]));
        const h2 pair = to_h2(x0, x1);
        if constexpr (kRest) {
          const h2 less = to_h2(x0 - (float)pair.x, x1 - (float)pair.y);
          rest[n][j] = less.x;
          rest[n][j + 1] = less.y;
          sum[n] += x0 + x1;
        } else {  // summed as rounded, so that the weights add up to one
          sum[n] = __builtin_amdgcn_fdot2(pair, h2{(_Float16)1.f, (_Float16)1.f}, sum[n], false);
        }
        p[n][j] = pair.x;
        p[n][j + 1] = pair.y;
      }
    }
    // ---- their product with the values
    h2 step[4], offset[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      step[j] = as_h2(__builtin_amdgcn_perm(now.vp[2 * j + 1], now.vp[2 * j], 0x05040100));
      offset[j] = as_h2(__builtin_amdgcn_perm(now.vp[2 * j + 1], now.vp[2 * j], 0x07060302));
    }
#pragma unroll
    for (int b = 0; b < (CT + 3) / 4; ++b) {  // two bytes of a token: four channels
      h2 v[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = __builtin_amdgcn_perm(now.v[2 * j + 1][b / 2], now.v[2 * j][b / 2], b & 1 ? 0x07060302 : 0x05040100);
        v[0][j] = low_codes(u, e, step[j], offset[j]);
        v[1][j] = high_codes(u, e, step[j], offset[j]);
        v[2][j] = low_codes(u >> 8, e, step[j], offset[j]);
        v[3][j] = high_codes(u >> 8, e, step[j], offset[j]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const h8 f = {v[c][0].x, v[c][0].y, v[c][1].x, v[c][1].y, v[c][2].x, v[c][2].y, v[c][3].x, v[c][3].y};
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          if constexpr (kRest) o[n][4 * b + c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, rest[n], o[n][4 * b + c], 0, 0, 0);
          o[n][4 * b + c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, p[n], o[n][4 * b + c], 0, 0, 0);
        }
      }
    }
  };
  for (int i = 0; i < steps; i += D) {
#pragma unroll
    for (int k = 0; k < D; ++k) {
      if (i + k >= steps) break;
      const int ahead = i + k + D - 1;
      if (ahead < steps) {
        if ((ahead & 31) == 0) in.pages(first + ahead * kStride, kStride, end);
        in.load(stage[(k + D - 1) % D], ahead & 31, first + ahead * kStride);
      }
      take(stage[k], first + (i + k) * kStride);
    }
  }

  // ---- the waves join
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    sum[n] = sum_over_rows(sum[n]);
    poisoned[n] = or_over_rows(poisoned[n]);
    if (g == 0) {
      lds_m[wave][16 * n + m] = top[n];
      lds_l[wave][16 * n + m] = sum[n];
    }
  }
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    if (n) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* to = &lds_o[wave][m][(4 * g + i) * CT];
      const float nan = (poisoned[n] >> ((4 * g + i) * CT / 128)) & 1 ? __builtin_nanf("") : 0.f;
#pragma unroll
      for (int c = 0; c < CT; ++c) to[c] = o[n][c][i] + nan;
    }
    __syncthreads();
    constexpr int kRowThreads = kWaves * 64 / 16;  // threads of a row
    const int row = (int)threadIdx.x / kRowThreads, r = t.row0 + 16 * n + row;
    if (r < t.rows) {
      float most = kNothing, base = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        most = fmaxf(most, lds_m[w][16 * n + row]);
        base = fmaxf(base, fabsf(lds_base[w][16 * n + row]));
      }
      float f[kWaves], total = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) f[w] = __builtin_amdgcn_exp2f(lds_m[w][16 * n + row] - most);
      Reference ref = {most, 0.f};
      float scale_of = 0.f;  // as it is
      if (rare(base != 0.f)) {
        scale_of = lds_scale[16 * n + row];
        const float in_range = scale_in_range(scale_of);
        const auto of_wave = [&](int w) { return Reference{lds_m[w][16 * n + row], lds_base[w][16 * n + row]}; };
        ref = of_wave(0);
#pragma unroll 1
        for (int w = 1; w < kWaves; ++w)
          if (between(of_wave(w), ref, in_range) > 0.f) ref = of_wave(w);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) f[w] = __builtin_amdgcn_exp2f(between(of_wave(w), ref, in_range));
      }
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total = fmaf(f[w], lds_l[w][16 * n + row], total);
      const int token = a.by_group.of(r), of = head * a.group + (r - token * a.group);
      const int64_t at = (int64_t)(t.token0 + token) * a.n_heads + of;
      const bool final = part < 0;
      const int64_t slot = (int64_t)part * a.tile_rows + 16 * n + row;
      const float inv = final ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
      if ((int)threadIdx.x % kRowThreads == 0) {
        if (!final) {
          const bool based = ref.base != 0.f;
          reinterpret_cast<float2*>(a.part_ml)[slot] = make_float2(based ? __builtin_nanf("") : ref.top, total);
          if (based) reinterpret_cast<float2*>(a.part_base)[slot] = make_float2(ref.base, scale_of);
        } else if (a.lse) {
          a.lse[at] = log_of_sum(ref, scale_of, total);
        }
      }
      for (int c = (int)threadIdx.x % kRowThreads * 4; c < a.c.head_dim; c += kRowThreads * 4) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = fmaf(f[w], lds_o[w][row][c + k], y[k]);
        if (!final) {
          *reinterpret_cast<f32x4*>(a.part_o + slot * a.c.head_dim + c) = f32x4{y[0], y[1], y[2], y[3]};
          continue;
        }
        const int64_t to = (int64_t)(t.token0 + token) * a.out.ld + (int64_t)of * a.out.ld_head + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] *= inv;
        store4<BF16>(a, to, y);
      }
    }
  }  });
}

// Joins the parts of rows whose cached tokens several blocks have taken. Block (tile, key head, R rows of the tile). Threads:
// 8 / R parts of a row at once, 4 channels each (twice: of heads past 128). Bound by latency: the loads of kJoin parts a
// thread go out together, the first ones before the parts' largest reference is known.
constexpr int kJoin = 4;
template <bool BF16, int H, int R>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a) {
  constexpr int G = 8 / R;  // groups of 32 threads for a row
  __shared__ float lds[8][128 * H + 4];
  __shared__ float lds_l[8];
  const int tile = (int)blockIdx.x, head = (int)blockIdx.y;
  const int before = a.prefix[tile], units = a.prefix[tile + 1] - before;
  const Split split(a.prefix[a.n_tiles] * a.c.n_kv, a.n_blocks);
  if (units == 0) return;
  const int first_unit = before * a.c.n_kv + head * units;
  const int first_block = split.of(first_unit), parts = split.of(first_unit + units - 1) - first_block + 1;
  if (parts <= 1) return;
  const RowTile t = row_tile(a, tile);
  const int group = (int)threadIdx.x / 32, lane = (int)threadIdx.x % 32;
  const int row = (int)blockIdx.z * R + group / G, mine = group % G;
  const int r = t.row0 + row;
  const bool there = row < a.tile_rows && r < t.rows;  // (as every thread of a row)
  const int first_part = 2 * first_block + (split.begin(first_block) == first_unit ? 0 : 1);
  const auto part = [&](int i) { return (int64_t)(i == 0 ? first_part : 2 * (first_block + i)) * a.tile_rows + (there ? row : 0); };
  f32x4 u[kJoin][H];
  float2 w[kJoin];
  const auto load = [&](int first) {
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const int64_t i = part(min(first + G * k, parts - 1));
      w[k] = ((const float2*)a.part_ml)[i];
#pragma unroll
      for (int h = 0; h < H; ++h)
        u[k][h] = *reinterpret_cast<const f32x4*>(a.part_o + i * a.c.head_dim + (4 * lane + 128 * h < a.c.head_dim ? 4 * lane + 128 * h : 0));
    }
  };
  load(mine);
  float most = kNothing, nan = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float top = ((const float2*)a.part_ml)[part(i)].x;
    most = fmaxf(most, top);
    nan = fmaf(top, 0.f, nan);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
  Reference ref = {most, 0.f};
  float scale = 0.f;
  const bool based = __any(nan != 0.f);
  const auto of_part = [&](int i, float top) {
    const bool here = __builtin_isnan(top);
    const float2 b = here ? ((const float2*)a.part_base)[part(i)] : make_float2(0.f, 0.f);
    if (here) scale = b.y;  // (of the row: the same in every part)
    return reference(top, b.x);
  };
  if (rare(based)) {
    for (int i = 0; i < parts; ++i) of_part(i, ((const float2*)a.part_ml)[part(i)].x);
    ref = {kNothing, 0.f};
    for (int i = 0; i < parts; ++i) {
      const Reference of = of_part(i, ((const float2*)a.part_ml)[part(i)].x);
      if (between(of, ref, scale_in_range(scale)) > 0.f) ref = of;
    }
  }
  float y[H][4] = {}, total = 0.f;
  for (int first = mine; first < parts; first += G * kJoin) {
    if (first != mine) load(first);
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      if (first + G * k >= parts) break;
      float f = __builtin_amdgcn_exp2f(w[k].x - most);
      if (rare(based)) f = __builtin_amdgcn_exp2f(between(of_part(first + G * k, w[k].x), ref, scale_in_range(scale)));
      total = fmaf(f, w[k].y, total);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) y[h][c] = fmaf(f, u[k][h][c], y[h][c]);
    }
  }
  if constexpr (G > 1) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) lds[group][128 * h + 4 * lane + c] = y[h][c];
    if (lane == 0) lds_l[group] = total;
    __syncthreads();
    if (mine) return;
    total = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) total += lds_l[group + i];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        y[h][c] = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i) y[h][c] += lds[group + i][128 * h + 4 * lane + c];
      }
  }
  if (!there) return;
  const int token = a.by_group.of(r), of = head * a.group + (r - token * a.group);
  if (lane == 0 && a.lse)
    a.lse[(int64_t)(t.token0 + token) * a.n_heads + of] = log_of_sum(ref, scale, total);
  const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const int c = 4 * lane + 128 * h;
    if (c >= a.c.head_dim) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[h][k] *= inv;
    store4<BF16>(a, (int64_t)(t.token0 + token) * a.out.ld + (int64_t)of * a.out.ld_head + c, y[h]);
  }
}

template <int HD, int NR, bool BF16>
void launch_rows(const AttnArgs& a, hipStream_t stream) {
  if (a.n_blocks) rows_kernel<HD, NR, BF16, true><<<attention_grid(a), kWaves * 64, 0, stream>>>(a);
  else rows_kernel<HD, NR, BF16, false><<<attention_grid(a), kWaves * 64, 0, stream>>>(a);
}

template <bool BF16>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  const bool one = a.tile_rows == 16;
  if (a.c.head_dim <= 64) one ? launch_rows<64, 1, BF16>(a, stream) : launch_rows<64, 2, BF16>(a, stream);
  else if (a.c.head_dim <= 128) one ? launch_rows<128, 1, BF16>(a, stream) : launch_rows<128, 2, BF16>(a, stream);
  else one ? launch_rows<256, 1, BF16>(a, stream) : launch_rows<256, 2, BF16>(a, stream);
  return hipGetLastError();
}

template <bool BF16, int R>
void launch_join_rows(const AttnArgs& a, int rows, hipStream_t stream) {
  const dim3 grid((unsigned)a.n_tiles, (unsigned)a.c.n_kv, (unsigned)((rows + R - 1) / R));
  if (a.c.head_dim <= 128) join_kernel<BF16, 1, R><<<grid, 256, 0, stream>>>(a);
  else join_kernel<BF16, 2, R><<<grid, 256, 0, stream>>>(a);
}

template <bool BF16>
hipError_t launch_join(const AttnArgs& a, hipStream_t stream) {
  const int rows = a.q_offsets ? a.tile_rows : min(a.tile_rows, a.each * a.group);
  // many parts of few rows: all of a block's threads for one row; few parts of many: 32 of them
  if ((int64_t)a.n_tiles * a.c.n_kv * 8 <= a.n_blocks) launch_join_rows<BF16, 1>(a, rows, stream);
  else launch_join_rows<BF16, 8>(a, rows, stream);
  return hipGetLastError();
}

}  // namespace

// Rows of a sequence and key head up to which a block of the kernel above takes 32 of them; past that the kernel for prompts
// (32 sequences of 32 rows over 6000 tokens: 76 us, as prompts 162; 16 of 128 rows over 9000: 157 us either way).
constexpr int kFewRows = 64;

size_t prefix_bytes(int n_tiles) { return ((size_t)(n_tiles + 1) * sizeof(int) + 255) / 256 * 256; }

size_t plan_attention(AttnArgs* a, bool ragged) {
  const int64_t rows_each = (a->n_tokens + a->n_seqs - 1) / a->n_seqs * a->group;
  a->tile_rows = rows_each <= 16 ? 16 : rows_each <= kFewRows ? 32 : prompt_rows(a->c.head_dim);
  a->tile_log2 = __builtin_ctz((unsigned)a->tile_rows);
  a->by_group = Divisor((uint32_t)a->group);
  a->by_kv = Divisor((uint32_t)a->c.n_kv);
  a->by_tiles = Divisor((uint32_t)((rows_each + a->tile_rows - 1) / a->tile_rows));
  if (ragged) a->n_tiles = (int)(a->n_tokens * a->group / a->tile_rows + a->n_seqs);
  else a->n_tiles = (int)(a->n_seqs * ((rows_each + a->tile_rows - 1) / a->tile_rows));
  int64_t span = a->max_kv;
  if (a->window && a->causal) span = min(span, (int64_t)a->window + a->tile_rows / a->group + kAlign);
  const int hd = a->c.head_dim <= 64 ? 64 : a->c.head_dim <= 128 ? 128 : 256;
  const int64_t pairs = (int64_t)a->n_tiles * a->c.n_kv, units = pairs * ((span + kUnit - 1) / kUnit);
  // Blocks of a split: as many as run at once. It costs some microseconds in each block and a second launch: not for short
  // spans, many tiles, or tiles of prompts that fill the compute units without it (9 prompts of up to 1500 tokens, 776 tiles
  // and key heads: 133 us at the time, split 291; 128 of 128 rows over 9000 tokens: 218 us, split 160).
  const int64_t at_once = 256 * (a->tile_rows > 32 ? 1 : live_waves(hd * a->tile_rows / 16));
  a->n_blocks = (int)min(at_once, units / kLeastUnits);
  if (a->n_tiles > kMostTiles || pairs >= at_once * (a->tile_rows > 32 ? 1 : 4) || span <= kLeastUnits * kUnit) a->n_blocks = 0;
  if (a->n_blocks == 0) return 0;
  return prefix_bytes(a->n_tiles) + (size_t)2 * a->n_blocks * a->tile_rows * (a->c.head_dim + 4) * sizeof(float);
}

void place_workspace(AttnArgs* a, void* workspace) {
  a->prefix = (int*)workspace;
  a->part_o = (float*)((char*)workspace + prefix_bytes(a->n_tiles));
  const size_t rows = (size_t)2 * a->n_blocks * a->tile_rows;
  a->part_ml = a->part_o + rows * a->c.head_dim;
  a->part_base = a->part_ml + 2 * rows;
}

hipError_t launch_kv4_attention(const AttnArgs& a, bool bf16, hipStream_t stream) {
  hipError_t e = a.tile_rows > 32 ? launch_kv4_prompt(a, bf16, stream) : bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
  if (e != hipSuccess || a.n_blocks == 0) return e;
  return bf16 ? launch_join<true>(a, stream) : launch_join<false>(a, stream);
}

}  // namespace awq
