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
// So no operand crosses a lane, and nothing goes through LDS until the waves join. Codes become float16 numbers offset +
// code * step with one rounding (2^-11 of the number at most); 1.7 vector operations a code.
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
  uint32_t k[2][KW], kp[2];
  uint32_t v[8][(VB + 3) / 4], vp[8];
  bool there[2];
};

template <int HD>
struct Loader {
  const uint8_t* codes;      // the key head's keys in page 0
  const uint32_t* params;
  int64_t page_codes, page_params, v_codes, v_params;  // from keys to values
  const int32_t* table;
  int page_log2, page_mask, row_bytes, lane_pages;
  uint32_t n_pages;
  int k_at[(HD + 127) / 128], v_at, k_group, v_group;  // this lane's bytes of a row, its groups' params (in words)

  // The pages of the wave's next 64 tiles of 16 tokens: lane i has tile i's (-1 past the end).
  __device__ __forceinline__ void pages(int t0, int stride, int end) {
    const int lane = threadIdx.x & 63, t = t0 + (lane >> 1) * stride + (lane & 1) * 16;
    lane_pages = t < end ? table[t >> page_log2] : -1;
  }
  __device__ __forceinline__ void load(Stage<HD>& s, int i, int t0) const {
    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
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
        const uint2 u = *reinterpret_cast<const uint2*>(kc + m * row_bytes + k_at[0]);
        s.k[h][0] = u.x, s.k[h][1] = u.y;
      } else {
#pragma unroll
        for (int c = 0; c < HD / 128; ++c) {
          const uint4 u = *reinterpret_cast<const uint4*>(kc + m * row_bytes + k_at[c]);
          s.k[h][4 * c] = u.x, s.k[h][4 * c + 1] = u.y, s.k[h][4 * c + 2] = u.z, s.k[h][4 * c + 3] = u.w;
        }
      }
      s.kp[h] = kp[k_group + m];
      const uint4 p = *reinterpret_cast<const uint4*>(vp + v_group + 4 * g);
      s.vp[4 * h] = p.x, s.vp[4 * h + 1] = p.y, s.vp[4 * h + 2] = p.z, s.vp[4 * h + 3] = p.w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* row = vc + (4 * g + j) * row_bytes + v_at;
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

// A lane's part of the queries' operand: rows m of NR tiles, channels g * HD/4 .. in the order of token_codes.
template <int HD, int NR, bool BF16>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const RowTile& t, int head, h8 (&q)[NR][HD / 32], float (&scale)[NR]) {
  using T = typename std::conditional<BF16, Bf16, F16>::type;
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const int r = t.row0 + 16 * n + m;
    const bool there = r < t.rows;
    const int token = r / a.group, of = r - token * a.group;
    const T* row = (const T*)a.q.p + (t.token0 + token) * a.q.ld + (int64_t)(head * a.group + of) * a.q.ld_head;
    float x[HD / 32][8], top = 0.f, nan = 0.f;
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) {
      const int c = g * (HD / 4) + s * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[s][k] = 0.f;
      if (there && c < a.c.head_dim) load_chunk(row, c, a.c.head_dim, x[s]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        top = fmaxf(top, fabsf(x[s][k]));
        nan = fmaf(x[s][k], 0.f, nan);
      }
    }
    float up, down;
    query_range<BF16>(max_over_rows(top), a.scale, up, down);
    scale[n] = fmaxf(fabsf(a.scale) * down, 0x1p-126f) + sum_over_rows(nan);  // NaN for a row with a NaN or an infinity
#pragma unroll
    for (int s = 0; s < HD / 32; ++s) {
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
      for (int k = 0; k < 8; ++k) q[n][s][k] = (_Float16)(x[s][order[k]] * up);
    }
  }
}

template <int HD, int NR, bool BF16>
__global__ __launch_bounds__(kWaves * 64) void rows_kernel(AttnArgs a) {
  constexpr int CT = HD / 16;  // channel tiles; a lane's channels are m * CT .. and, of the result, (4 g + i) * CT ..
  constexpr int kPitch = HD + 4;
  __shared__ float lds_o[kWaves][16][kPitch];
  __shared__ float lds_m[kWaves][16 * NR], lds_l[kWaves][16 * NR];
  const RowTile t = row_tile(a, (int)blockIdx.x);
  if (t.row0 >= t.rows) return;
  const KvSpan span = kv_span(a, t);
  const int part = (int)blockIdx.z;
  if (part >= max(span.parts, 1)) return;
  const int head = (int)blockIdx.y;
  const int begin = span.begin + part * span.chunk, end = min(span.end, begin + span.chunk);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;

  h8 q[NR][HD / 32];
  float scale[NR];
  load_queries<HD, NR, BF16>(a, t, head, q, scale);
  int lo[NR], hi[NR], all_lo, all_hi, unused;
#pragma unroll
  for (int n = 0; n < NR; ++n) row_range(a, t, t.row0 + 16 * n + m, lo[n], hi[n]);
  // tokens in [all_lo, all_hi) are seen by every row of the tile
  row_range(a, t, t.row0, unused, all_hi);
  row_range(a, t, min(t.row0 + 16 * NR, t.rows) - 1, all_lo, unused);

  Loader<HD> in;
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
    const int at = g * (HD / 8) + 16 * c;
    in.k_at[c] = at < in.row_bytes ? at : 0;
  }
  in.k_group = min(g * (HD / 4) / 128, a.c.n_groups - 1) * page;
  in.v_at = m * (HD / 32) < in.row_bytes ? m * (HD / 32) : 0;
  in.v_group = min(m * CT / 128, a.c.n_groups - 1) * page;

  f32x4 o[NR][CT];
  float top[NR], sum[NR];  // the reference of a row's numerators, and their sum in this lane
  uint32_t poisoned[NR];  // groups (bits) whose values a row has seen a NaN in
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    top[n] = kNothing;
    sum[n] = 0.f;
    poisoned[n] = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) o[n][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  constexpr int kStride = kWaves * kStep;
  const int first = begin + wave * kStep;
  const int steps = first < end ? (end - first + kStride - 1) / kStride : 0;
  // 32 tokens from t0 on
  const auto take = [&](Stage<HD>& now, int t0) {
    // ---- scores
    f32x4 s[NR][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = finite_or_nan(now.kp[h]);
      const h2 p = as_h2(w), step = h2{p.x, p.x}, offset = h2{p.y, p.y};
#pragma unroll
      for (int n = 0; n < NR; ++n) s[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        const h8 k = token_codes(now.k[h][c], step, offset);
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][c], s[n][h], 0, 0, 0);
      }
    }
    const bool whole = t0 >= all_lo && t0 + kStep <= all_hi && t0 + kStep <= end && now.there[0] && now.there[1];
    // ---- values that are not finite: out of the products, noted for the rows that see them
    uint32_t bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) bad |= ((now.vp[j] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
    if (__any(bad != 0)) {
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
    h8 p[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float x[8], most = -__builtin_inff();
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * h + j] = s[n][h][j];
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = t0 + 16 * h + 4 * g + j;
            if (at < lo[n] || at >= min(hi[n], end) || !now.there[h]) x[4 * h + j] = -__builtin_inff();
          }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, x[j]);
      most = max_over_rows(most) * scale[n];
      // The numerators are powers from a reference that is set 2^7 below the largest score and moves only when they would
      // pass 2^15: float16 holds them, down to 2^-31 of the largest.
      if (__any(most > top[n] + 15.f)) {
        const float higher = fmaxf(most - 7.f, top[n]);
        const float f = __builtin_amdgcn_exp2f(top[n] - higher);
        top[n] = higher;
        sum[n] *= f;
#pragma unroll
        for (int c = 0; c < CT; ++c) o[n][c] *= f;
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        // rounded towards zero, and summed as rounded: the weights add up to one, and the rounding's bias cancels
        const auto two = __builtin_amdgcn_cvt_pkrtz(__builtin_amdgcn_exp2f(fmaf(x[j], scale[n], -top[n])),
                                                    __builtin_amdgcn_exp2f(fmaf(x[j + 1], scale[n], -top[n])));
        const h2 pair = __builtin_bit_cast(h2, two);
        sum[n] = __builtin_amdgcn_fdot2(pair, h2{(_Float16)1.f, (_Float16)1.f}, sum[n], false);
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
        v[0][j] = low_codes(u, step[j], offset[j]);
        v[1][j] = high_codes(u, step[j], offset[j]);
        v[2][j] = low_codes(u >> 8, step[j], offset[j]);
        v[3][j] = high_codes(u >> 8, step[j], offset[j]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const h8 f = {v[c][0].x, v[c][0].y, v[c][1].x, v[c][1].y, v[c][2].x, v[c][2].y, v[c][3].x, v[c][3].y};
#pragma unroll
        for (int n = 0; n < NR; ++n) o[n][4 * b + c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f, p[n], o[n][4 * b + c], 0, 0, 0);
      }
    }
  };
  Stage<HD> even, odd;
  if (steps > 0) {
    in.pages(first, kStride, end);
    in.load(even, 0, first);
  }
  for (int i = 0; i < steps; i += 2) {
    const int t0 = first + i * kStride;
    if (i + 1 < steps) in.load(odd, (i + 1) & 31, t0 + kStride);
    take(even, t0);
    if (i + 1 >= steps) break;
    if (i + 2 < steps) {
      if (((i + 2) & 31) == 0) in.pages(t0 + 2 * kStride, kStride, end);
      in.load(even, (i + 2) & 31, t0 + 2 * kStride);
    }
    take(odd, t0 + kStride);
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
  const int64_t all_rows = a.n_tokens * a.n_heads;
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
      float most = kNothing;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) most = fmaxf(most, lds_m[w][16 * n + row]);
      float f[kWaves], total = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = __builtin_amdgcn_exp2f(lds_m[w][16 * n + row] - most);
        total = fmaf(f[w], lds_l[w][16 * n + row], total);
      }
      const int token = r / a.group, of = head * a.group + (r - token * a.group);
      const int64_t at = (t.token0 + token) * a.n_heads + of;
      const bool final = span.parts <= 1;
      const float inv = final ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
      if ((int)threadIdx.x % kRowThreads == 0) {
        if (!final) {
          float* ml = a.part_ml + 2 * (part * all_rows + at);
          ml[0] = most;
          ml[1] = total;
        } else if (a.lse) {
          a.lse[at] = total == 0.f ? -__builtin_inff() : (most + __log2f(total)) * kLn2;
        }
      }
      for (int c = (int)threadIdx.x % kRowThreads * 4; c < a.c.head_dim; c += kRowThreads * 4) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = fmaf(f[w], lds_o[w][row][c + k], y[k]);
        if (!final) {
          *reinterpret_cast<f32x4*>(a.part_o + (part * all_rows + at) * a.c.head_dim + c) = f32x4{y[0], y[1], y[2], y[3]};
          continue;
        }
        const int64_t to = (t.token0 + token) * a.out.ld + (int64_t)of * a.out.ld_head + c;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] *= inv;
        store4<BF16>(a, to, y);
      }
    }
  }
}

// Joins the parts of rows whose cached tokens several blocks have taken. Block (tile, key head, row of the tile); threads:
// 8 parts at once, 4 channels each.
template <bool BF16>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a) {
  __shared__ float lds[8][260];
  __shared__ float lds_l[8];
  const RowTile t = row_tile(a, (int)blockIdx.x);
  const int r = t.row0 + (int)blockIdx.z;
  if (t.row0 >= t.rows || r >= t.rows) return;
  const KvSpan span = kv_span(a, t);
  if (span.parts <= 1) return;
  const int head = (int)blockIdx.y, token = r / a.group, of = head * a.group + (r - token * a.group);
  const int64_t all_rows = a.n_tokens * a.n_heads, at = (t.token0 + token) * a.n_heads + of;
  float most = kNothing;
  for (int i = threadIdx.x & 63; i < span.parts; i += 64) most = fmaxf(most, a.part_ml[2 * (i * all_rows + at)]);
#pragma unroll
  for (int d = 32; d; d >>= 1) most = fmaxf(most, __shfl_xor(most, d));
  const int group = (int)threadIdx.x / 32, lane = (int)threadIdx.x % 32;
  float y[2][4] = {}, total = 0.f;
  for (int i = group; i < span.parts; i += 8) {
    const float* ml = a.part_ml + 2 * (i * all_rows + at);
    const float f = __builtin_amdgcn_exp2f(ml[0] - most);
    total = fmaf(f, ml[1], total);
    const float* o = a.part_o + (i * all_rows + at) * a.c.head_dim;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 128 * h + 4 * lane;
      if (c < a.c.head_dim) {
        const f32x4 u = *reinterpret_cast<const f32x4*>(o + c);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[h][k] = fmaf(f, u[k], y[h][k]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int k = 0; k < 4; ++k) lds[group][128 * h + 4 * lane + k] = y[h][k];
  if (lane == 0) lds_l[group] = total;
  __syncthreads();
  const int c = threadIdx.x;
  total = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) total += lds_l[i];
  if (c == 0 && a.lse) a.lse[at] = total == 0.f ? -__builtin_inff() : (most + __log2f(total)) * kLn2;
  if (c >= a.c.head_dim) return;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) z += lds[i][c];
  z = total == 0.f ? 0.f : z / total;
  const int64_t to = (t.token0 + token) * a.out.ld + (int64_t)of * a.out.ld_head + c;
  if (a.out_f32) ((float*)a.out.p)[to] = z;
  else if (BF16) ((Bf16*)a.out.p)[to] = from_f32<Bf16>(z);
  else ((F16*)a.out.p)[to] = from_f32<F16>(z);
}

template <int HD, bool BF16>
void launch_rows(const AttnArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)a.n_tiles, (unsigned)a.c.n_kv, (unsigned)a.n_chunks);
  if (a.tile_rows == 16) rows_kernel<HD, 1, BF16><<<grid, kWaves * 64, 0, stream>>>(a);
  else rows_kernel<HD, 2, BF16><<<grid, kWaves * 64, 0, stream>>>(a);
}

template <bool BF16>
hipError_t launch(const AttnArgs& a, hipStream_t stream) {
  if (a.c.head_dim <= 64) launch_rows<64, BF16>(a, stream);
  else if (a.c.head_dim <= 128) launch_rows<128, BF16>(a, stream);
  else launch_rows<256, BF16>(a, stream);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_join(const AttnArgs& a, hipStream_t stream) {
  join_kernel<BF16><<<dim3((unsigned)a.n_tiles, (unsigned)a.c.n_kv, (unsigned)a.tile_rows), 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// Rows of a sequence and key head up to which a block of the kernel above takes 32 of them; past that the kernel for prompts.
constexpr int kFewRows = 64;

size_t plan_attention(AttnArgs* a, bool ragged) {
  const int64_t rows_each = (a->n_tokens + a->n_seqs - 1) / a->n_seqs * a->group;
  a->tile_rows = rows_each <= 16 ? 16 : rows_each <= kFewRows ? 32 : prompt_rows(a->c.head_dim);
  if (ragged) a->n_tiles = (int)(a->n_tokens * a->group / a->tile_rows + a->n_seqs);
  else a->n_tiles = (int)(a->n_seqs * ((rows_each + a->tile_rows - 1) / a->tile_rows));
  int64_t span = a->max_kv;
  if (a->window && a->causal) span = min(span, (int64_t)a->window + a->tile_rows / a->group + kAlign);
  constexpr int64_t kBlocks = 1024, kLeast = 256;
  const int64_t blocks = (int64_t)a->n_tiles * a->c.n_kv;
  int64_t chunks = max((int64_t)1, min(kBlocks / blocks, span / kLeast));
  a->chunk = (int)(((span + chunks - 1) / chunks + kWaves * kStep - 1) / (kWaves * kStep) * (kWaves * kStep));
  a->chunk = max(a->chunk, kWaves * kStep);
  chunks = max((int64_t)1, (span + a->chunk - 1) / a->chunk);
  a->n_chunks = (int)chunks;
  if (chunks == 1) return 0;
  return (size_t)chunks * (size_t)a->n_tokens * a->n_heads * (a->c.head_dim + 2);
}

hipError_t launch_kv4_attention(const AttnArgs& a, bool bf16, hipStream_t stream) {
  hipError_t e = a.tile_rows > 32 ? launch_kv4_prompt(a, bf16, stream) : bf16 ? launch<true>(a, stream) : launch<false>(a, stream);
  if (e != hipSuccess || a.n_chunks == 1) return e;
  return bf16 ? launch_join<true>(a, stream) : launch_join<false>(a, stream);
}

}  // namespace awq
