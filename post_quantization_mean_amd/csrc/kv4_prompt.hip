// Attention over the 4-bit cache with many rows of a key head: prompts.
//
// Bound by the matrix units: 4 head_dim operations a row and cached token. A block takes 32 RT rows for each of its waves (a
// row: one query head of one new token) and goes over the cached tokens in tiles of kTile, whose keys and values its
// threads turn into float16 in LDS once for all of its rows (1.7 vector operations a code, a quarter of what the softmax
// needs). The tile two ahead is on its way from memory and the next one is being written while a tile is used: two LDS stages, one
// barrier a tile. With v_mfma_f32_32x32x16_f16:
//   S^T = K Q^T   A: token lane % 32, 8 channels; B: the same channels of row lane % 32; D: tokens 4 h + 8 j + 0 .. 3 of that
//                 row (h = lane / 32, j = 0 .. 3).
//   O^T = V^T P^T B is what the softmax left in the lane: tokens 4 h + 0 .. 3 and 8 + 4 h + 0 .. 3 of each 16; values lie in LDS
//                 by channel, those 8 tokens side by side.
// Rounding: as in kv4_attention.hip.
#include <type_traits>

#include "kv4_device.h"

namespace awq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int HD, int WAVES>
struct Tile {
  static constexpr int kTokens = WAVES * 2048 / HD;  // one piece of work for each thread: 64 codes
  static constexpr int kOctets = kTokens / 8;        // of 8 tokens
  static constexpr int kKeyRow = HD * 2, kValueRow = kTokens * 2;  // bytes
  static constexpr int kStage = kTokens * HD * 4;
  // 16-byte chunk c of a row: spread over the banks by the row
  static __device__ __forceinline__ int key_at(int token, int c) {
    constexpr int n = HD / 8;  // chunks of a row
    return token * kKeyRow + ((c ^ (n >= 16 ? token & 15 : (token >> 1) & 7)) << 4);
  }
  static __device__ __forceinline__ int value_at(int channel, int o) {
    constexpr int n = kOctets;
    return kTokens * kKeyRow + channel * kValueRow + ((o ^ (n >= 16 ? channel & 15 : n == 8 ? (channel >> 1) & 7 : (channel >> 2) & 3)) << 4);
  }
  // first token of an octet's two runs of four (the second one lies 8 further)
  static __device__ __forceinline__ int octet_token(int o) { return (o >> 1) * 16 + (o & 1) * 4; }
};

// What a block needs to fetch its key head's cached tokens.
struct Source {
  const uint8_t* codes;
  const uint32_t* params;
  int64_t page_codes, page_params, v_codes, v_params;
  const int32_t* table;
  int page_log2, page_mask, row_bytes;
  uint32_t n_pages;
  __device__ __forceinline__ Source(const AttnArgs& a, const RowTile& t, int head) {
    const int page = 1 << a.c.page_log2;
    row_bytes = a.c.head_dim / 2;
    codes = a.c.codes + (int64_t)head * page * row_bytes;
    params = a.c.params + (int64_t)head * a.c.n_groups * page;
    page_codes = a.c.page_codes;
    page_params = a.c.page_params;
    v_codes = (int64_t)a.c.n_kv * page * row_bytes;
    v_params = (int64_t)a.c.n_kv * a.c.n_groups * page;
    table = a.table + (int64_t)t.seq * a.ld_table;
    page_log2 = a.c.page_log2;
    page_mask = page - 1;
    n_pages = (uint32_t)a.c.n_pages;
  }
};

// A thread's part of turning tiles into float16: one octet of tokens of 8 channels of the values, or 2 x 32 channels of
// tokens of the keys (the waves of a block divide evenly: the choice is uniform in a wave).
template <int HD, int WAVES>
struct Producer {
  using L = Tile<HD, WAVES>;
  static constexpr int kPieces = HD / 32;  // 32 channels of a token's keys
  uint32_t w[8], p[8];                     // codes, params of the tile on its way
  int id[2], next_id[2];                   // its pages, and those of the tile after it
  bool values;
  int octet, channels;                     // values
  int token[2], piece[2];                  // keys
  int at, group;                           // this thread's bytes of a row (keys: both pieces), params of its group
  int key_at[2], key_group[2];

  __device__ __forceinline__ Producer(const AttnArgs& a) {
    const int tid = threadIdx.x, row_bytes = a.c.head_dim / 2, page = 1 << a.c.page_log2;
    values = __builtin_amdgcn_readfirstlane(tid) < WAVES * 32;
    octet = tid % L::kOctets;
    channels = tid / L::kOctets * 8 % HD;
    // channels past the head's last one repeat its first ones: their queries are zeros, their results are not stored
    at = channels < a.c.head_dim ? channels / 2 : 0;
    group = min(channels / 128, a.c.n_groups - 1) * page;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int task = (tid + i * WAVES * 32) % (WAVES * 64);
      token[i] = task / kPieces;
      piece[i] = task % kPieces;
      key_at[i] = piece[i] * 16 < row_bytes ? piece[i] * 16 : 0;
      key_group[i] = min(piece[i] / 4, a.c.n_groups - 1) * page;
    }
  }
  __device__ __forceinline__ int first_token(int i) const { return values ? L::octet_token(octet) : token[i]; }
  __device__ __forceinline__ void pages(const Source& s, int t0, int end) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + first_token(i);
      next_id[i] = t < end ? s.table[t >> s.page_log2] : -1;
    }
  }
  __device__ __forceinline__ void load(const Source& s, int t0) {
    id[0] = next_id[0];
    id[1] = next_id[1];
    if (values) {
      const int64_t page = (uint32_t)id[0] < s.n_pages ? id[0] : 0;
      const int in_page = (t0 + L::octet_token(octet)) & s.page_mask;
      const uint8_t* c = s.codes + s.v_codes + page * s.page_codes + in_page * s.row_bytes + at;
      const uint32_t* q = s.params + s.v_params + page * s.page_params + group + in_page;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(c + (i / 4 * 8 + i % 4) * s.row_bytes);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = *reinterpret_cast<const uint4*>(q + 8 * i);
        p[4 * i] = u.x, p[4 * i + 1] = u.y, p[4 * i + 2] = u.z, p[4 * i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t page = (uint32_t)id[i] < s.n_pages ? id[i] : 0;
        const int in_page = (t0 + token[i]) & s.page_mask;
        const uint4 u = *reinterpret_cast<const uint4*>(s.codes + page * s.page_codes + in_page * s.row_bytes + key_at[i]);
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        p[i] = s.params[page * s.page_params + key_group[i] + in_page];
      }
    }
  }
  // bad: for each octet (and group) the tokens whose values are not finite, zeros in LDS then; gone: octets on no page
  __device__ __forceinline__ void store(const Source& s, char* stage, uint8_t* bad, uint8_t* gone) {
    const uint32_t e = code_exponent();
    if (values) {
      uint32_t any = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) any |= ((p[i] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
      int tokens = 0;
      if (any) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (not_finite(p[i])) tokens |= 1 << i, p[i] = 0;
      }
      if (channels % 128 == 0) bad[channels / 128 * 16 + octet] = (uint8_t)tokens;
      if (channels == 0) gone[octet] = (uint32_t)id[0] < s.n_pages ? 0 : 1;
      h2 step[4], offset[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        step[j] = as_h2(__builtin_amdgcn_perm(p[2 * j + 1], p[2 * j], 0x05040100));
        offset[j] = as_h2(__builtin_amdgcn_perm(p[2 * j + 1], p[2 * j], 0x07060302));
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t u = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], b ? 0x07060302 : 0x05040100);
          v[0][j] = as_u32(low_codes(u, e, step[j], offset[j]));
          v[1][j] = as_u32(high_codes(u, e, step[j], offset[j]));
          v[2][j] = as_u32(low_codes(u >> 8, e, step[j], offset[j]));
          v[3][j] = as_u32(high_codes(u >> 8, e, step[j], offset[j]));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(stage + L::value_at(channels + 4 * b + c, octet)) = make_uint4(v[c][0], v[c][1], v[c][2], v[c][3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const h2 q = as_h2(finite_or_nan(p[i]));
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<h8*>(stage + L::key_at(token[i], piece[i] * 4 + c)) = token_codes(w[4 * i + c], e, h2{q.x, q.x}, h2{q.y, q.y});
      }
    }
  }
};

__device__ __forceinline__ float max_over_halves(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_over_halves(float v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

template <int HD, int RT, int WAVES, bool BF16, bool SPLIT>
__global__ __launch_bounds__(WAVES * 64) void prompt_kernel(AttnArgs a) {
  using T = typename std::conditional<BF16, Bf16, F16>::type;
  using L = Tile<HD, WAVES>;
  constexpr int KS = HD / 16, CT = HD / 32, ST = L::kTokens / 32;
  __shared__ __attribute__((aligned(16))) char lds[2][L::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds_bad[2][2][16], lds_gone[2][16];
  __shared__ int lds_prefix[SPLIT ? kPrefixInts : 1];
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for_pieces<SPLIT>(a, lds_prefix, [&](const RowTile& t, int head, int begin, int end, int part) {
  const int lane = fresh_lane(), half = lane >> 5, m = lane & 31;
  const int wave_row = t.row0 + wave * 32 * RT;

  const Source src(a, t, head);
  Producer<HD, WAVES> in(a);
  const int tiles = begin < end ? (end - begin + L::kTokens - 1) / L::kTokens : 0;
  in.pages(src, begin, end);
  if (tiles > 0) in.load(src, begin);
  in.pages(src, begin + L::kTokens, end);

  // ---- this wave's queries
  h8 q[RT][KS];
  float scale[RT];
  int lo[RT], hi[RT];
#pragma unroll
  for (int n = 0; n < RT; ++n) {
    const int r = wave_row + 32 * n + m;
    const bool there = r < t.rows;
    const int token = a.by_group.of(r), of = r - token * a.group;
    const T* row = (const T*)a.q.p + (int64_t)(t.token0 + token) * a.q.ld + (int64_t)(head * a.group + of) * a.q.ld_head;
    row_range(a, t, r, lo[n], hi[n]);
    hi[n] = min(hi[n], end);
    float top = 0.f, nan = 0.f;
    uint4 raw[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = 16 * s + 8 * half;
      raw[s] = make_uint4(0, 0, 0, 0);
      if (there && c < a.c.head_dim) raw[s] = __builtin_bit_cast(uint4, *reinterpret_cast<const Chunk<T>*>(row + c));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = raw_f32<T>(raw[s], k);
        top = fmaxf(top, fabsf(x));
        nan = fmaf(x, 0.f, nan);
      }
    }
    float up, down;
    query_range<BF16>(max_over_halves(top), a.scale, up, down);
    scale[n] = fmaxf(fabsf(a.scale) * down, 0x1p-126f) + sum_over_halves(nan);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
      for (int k = 0; k < 8; ++k) q[n][s][k] = (_Float16)(raw_f32<T>(raw[s], order[k]) * up);
    }
  }
  // tokens that every row of the wave sees, and that any of them sees
  int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;
  if (wave_row < t.rows) {
    row_range(a, t, wave_row, any_lo, all_hi);
    row_range(a, t, min(wave_row + 32 * RT, t.rows) - 1, all_lo, any_hi);
    all_hi = min(all_hi, end);
    any_hi = min(any_hi, end);
  }

  f32x16 o[RT][CT];
  float top[RT], sum[RT];
  uint32_t poisoned[RT];
#pragma unroll
  for (int n = 0; n < RT; ++n) {
    top[n] = kNothing;
    sum[n] = 0.f;
    poisoned[n] = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[n][c][i] = 0.f;
  }

  if (tiles > 0) {
    in.store(src, lds[0], lds_bad[0][0], lds_gone[0]);
    if (tiles > 1) {
      in.load(src, begin + L::kTokens);
      in.pages(src, begin + 2 * L::kTokens, end);
    }
  }
  for (int i = 0; i < tiles; ++i) {
    const int t0 = begin + i * L::kTokens, b = i & 1;
    char* const stage = lds[b];
    __syncthreads();
    if (i + 1 < tiles) {
      in.store(src, lds[b ^ 1], lds_bad[b ^ 1][0], lds_gone[b ^ 1]);
      if (i + 2 < tiles) {
        in.load(src, t0 + 2 * L::kTokens);
        in.pages(src, t0 + 3 * L::kTokens, end);
      }
    }
    if (t0 >= any_hi || t0 + L::kTokens <= any_lo) continue;
    const uint4 gone = *reinterpret_cast<const uint4*>(lds_gone[b]);
    const bool whole = t0 >= all_lo && t0 + L::kTokens <= all_hi &&
                       (L::kOctets < 8 ? gone.x == 0 : L::kOctets < 16 ? (gone.x | gone.y) == 0 : (gone.x | gone.y | gone.z | gone.w) == 0);
#pragma unroll
    for (int st = 0; st < ST; ++st) {
      // ---- scores
      f32x16 s[RT];
#pragma unroll
      for (int n = 0; n < RT; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[n][j] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const h8 f = *reinterpret_cast<const h8*>(stage + L::key_at(32 * st + m, 2 * k + half));
#pragma unroll
        for (int n = 0; n < RT; ++n) s[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, q[n][k], s[n], 0, 0, 0);
      }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int at = 32 * st + 4 * half + 8 * (j / 4) + j % 4;
          const bool gone_j = lds_gone[b][4 * st + 2 * (j / 8) + half] != 0;
#pragma unroll
          for (int n = 0; n < RT; ++n)
            if (t0 + at < lo[n] || t0 + at >= hi[n] || gone_j) s[n][j] = -__builtin_inff();
        }
      }
      // ---- values that are not finite
      {
        uint32_t any = *reinterpret_cast<const uint32_t*>(&lds_bad[b][0][4 * st]);
        if (HD > 128) any |= *reinterpret_cast<const uint32_t*>(&lds_bad[b][1][4 * st]);
        if (__builtin_amdgcn_readfirstlane((int)any) != 0) {
#pragma unroll
          for (int c = 0; c < (HD + 127) / 128; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int octet = 4 * st + 2 * (j / 8) + half, at = t0 + 32 * st + 4 * half + 8 * (j / 4) + j % 4;
              const bool hit = c < a.c.n_groups && (lds_bad[b][c][octet] >> (j % 8) & 1) && !lds_gone[b][octet];
#pragma unroll
              for (int n = 0; n < RT; ++n)
                if (hit && at >= lo[n] && at < hi[n]) poisoned[n] |= 1u << c;
            }
        }
      }
      // ---- numerators
      h8 p[RT][2];
#pragma unroll
      for (int n = 0; n < RT; ++n) {
        float most = s[n][0];
#pragma unroll
        for (int j = 1; j < 16; ++j) most = fmaxf(most, s[n][j]);
        most = max_over_halves(most) * scale[n];
        if (__any(most > top[n] + 15.f)) {
          const float higher = fmaxf(most - 7.f, top[n]);
          const float f = __builtin_amdgcn_exp2f(top[n] - higher);
          top[n] = higher;
          sum[n] *= f;
#pragma unroll
          for (int c = 0; c < CT; ++c) o[n][c] *= f;
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const auto two = __builtin_amdgcn_cvt_pkrtz(__builtin_amdgcn_exp2f(fmaf(s[n][j], scale[n], -top[n])),
                                                      __builtin_amdgcn_exp2f(fmaf(s[n][j + 1], scale[n], -top[n])));
          const h2 pair = __builtin_bit_cast(h2, two);
          sum[n] = __builtin_amdgcn_fdot2(pair, h2{(_Float16)1.f, (_Float16)1.f}, sum[n], false);
          p[n][j / 8][j % 8] = pair.x;
          p[n][j / 8][j % 8 + 1] = pair.y;
        }
      }
      // ---- their product with the values
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const h8 f = *reinterpret_cast<const h8*>(stage + L::value_at(32 * c + m, 4 * st + 2 * u + half));
#pragma unroll
          for (int n = 0; n < RT; ++n) o[n][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, p[n][u], o[n][c], 0, 0, 0);
        }
    }
  }

  // ---- results: a lane has channels 32 c + 8 j + 4 half + 0 .. 3 of its rows
  const bool final = part < 0;
#pragma unroll
  for (int n = 0; n < RT; ++n) {
    const float total = sum_over_halves(sum[n]);
    const auto both = __builtin_amdgcn_permlane32_swap(poisoned[n], poisoned[n], false, false);
    poisoned[n] = both[0] | both[1];
    const int r = wave_row + 32 * n + m;
    if (r >= t.rows) continue;
    const int token = a.by_group.of(r), of = head * a.group + (r - token * a.group);
    const int64_t at = (int64_t)(t.token0 + token) * a.n_heads + of;
    const int64_t slot = (int64_t)part * a.tile_rows + (r - t.row0);
    if (half == 0) {
      if (!final) {
        float* ml = a.part_ml + 2 * slot;
        ml[0] = top[n];
        ml[1] = total;
      } else if (a.lse) {
        a.lse[at] = total == 0.f ? -__builtin_inff() : (top[n] + __log2f(total)) * kLn2;
      }
    }
    const float inv = final ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const float nan = (poisoned[n] >> (c / 4)) & 1 ? __builtin_nanf("") : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int channel = 32 * c + 8 * j + 4 * half;
        if (channel >= a.c.head_dim) continue;
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = fmaf(o[n][c][4 * j + k], inv, nan);
        if (!final) {
          *reinterpret_cast<f32x4*>(a.part_o + slot * a.c.head_dim + channel) = f32x4{y[0], y[1], y[2], y[3]};
          continue;
        }
        store4<BF16>(a, (int64_t)(t.token0 + token) * a.out.ld + (int64_t)of * a.out.ld_head + channel, y);
      }
    }
  }
  });
}

template <int HD, int RT, int WAVES>
void launch(const AttnArgs& a, bool bf16, hipStream_t stream) {
  static_assert(prompt_rows(HD) == 32 * RT * WAVES, "rows of a block");
  const dim3 grid = a.n_blocks ? dim3((unsigned)a.n_blocks) : dim3((unsigned)a.n_tiles, (unsigned)a.c.n_kv);
  if (a.n_blocks) {
    if (bf16) prompt_kernel<HD, RT, WAVES, true, true><<<grid, WAVES * 64, 0, stream>>>(a);
    else prompt_kernel<HD, RT, WAVES, false, true><<<grid, WAVES * 64, 0, stream>>>(a);
  } else {
    if (bf16) prompt_kernel<HD, RT, WAVES, true, false><<<grid, WAVES * 64, 0, stream>>>(a);
    else prompt_kernel<HD, RT, WAVES, false, false><<<grid, WAVES * 64, 0, stream>>>(a);
  }
}

}  // namespace

hipError_t launch_kv4_prompt(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (a.c.head_dim <= 64) launch<64, 2, 4>(a, bf16, stream);
  else if (a.c.head_dim <= 128) launch<128, 2, 4>(a, bf16, stream);
  else launch<256, 1, 4>(a, bf16, stream);
  return hipGetLastError();
}

}  // namespace awq
