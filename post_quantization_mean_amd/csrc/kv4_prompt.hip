// Attention over the 4-bit cache with many rows of a key head: prompts.
//
// Bound by the matrix units and the vector units that feed them: 4 head_dim operations a row and cached token, beside one
// exponential. A block takes 32 rows for each of its waves (a row: one query head of one new token) and goes over the cached
// tokens in tiles of kTokens, whose keys and values its threads turn into float16 in LDS once for all of its rows (1.7
// vector operations a code). The tile after the one in use is written to LDS between its products, the one after that is on
// its way from memory: two LDS stages, one barrier a tile. With v_mfma_f32_32x32x16_f16:
//   S^T = K Q^T   A: token lane % 32, 8 channels; B: the same channels of row lane % 32; D: tokens 4 h + 8 j + 0 .. 3 of that
//                 row (h = lane / 32, j = 0 .. 3).
//   O^T = V^T P^T B is what the softmax left in the lane: tokens 4 h + 0 .. 3 and 8 + 4 h + 0 .. 3 of each 16; values lie in LDS
//                 by channel, those 8 tokens side by side.
// A wave's products and its softmax overlap: while the scores of 32 tokens become numerators, the next 32 tokens' scores
// are multiplied, and while their maximum is found, the 32 before them meet the values. 32 rows a wave, so that two
// waves of a SIMD fit its registers without the accumulators' moves between its two files: 64 rows a wave, one wave a
// SIMD, took 2.93 ms instead of 1.78 for 4096 tokens of 64 heads on 8 behind 8192.
// Rounding: keys and values become float16 numbers with one rounding each, 2^-11 of the number at most; numerators are rounded to
// the nearest.
//
// 4096 tokens of 64 heads on 8 of 128 behind 8192: 1.47 - 1.54 ms (890 - 930 TFLOP/s; a large float16 library product reaches 1130
// on this card). 4096 causal tokens of 32 heads with their own keys: 175 us (785). 9 prompts of up to 1500 tokens, 32 heads on 8
// of 64: 105 us; heads of 64 have half the products for each exponential (4 x 2048 tokens behind 2048: 305 us, 675 TFLOP/s;
// as two blocks of four waves a compute unit 338, the prompts alike), heads of 256 one wave a SIMD (535). Heads of 32 run as 64, of 96
// as 128, of 160 to 224 as 256, with products of zeros (4096 tokens of 32 heads of 96 173 us, of 128 171).
#include <type_traits>

#include "kv4_device.h"

namespace awq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int HD, int WAVES>
struct Tile {
  static constexpr int kTokens = WAVES * 2048 / HD;  // a thread turns 32 codes of keys and 32 of values
  static constexpr int kQuads = kTokens / 4, kFlags = (HD + 127) / 128 * kQuads;
  // Rows of LDS: a token's keys, a channel's values. Sixteen bytes more than they hold, so that sixteen rows' chunks at the same
  // place lie in different banks and a chunk's place is a constant.
  static constexpr int kKeyRow = HD * 2 + 16, kValueRow = kTokens * 2 + 16;
  static constexpr int kValues = kTokens * kKeyRow, kStage = kValues + HD * kValueRow;
  static __device__ __forceinline__ int key_at(int token, int c) { return token * kKeyRow + c * 16; }
  // A channel's row: channels 8 i + k lie in rows k HD/8 + i, which the lanes that write them (i) find in different banks, and
  // which leaves a lane of the result eight channels side by side.
  static __device__ __forceinline__ int value_row(int channel) { return channel % 8 * (HD / 8) + channel / 8; }
  // Chunk o of a row: the eight tokens 16 (o / 2) + 4 (o % 2) + 0 .. 3 and 8 + those.
  static __device__ __forceinline__ int value_at(int row, int o) { return kValues + row * kValueRow + o * 16; }
};

// A wave's part of turning tiles into float16: the keys and values of kTokens / WAVES consecutive tokens; a lane has 32 channels
// of one token's keys, and 8 channels of four tokens' values. Sixteen tokens lie on one page, so that addresses are a
// page's, the wave's, and an offset of the lane's that stays.
template <int HD, int WAVES>
struct Producer {
  using L = Tile<HD, WAVES>;
  static constexpr int kMine = L::kTokens / WAVES, kRuns = kMine > 16 ? kMine / 16 : 1;  // runs of 16 tokens of a wave
  const uint8_t* codes;                  // the key head's keys in page 0, and what lies from keys to values
  const uint32_t* params;
  int64_t page_codes, page_params, v_codes, v_params;
  const int32_t* table;
  int page_log2, page_mask, row_bytes, first;  // first: the wave's first token in a tile
  uint32_t n_pages;
  int id[kRuns], next_id[kRuns];         // pages of the tile on its way, and of the one after it
  uint32_t k[4], kp, v[4], vp[4];        // codes and params of the tile on its way
  int k_run, v_run, k_off, kp_off, v_off, vp_off, k_lds, v_lds, flag, gone;

  __device__ __forceinline__ Producer(const AttnArgs& a, const RowTile& t, int head, int wave, int lane) {
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
    first = wave * kMine;
    const int token = lane / (HD / 32), piece = lane % (HD / 32);
    // channels past the head's last one repeat its first ones: their queries are zeros, their results are not stored
    k_off = token % 16 * row_bytes + (piece * 16 < row_bytes ? piece * 16 : 0);
    kp_off = min(piece / 4, a.c.n_groups - 1) * page + token % 16;
    k_lds = L::key_at(first + token, 4 * piece);
    const int quads = kMine / 4, quad = lane % quads, octet = lane / quads;  // quads 2 o and 2 o + 1 are chunk o
    const int in_tile = first / 4 + quad, at = in_tile / 2 % 2 * 4 + in_tile % 2 * 8;  // in its run
    v_off = at * row_bytes + (octet * 4 < row_bytes ? octet * 4 : 0);
    vp_off = min(octet / 16, a.c.n_groups - 1) * page + at;
    v_lds = L::value_at(octet, in_tile / 2) + in_tile % 2 * 8;
    flag = octet / 16 * L::kQuads + in_tile;  // (the lanes of a group's channels write the same)
    k_run = kRuns > 1 ? token / 16 : 0;
    v_run = kRuns > 1 ? quad / 4 : 0;
    gone = 0;
  }
  __device__ __forceinline__ void pages(int t0, int end) {
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int t = t0 + (first & ~15) + 16 * i;
      next_id[i] = t < end ? table[t >> page_log2] : -1;
    }
  }
  __device__ __forceinline__ bool there(int i) const { return (uint32_t)id[i] < n_pages; }
  // The lane's page and place in it: offsets of bytes of codes and of words of params.
  __device__ __forceinline__ void place(int t0, int run, int64_t& c, int64_t& p) const {
    int in_page = t0 & page_mask;
    int64_t page = there(0) ? id[0] : 0;
    c = page * page_codes + (int64_t)in_page * row_bytes;
    p = page * page_params + in_page;
#pragma unroll
    for (int i = 1; i < kRuns; ++i) {
      in_page = (t0 + 16 * i) & page_mask;
      page = there(i) ? id[i] : 0;
      if (run == i) c = page * page_codes + (int64_t)in_page * row_bytes, p = page * page_params + in_page;
    }
  }
  __device__ __forceinline__ void load_keys(int t0) {
#pragma unroll
    for (int i = 0; i < kRuns; ++i) id[i] = __builtin_amdgcn_readfirstlane(next_id[i]);
    int64_t c, p;
    place(t0 + first, k_run, c, p);
    const uint4 u = *reinterpret_cast<const uint4*>(codes + c + (uint32_t)k_off);
    k[0] = u.x, k[1] = u.y, k[2] = u.z, k[3] = u.w;
    kp = params[p + (uint32_t)kp_off];
  }
  __device__ __forceinline__ void load_values(int t0) {  // after load_keys
    int64_t c, p;
    place(t0 + (first & ~15), v_run, c, p);
    gone = there(0) ? 0 : 16;
#pragma unroll
    for (int i = 1; i < kRuns; ++i)
      if (v_run == i) gone = there(i) ? 0 : 16;
    const uint8_t* from = codes + v_codes + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(from + i * row_bytes + (uint32_t)v_off);
    const uint4 u = *reinterpret_cast<const uint4*>(params + v_params + p + (uint32_t)vp_off);
    vp[0] = u.x, vp[1] = u.y, vp[2] = u.z, vp[3] = u.w;
  }
  // Half of the keys (two words).
  template <int HALF>
  __device__ __forceinline__ void store_keys(char* stage, uint32_t e) {
    const h2 q = as_h2(finite_or_nan(kp));
#pragma unroll
    for (int c = 2 * HALF; c < 2 * HALF + 2; ++c)
      *reinterpret_cast<h8*>(stage + k_lds + 16 * c) = token_codes(k[c], e, h2{q.x, q.x}, h2{q.y, q.y});
  }
  // Half of the values (four channels). flags: for each group and quad a byte: the tokens whose values are not
  // finite (bits 0 - 3; zeros in LDS then), and whether they lie on no page (bit 4).
  template <int HALF>
  __device__ __forceinline__ void store_values(char* stage, uint8_t* flags, uint32_t e) {
    if constexpr (HALF == 0) {
      int bad = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool b = not_finite(vp[i]);
        bad |= b ? 1 << i : 0;
        vp[i] = b ? 0 : vp[i];
      }
      flags[flag] = (uint8_t)(bad | gone);
    }
    h2 step[2], offset[2];
    uint32_t f[4][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      step[j] = as_h2(__builtin_amdgcn_perm(vp[2 * j + 1], vp[2 * j], 0x05040100));
      offset[j] = as_h2(__builtin_amdgcn_perm(vp[2 * j + 1], vp[2 * j], 0x07060302));
      const uint32_t u = __builtin_amdgcn_perm(v[2 * j + 1], v[2 * j], HALF ? 0x07060302 : 0x05040100);
      f[0][j] = as_u32(low_codes(u, e, step[j], offset[j]));
      f[1][j] = as_u32(high_codes(u, e, step[j], offset[j]));
      f[2][j] = as_u32(low_codes(u >> 8, e, step[j], offset[j]));
      f[3][j] = as_u32(high_codes(u >> 8, e, step[j], offset[j]));
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint2*>(stage + v_lds + (4 * HALF + c) * (HD / 8) * L::kValueRow) = make_uint2(f[c][0], f[c][1]);
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

template <int HD, int WAVES, bool BF16, bool SPLIT>
__global__ __launch_bounds__(WAVES * 64, WAVES == 8 ? 2 : 1) void prompt_kernel(AttnArgs a) {
  using T = typename std::conditional<BF16, Bf16, F16>::type;
  using L = Tile<HD, WAVES>;
  constexpr int KS = HD / 16, CT = HD / 32, ST = L::kTokens / 32;
  constexpr bool PIPED = HD <= 128;  // (heads past 128 leave no registers for it)
  __shared__ __attribute__((aligned(16))) char lds[2][L::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t lds_flags[2][L::kFlags];
  __shared__ int lds_prefix[SPLIT ? kPrefixInts : 1];
  __shared__ float lds_base[WAVES * 32], lds_scale[WAVES * 32];  // of the rows' references, and their scales as they are
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  for_pieces<SPLIT>(a, lds_prefix, [&](const RowTile& t, int head, int begin, int end, int part) {
  const int lane = fresh_lane(), half = lane >> 5, m = lane & 31;
  const int r = t.row0 + wave * 32 + m;  // the lane's row
  const uint32_t e = code_exponent();

  Producer<HD, WAVES> in(a, t, head, wave, lane);
  const int tiles = begin < end ? (end - begin + L::kTokens - 1) / L::kTokens : 0;
  in.pages(begin, end);
  in.load_keys(begin);
  in.load_values(begin);
  in.pages(begin + L::kTokens, end);

  // ---- this wave's queries
  h8 q[KS];
  int lo, hi;
  row_range(a, t, r, lo, hi);
  hi = min(hi, end);
  float scale;
  {
    const bool there = r < t.rows;
    const int row = min(r, t.rows - 1), token = a.by_group.of(row), of = row - token * a.group;
    const T* from = (const T*)a.q.p + (int64_t)(t.token0 + token) * a.q.ld + (int64_t)(head * a.group + of) * a.q.ld_head;
    float size = 0.f, nan = 0.f;
    uint4 raw[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = 16 * s + 8 * half;
      raw[s] = __builtin_bit_cast(uint4, *reinterpret_cast<const Chunk<T>*>(from + (c < a.c.head_dim ? c : 0)));
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (!there || 16 * s + 8 * half >= a.c.head_dim) raw[s] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = raw_f32<T>(raw[s], k);
        size = fmaxf(size, fabsf(x));
        nan = fmaf(x, 0.f, nan);
      }
    }
    float up, down;
    query_range<BF16>(max_over_halves(size), a.scale, up, down);
    const float as_is = fminf(fmaxf(fabsf(a.scale) * down, 0x1p-126f), kLargestFloat);
    lds_scale[wave * 32 + m] = as_is;
    scale = scale_in_range(as_is);
    // a row with a NaN or an infinity has NaN for every score, its scale stays a number: where it sees nothing it is nothing
    nan = sum_over_halves(nan);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
      for (int k = 0; k < 8; ++k) q[s][k] = (_Float16)fmaf(raw_f32<T>(raw[s], order[k]), up, nan);
    }
  }
  // tokens that every row of the wave sees, and that any of them sees
  int all_lo = 0, all_hi = 0, any_lo = 0, any_hi = 0;
  const int wave_row = t.row0 + wave * 32;
  if (wave_row < t.rows) {
    row_range(a, t, wave_row, any_lo, all_hi);
    row_range(a, t, min(wave_row + 32, t.rows) - 1, all_lo, any_hi);
    all_hi = min(all_hi, end);
    any_hi = min(any_hi, end);
  }

  f32x16 o[CT];
  float top = kNothing, sum = 0.f;  // the reference of the row's numerators, and their sum in this lane
  uint64_t based = 0;  // lanes whose reference has a base
  lds_base[wave * 32 + m] = 0.f;
  uint32_t poisoned = 0;  // groups (bits) whose values the row has seen a NaN in
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[c][j] = 0.f;

  // ---- the steps of 32 tokens of a tile
  const auto key = [&](const char* stage, int st, int k) { return *reinterpret_cast<const h8*>(stage + L::key_at(32 * st + m, 2 * k + half)); };
  const auto value = [&](const char* stage, int st, int j) {  // j: channel tile j % CT of the sixteen tokens j / CT
    return *reinterpret_cast<const h8*>(stage + L::value_at(32 * (j % CT) + m, 4 * st + 2 * (j / CT) + half));
  };
  const auto scores = [&](const char* stage, int st) {
    f32x16 s;
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(key(stage, st, k), q[k], s, 0, 0, 0);
    return s;
  };
  // The numerators' reference: 2^7 below the largest score, moved only when a numerator would pass 2^15.
  const auto refer = [&](f32x16& s, float most) {
    if (rare((based | __ballot(most * scale > top + kMost)) != 0)) {
      float& base = lds_base[wave * 32 + m];
      Reference ref = {top, base};
      const float f = move_reference(ref, max_over_halves(most), scale);
      top = ref.top;
      sum *= f;
#pragma unroll
      for (int c = 0; c < CT; ++c) o[c] *= f;
      base = ref.base;
      based = __ballot(ref.base != 0.f);
    }
    if (rare(based != 0)) {
      const float base = lds_base[wave * 32 + m];
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] -= base;
    }
  };
  const auto largest = [](const f32x16& s) {
    float most = s[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) most = fmaxf(most, s[j]);
    return most;
  };
  // two of a lane's sixteen numerators
  const auto numerators = [&](const f32x16& s, int j, h8 (&p)[2]) {
    // summed as rounded, so that the weights add up to one
    const h2 pair = to_h2(__builtin_amdgcn_exp2f(fmaf(s[j], scale, -top)), __builtin_amdgcn_exp2f(fmaf(s[j + 1], scale, -top)));
    sum = __builtin_amdgcn_fdot2(pair, h2{(_Float16)1.f, (_Float16)1.f}, sum, false);
    p[j / 8][j % 8] = pair.x;
    p[j / 8][j % 8 + 1] = pair.y;
  };
  // A quarter of tile i + 1's way into LDS; the loads of tile i + 2. (Past the last tile: of page 0, into a stage that nobody
  // reads.)
  const auto produce = [&](int quarter, int i, char* stage, uint8_t* flags) {
    const int t2 = begin + (i + 2) * L::kTokens;
    if (quarter == 0) in.template store_keys<0>(stage, e);
    if (quarter == 1) {
      in.template store_keys<1>(stage, e);
      in.load_keys(t2);
    }
    if (quarter == 2) in.template store_values<0>(stage, flags, e);
    if (quarter == 3) {
      in.template store_values<1>(stage, flags, e);
      in.load_values(t2);
      in.pages(t2 + L::kTokens, end);
    }
  };

  saturate_float16(true);
#pragma unroll
  for (int quarter = 0; quarter < 4; ++quarter) produce(quarter, -1, lds[0], lds_flags[0]);
  saturate_float16(false);
  for (int i = 0; i < tiles; ++i) {
    const int t0 = begin + i * L::kTokens, b = i & 1;
    const char* const stage = lds[b];
    char* const next = lds[b ^ 1];
    uint8_t* const next_flags = lds_flags[b ^ 1];
    __syncthreads();
    const uint32_t flag = lane < L::kFlags / 4 ? reinterpret_cast<const uint32_t*>(lds_flags[b])[lane] : 0;
    const bool odd = __any(flag != 0);  // pages or values that are not there
    if (PIPED && t0 >= all_lo && t0 + L::kTokens <= all_hi && !odd) {
      // A step's products one after the other (the next step's scores, then this step's values), each beside a share of what
      // the vector units have to do meanwhile (this step's numerators, then the next tile's way into LDS and the next
      // step's maximum); their operands come from LDS kAhead products before. The order is kept by barriers. The values'
      // products may run with their conversion's mode: where a numerator is NaN, so is the row's sum.
      constexpr int kAhead = 4, PS = 2 * CT, kAll = (ST - 1) * (KS + PS) + PS;
      h8 ring[kAhead];
      const auto fetch = [&](int n) {  // operand n of the tile
        if (n >= kAll) return;
        const int st = n / (KS + PS), j = n % (KS + PS) + (st == ST - 1 ? KS : 0);
        ring[n % kAhead] = j < KS ? key(stage, st + 1, j) : value(stage, st, j - KS);
      };
      f32x16 s = scores(stage, 0);
#pragma unroll
      for (int n = 0; n < kAhead; ++n) fetch(n);
      refer(s, largest(s));
      h8 p[2];
#pragma unroll
      for (int st = 0; st < ST; ++st) {
        const bool more = st + 1 < ST;
        const int n0 = st * (KS + PS);
        f32x16 s_next;
#pragma unroll
        for (int j = 0; j < 16; ++j) s_next[j] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if (more) {
            s_next = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[(n0 + k) % kAhead], q[k], s_next, 0, 0, 0);
            fetch(n0 + k + kAhead);
          }
#pragma unroll
          for (int j = 16 * k / KS; j < 16 * (k + 1) / KS; j += 2) numerators(s, j, p);
          if (more) __builtin_amdgcn_sched_barrier(0);
        }
        float most = -__builtin_inff();
        saturate_float16(true);
#pragma unroll
        for (int j = 0; j < PS; ++j) {
          const int n = n0 + (more ? KS : 0) + j;
          o[j % CT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[n % kAhead], p[j / CT], o[j % CT], 0, 0, 0);
          fetch(n + kAhead);
          if (j == 0) {
#pragma unroll
            for (int k = 4 * st / ST; k < 4 * (st + 1) / ST; ++k) produce(k, i, next, next_flags);
          }
          if (more && j >= PS / 2) {
#pragma unroll
            for (int k = 32 * j / PS - 16; k < 32 * (j + 1) / PS - 16; ++k) most = fmaxf(most, s_next[k]);
          }
          if (j >= PS / 2) __builtin_amdgcn_sched_barrier(0);
        }
        saturate_float16(false);
        if (more) {
          s = s_next;
          refer(s, most);
        }
      }
      continue;
    }
    // ---- tiles that some of the wave's rows see in part
    saturate_float16(true);
#pragma unroll
    for (int k = 0; k < 4; ++k) produce(k, i, next, next_flags);
    saturate_float16(false);
#pragma unroll 1
    for (int st = 0; st < ST; ++st) {
      const int t1 = t0 + 32 * st;
      if (t1 >= any_hi || t1 + 32 <= any_lo) continue;
      f32x16 s = scores(stage, st);
      if (t1 < all_lo || t1 + 32 > all_hi) {
        asm volatile("");  // a branch, not selects in every step
        const int from = lo - t1 - 4 * half, to = hi - t1 - 4 * half;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (8 * (j / 4) + j % 4 < from || 8 * (j / 4) + j % 4 >= to) s[j] = -__builtin_inff();
      }
      if (rare(odd)) {
        asm volatile("");
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int at = t1 + 4 * half + 8 * (j / 4) + j % 4;
          const uint8_t* flags = &lds_flags[b][8 * st + 4 * (j / 8) + 2 * half + j / 4 % 2];
          const bool seen = at >= lo && at < hi && !(flags[0] & 16);
          if (!seen) s[j] = -__builtin_inff();
#pragma unroll
          for (int c = 0; c < (HD + 127) / 128; ++c)
            if (seen && (flags[c * L::kQuads] >> (j % 4) & 1)) poisoned |= 1u << c;
        }
      }
      refer(s, largest(s));
      h8 p[2];
#pragma unroll
      for (int j = 0; j < 16; j += 2) numerators(s, j, p);
#pragma unroll
      for (int j = 0; j < 2 * CT; ++j) o[j % CT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(value(stage, st, j), p[j / CT], o[j % CT], 0, 0, 0);
    }
  }

  // ---- results: row 32 c + 8 j + 4 half + k of LDS, register 4 j + k of accumulator c, is eight channels' row (value_row): a
  // lane has them side by side
  const bool final = part < 0;
  const float total = sum_over_halves(sum);
  const auto both = __builtin_amdgcn_permlane32_swap(poisoned, poisoned, false, false);
  poisoned = both[0] | both[1];
  if (r < t.rows) {
    const int token = a.by_group.of(r), of = head * a.group + (r - token * a.group);
    const int64_t slot = (int64_t)part * a.tile_rows + (r - t.row0);
    if (half == 0) {
      const float base = lds_base[wave * 32 + m];
      if (!final) {
        reinterpret_cast<float2*>(a.part_ml)[slot] = make_float2(base != 0.f ? __builtin_nanf("") : top, total);
        if (base != 0.f) reinterpret_cast<float2*>(a.part_base)[slot] = make_float2(base, lds_scale[wave * 32 + m]);
      } else if (a.lse) {
        a.lse[(int64_t)(t.token0 + token) * a.n_heads + of] = log_of_sum({top, base}, lds_scale[wave * 32 + m], total);
      }
    }
    const float inv = final ? (total == 0.f ? 0.f : 1.f / total) : 1.f;
    constexpr int kOct = HD / 8;  // rows of the channels 8 i + 0
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) {  // the lane's groups of eight channels: row 8 (i / 4) + 4 half + i % 4 of them
      const int octet = 8 * (i / 4) + 4 * half + i % 4, channel = 8 * octet;
      if (channel >= a.c.head_dim) continue;
      const float nan = (poisoned >> (channel / 128)) & 1 ? __builtin_nanf("") : 0.f;
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int row = k * kOct + 8 * (i / 4);  // without half and i % 4
        y[k] = fmaf(o[row / 32][row % 32 / 8 * 4 + i % 4], inv, nan);
      }
      if (!final) {
        f32x4* to = reinterpret_cast<f32x4*>(a.part_o + slot * a.c.head_dim + channel);
        to[0] = f32x4{y[0], y[1], y[2], y[3]};
        to[1] = f32x4{y[4], y[5], y[6], y[7]};
        continue;
      }
      const int64_t to = (int64_t)(t.token0 + token) * a.out.ld + (int64_t)of * a.out.ld_head + channel;
      store4<BF16>(a, to, {y[0], y[1], y[2], y[3]});
      store4<BF16>(a, to + 4, {y[4], y[5], y[6], y[7]});
    }
  }
  });
}

template <int HD, int WAVES>
void launch(const AttnArgs& a, bool bf16, hipStream_t stream) {
  static_assert(prompt_rows(HD) == 32 * WAVES, "rows of a block");
  const dim3 grid = attention_grid(a);
  if (a.n_blocks) {
    if (bf16) prompt_kernel<HD, WAVES, true, true><<<grid, WAVES * 64, 0, stream>>>(a);
    else prompt_kernel<HD, WAVES, false, true><<<grid, WAVES * 64, 0, stream>>>(a);
  } else {
    if (bf16) prompt_kernel<HD, WAVES, true, false><<<grid, WAVES * 64, 0, stream>>>(a);
    else prompt_kernel<HD, WAVES, false, false><<<grid, WAVES * 64, 0, stream>>>(a);
  }
}

}  // namespace

hipError_t launch_kv4_prompt(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (a.c.head_dim <= 64) launch<64, 8>(a, bf16, stream);
  else if (a.c.head_dim <= 128) launch<128, 8>(a, bf16, stream);
  else launch<256, 4>(a, bf16, stream);
  return hipGetLastError();
}

}  // namespace awq
