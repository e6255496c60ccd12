// The experts' products: every row of x times the dequantized 4-bit weights of its own expert, with the
// rows sorted by expert, and the gradient with respect to the rows.
//
// The rows of each expert are known only on the device (offsets), so a launch covers the most row tiles
// that any split of n_rows over the experts can need, and each block finds its expert and rows by a scan
// of the offsets; blocks past the last tile leave at once.
//
// Dequantization, operand layouts and rounding are those of w4a16.hip.
#include "awq_moe.h"
#include "moe.h"
#include "w4a16_device.h"
#include "w4a16_tile.h"

namespace awq {
namespace {

constexpr int kGroup = 128;

// ---------------------------------------------------------------- row tiles

struct RowTile {
  int expert, row0, rows;  // rows row0 .. row0 + rows - 1 of the expert's
};

// Tile `idx` of the experts' rows in tiles of bm rows. Every wave scans the offsets for itself. Offsets are
// clamped to [0, n_rows] and to ascend, so that no caller's value leads out of the rows.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int n_experts, int n_rows, int bm,
                                          int idx, RowTile& t) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int s = 0; s < n_experts; s += 64) {
    int lo = 0, hi = 0;
    if (s + lane < n_experts) {
      lo = min(max(offsets[s + lane], 0), n_rows);
      hi = min(max(offsets[s + lane + 1], lo), n_rows);
    }
    const int mine = (hi - lo + bm - 1) / bm;
    int incl = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(incl, m, 64);
      if (lane >= m) incl += o;
    }
    const uint64_t past = __ballot(base + incl > idx);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = base + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(mine, l);
      const int r0 = __builtin_amdgcn_readlane(lo, l) + (idx - first) * bm;
      t.expert = s + l;
      t.row0 = r0;
      t.rows = min(bm, __builtin_amdgcn_readlane(hi, l) - r0);
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// The most tiles of bm rows that n_rows rows of n_experts experts can take: each expert with rows wastes
// less than one tile.
int64_t most_tiles(int64_t n_rows, int n_experts, int bm) {
  const int64_t used = n_rows < n_experts ? n_rows : n_experts;
  return used + (n_rows - used) / bm;
}

// act(g) * u in float32
__device__ __forceinline__ float gated(float g, float u, int mode) {
  const float a = mode == AWQ_GROUPED_GATED_SILU ? g / (1.0f + __expf(-g)) : (g <= 0.0f ? 0.0f : g);  // NaN stays
  return a * u;
}

// ---------------------------------------------------------------- few rows per expert

constexpr int kSmallWaves = 8;

// 16 MT rows x 16 NT output rows per block; the eight waves take contiguous ranges of the groups and
// their partial products are added in wave order. GATED: tile 0 is of the gate, tile 1 of the up matrix.
template <int KIND, typename OutT, int NT, int MT, bool GATED>
__global__ __launch_bounds__(64 * kSmallWaves) void grouped_small_kernel(GroupedArgs a) {
  static_assert(!GATED || NT == 2, "a gate tile and an up tile");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, 16 * MT, blockIdx.y, t)) return;
  const int n = lane & 15, kq = lane >> 4;
  const int G = a.d_in / kGroup, GZ = (G + 1) / 2;
  const int width = GATED ? a.d_out / 2 : a.d_out;  // of y
  const int col0 = blockIdx.x * (GATED ? 16 : 16 * NT);
  const int g_begin = (G * wave) / kSmallWaves, g_end = (G * (wave + 1)) / kSmallWaves;
  const uint8_t* crow[NT];
  const uint16_t* srow[NT];
  const uint8_t* zrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int c = min(col0 + (GATED ? 0 : 16 * j) + n, width - 1);
    const int64_t row = (int64_t)t.expert * a.d_out + (GATED ? j * width : 0) + c;
    crow[j] = a.codes + row * (a.d_in / 2) + kq * 16;
    srow[j] = a.steps + row * G;
    zrow[j] = a.zeros + row * GZ;
  }
  const uint16_t* xrow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xrow[m] = (const uint16_t*)a.x.p + (int64_t)(t.row0 + min(16 * m + n, t.rows - 1)) * a.x.ld + kq * 32;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g = g_begin; g < g_end; ++g) {
    uint4 cw[NT];
    float st[NT], nzs[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      cw[j] = *reinterpret_cast<const uint4*>(crow[j] + (int64_t)g * (kGroup / 2));
      group_params(srow[j][g], zrow[j][g >> 1], g, st[j], nzs[j]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint4 x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) x[m] = *reinterpret_cast<const uint4*>(xrow[m] + g * kGroup + s * 8);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint32_t w = s == 0 ? cw[j].x : s == 1 ? cw[j].y : s == 2 ? cw[j].z : cw[j].w;
        const uint4 b = dequant8<KIND>(w, st[j], nzs[j]);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][j] = mma<KIND>(x[m], b, acc[m][j]);
      }
    }
  }
  __shared__ f32x4 red[kSmallWaves][MT * NT][64];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave][m * NT + j][lane] = acc[m][j];
  __syncthreads();
  constexpr int kSums = GATED ? MT : MT * NT;
  if (wave < kSums) {
    f32x4 s[GATED ? 2 : 1];
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
      const int at = GATED ? 2 * wave + q : wave;
      s[q] = red[0][at][lane];
#pragma unroll
      for (int w = 1; w < kSmallWaves; ++w) s[q] += red[w][at][lane];
    }
    const int m = GATED ? wave : wave / NT, j = GATED ? 0 : wave % NT;
    const int c = col0 + 16 * j + n;
    OutT* y = (OutT*)a.y.p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * m + 4 * kq + i;
      float v = s[0][i];
      if constexpr (GATED) v = gated(v, s[1][i], a.mode);
      if (c < width && r < t.rows) y[(int64_t)(t.row0 + r) * a.y.ld + c] = to_out<OutT>(v, KIND);
    }
  }
}

// ---------------------------------------------------------------- the gradient with respect to the rows

// 16 MT rows of d_x x one group's 128 columns per wave; the contraction runs over the output rows o. Lane
// n = l mod 16 of lane group kq reads, for each of its eight k = 8 kq + e, the word of row o + k that holds
// columns 8 n .. 8 n + 7, so that its eight column tiles j (column 8 n + j in column place n) each find
// their eight consecutive k in the lane's own registers: the transposition costs no exchange.
template <int KIND, typename OutT, int MT>
__global__ __launch_bounds__(256) void grouped_backward_simple_kernel(GroupedArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, 16 * MT, blockIdx.y, t)) return;
  const int G = a.d_in / kGroup, GZ = (G + 1) / 2;
  const int g = blockIdx.x * 4 + wave;
  if (g >= G) return;
  const int n = lane & 15, kq = lane >> 4;
  const int64_t row_e = (int64_t)t.expert * a.d_out;
  f32x4 acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int o0 = 0; o0 < a.d_out; o0 += 32) {
    uint32_t w[8];
    float st[8], nzs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int o = o0 + 8 * kq + e;
      const int64_t row = row_e + min(o, a.d_out - 1);
      w[e] = *reinterpret_cast<const uint32_t*>(a.codes + row * (a.d_in / 2) + g * (kGroup / 2) + 4 * n);
      group_params(a.steps[row * G + g], a.zeros[row * GZ + (g >> 1)], g, st[e], nzs[e]);
      if (o >= a.d_out) w[e] = 0, st[e] = nzs[e] = 0.f;
    }
    uint4 x[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint16_t* xr = (const uint16_t*)a.x.p + (int64_t)(t.row0 + min(16 * m + n, t.rows - 1)) * a.x.ld;
      const int o = o0 + 8 * kq;
      x[m] = make_uint4(0, 0, 0, 0);
      if (o + 8 <= a.d_out) {
        x[m] = *reinterpret_cast<const uint4*>(xr + o);
      } else if (o < a.d_out) {
        uint32_t q[4] = {0, 0, 0, 0};
        for (int e = 0; o + e < a.d_out; ++e) q[e >> 1] |= (uint32_t)xr[o + e] << (16 * (e & 1));
        x[m] = make_uint4(q[0], q[1], q[2], q[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf((float)((w[e] >> (4 * j)) & 15u), st[e], nzs[e]);
      const uint4 b = make_uint4(pack2(v[0], v[1], KIND), pack2(v[2], v[3], KIND), pack2(v[4], v[5], KIND),
                                 pack2(v[6], v[7], KIND));
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][j] = mma<KIND>(x[m], b, acc[m][j]);
    }
  }
  OutT* y = (OutT*)a.y.p;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * m + 4 * kq + i;
      if (r >= t.rows) continue;
      OutT* yr = y + (int64_t)(t.row0 + r) * a.y.ld + g * kGroup + 8 * n;
#pragma unroll
      for (int j = 0; j < 8; ++j) yr[j] = to_out<OutT>(acc[m][j][i], KIND);
    }
}

// ---------------------------------------------------------------- many rows per expert

constexpr int kTileThreads = 256;
constexpr int64_t kTileMinRows = 64;  // rows per expert, on average, from which the tile kernels are taken

// The tile's rows of x.
__device__ __forceinline__ TileTokens tile_tokens(const GroupedArgs& a, const RowTile& t, int width) {
  const int row_bytes = (int)a.x.ld * 2;
  return {make_rsrc((const uint16_t*)a.x.p + (int64_t)t.row0 * a.x.ld,
                    (uint32_t)(t.rows - 1) * (uint32_t)row_bytes + (uint32_t)width * 2u),
          row_bytes};
}

// The export of one expert as range-checked buffers.
struct ExpertBuffers {
  __amdgpu_buffer_rsrc_t codes, steps, zeros;
};
__device__ __forceinline__ ExpertBuffers expert_buffers(const GroupedArgs& a, int expert) {
  const int G = a.d_in / kGroup, GZ = (G + 1) / 2;
  const int64_t row = (int64_t)expert * a.d_out;
  return {__builtin_amdgcn_make_buffer_rsrc((void*)(a.codes + row * (a.d_in / 2)), (short)0, a.d_out * (a.d_in / 2),
                                            0x00020000),
          __builtin_amdgcn_make_buffer_rsrc((void*)(a.steps + row * G), (short)0, a.d_out * G * 2, 0x00020000),
          __builtin_amdgcn_make_buffer_rsrc((void*)(a.zeros + row * GZ), (short)0, a.d_out * GZ, 0x00020000)};
}

// 256 rows x 256 output rows of one expert (the tile loop of w4a16_tile.h); a tile of at most 128 rows takes
// the 128-row form, which multiplies half as much. GATED: blocks of 32 output rows alternate between the gate
// and the up matrix (128 columns of y per tile), so that a lane holds both products of its elements.
template <int KIND, typename OutT, bool GATED, int FN>
__device__ __forceinline__ void grouped_tile(const GroupedArgs& a, const RowTile& t, int col0, char* lds) {
  const int tid = threadIdx.x;
  const int G = a.d_in / kGroup, GZ = (G + 1) / 2;
  const int width = GATED ? a.d_out / 2 : a.d_out;
  const int c = col0 + (GATED ? (tid >> 6) * 32 + (tid & 31) : tid);
  // this thread's output row; d_out, whose offsets lie past the buffers, where there is none
  const int row = c < width ? (GATED && (tid & 32) ? width + c : c) : a.d_out;
  const ExpertBuffers b = expert_buffers(a, t.expert);
  RowWeights<KIND> weights(b.codes, b.steps, b.zeros, row * (a.d_in / 2), row * G * 2, row * GZ);
  f32x16 acc[4][FN];
  w4a16_tile_loop<KIND, FN>(tile_tokens(a, t, a.d_in), weights, a.d_in / 64, false, lds, acc);

  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / (8 / FN), wn = wave % (8 / FN), fr = lane & 31, fh = lane >> 5;
  OutT* y = (OutT*)a.y.p + (int64_t)t.row0 * a.y.ld;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < FN; j += GATED ? 2 : 1) {
      const int at = col0 + (GATED ? (wn * FN + j) * 16 + fr : (wn * FN + j) * 32 + fr);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = wm * 128 + 32 * i + 8 * (e >> 2) + 4 * fh + (e & 3);
        float v = acc[i][j][e];
        if constexpr (GATED) v = gated(v, acc[i][j + 1][e], a.mode);
        if (r < t.rows && at < width) y[(int64_t)r * a.y.ld + at] = to_out<OutT>(v, KIND);
      }
    }
}

template <int KIND, typename OutT, bool GATED>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grouped_tile_kernel(GroupedArgs a, int tiles_m, int tiles_n, int first) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kTileStage];
  int tm, tn;
  tile_of(first + (int)blockIdx.x, tiles_m, tiles_n, tm, tn);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, kTileTok, tm, t)) return;
  const int col0 = tn * (GATED ? 128 : 256);
  if (t.rows > 128) grouped_tile<KIND, OutT, GATED, 4>(a, t, col0, lds);
  else grouped_tile<KIND, OutT, GATED, 2>(a, t, col0, lds);
}

// Weights of the gradient with respect to the rows: the contraction runs over the output rows o, and an LDS
// row holds one input channel c of the tile's 256. Thread (cq, oo) = (t mod 32, t / 32) dequantizes the 8 x 8
// block of channels 8 cq .. 8 cq + 7 and step rows 8 oo .. 8 oo + 7: it loads, of each of its eight rows, the
// word with its eight channels (128 contiguous bytes per row across the lanes), and its chunk j is the eight
// rows' nibbles of one channel, so the transposition costs nothing but the order of the nibbles. Lanes take the
// channels in different orders (channel j ^ m of chunk j, a shift amount per lane) so that 16 lanes write
// distinct LDS banks. The 64 rows' steps and zero points are prepared once per step by 128 threads and shared
// through LDS, double-buffered.
template <int KIND, bool EVEN>
struct ColumnWeights {
  static constexpr bool kEvenSteps = EVEN;
  __amdgpu_buffer_rsrc_t cr, sr, zr;
  float2 (*shared)[2][64];  // [set][group of the tile][row of the step]: step, -zero * step
  int row_bytes, G, GZ, c_off, g0, m4;
  uint32_t place0;
  uint32_t cw[2][8];
  uint32_t sw[2], zw[2];
  float st[8], nz[8];
  float dv[2];
  uint32_t db[2], dq[4];

  __device__ __forceinline__ ColumnWeights(const ExpertBuffers& b, float2 (*lds)[2][64], int d_in, int col0)
      : cr(b.codes), sr(b.steps), zr(b.zeros), shared(lds) {
    const int cq = threadIdx.x & 31, oo = threadIdx.x >> 5;
    row_bytes = d_in / 2;
    G = d_in / kGroup;
    GZ = (G + 1) / 2;
    g0 = col0 / kGroup;
    c_off = 8 * oo * row_bytes + col0 / 2 + 4 * cq;
    const int m = (((cq >> 2) & 1) << 2) | ((cq >> 3) & 1);
    m4 = 4 * m;
    // channel 8 cq + (j ^ m), chunk oo of its row
    place0 = kTileTok * kTileKB + cq * 1024 + (m << 7) + ((oo ^ m ^ (cq & 3)) << 4);
  }
  static __device__ __forceinline__ int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 3); }
  // the last block, which may be cut by d_out, comes first
  static __device__ __forceinline__ int block_of(int step, int k_steps) { return step == 0 ? k_steps - 1 : step - 1; }
  __device__ __forceinline__ void load(int set, int step, int k_steps) {
    const int o0 = block_of(step, k_steps) * 64;
    const uint32_t at = (uint32_t)(o0 * row_bytes) + (uint32_t)c_off;  // rows past d_out lie past the buffer
#pragma unroll
    for (int e = 0; e < 8; ++e)
      cw[set][e] = __builtin_amdgcn_raw_buffer_load_b32(cr, (int)(at + (uint32_t)(e * row_bytes)), 0, 0);
    const int o = o0 + (threadIdx.x & 63), g = g0 + ((threadIdx.x >> 6) & 1);  // used by threads 0 .. 127
    sw[set] = __builtin_amdgcn_raw_buffer_load_b16(sr, (o * G + g) * 2, 0, 0);
    zw[set] = __builtin_amdgcn_raw_buffer_load_b8(zr, o * GZ + (g >> 1), 0, 0);
  }
  __device__ __forceinline__ void publish(int set) {
    if (threadIdx.x < 128) {
      float s, z;
      tile_group_params(sw[set], zw[set], g0 + (threadIdx.x >> 6), s, z);
      shared[set][threadIdx.x >> 6][threadIdx.x & 63] = make_float2(s, z);
    }
  }
  __device__ __forceinline__ void published() { __syncthreads(); }
  __device__ __forceinline__ void params(int set, int) {
    const float4* p = reinterpret_cast<const float4*>(&shared[set][(threadIdx.x >> 4) & 1][8 * (threadIdx.x >> 5)]);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float4 v = p[e / 2];
      st[e] = v.x, nz[e] = v.y, st[e + 1] = v.z, nz[e + 1] = v.w;
    }
  }
  __device__ __forceinline__ uint32_t nibble(int set, int e, int j) const {
    return __builtin_amdgcn_ubfe(cw[set][e], (uint32_t)((4 * j) ^ m4), 4);
  }
  __device__ __forceinline__ uint4* place(char* stage, int j) const {
    return reinterpret_cast<uint4*>(stage + (place0 ^ (uint32_t)((j << 7) | (j << 4))));
  }
  __device__ __forceinline__ void chunk(char* stage, int set, int j) const {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf((float)nibble(set, e, j), st[e], nz[e]);
    *place(stage, j) = make_uint4(pack2(v[0], v[1], KIND), pack2(v[2], v[3], KIND), pack2(v[4], v[5], KIND),
                                  pack2(v[6], v[7], KIND));
  }
  // a chunk in eight parts, as RowWeights: pair p's nibbles are taken out in part 2 p and multiplied and packed in
  // part 2 p + 1, with the next pair's beginning
  __device__ __forceinline__ void part(char* stage, int set, int j, int m) {
    const int e = m & ~1;
    if ((m & 1) == 0) {
      db[0] = nibble(set, e, j);
      db[1] = nibble(set, e + 1, j);
      dv[0] = ubyte_f32<0>(db[0]);
      dv[1] = ubyte_f32<0>(db[1]);
    } else {
      dq[m >> 1] = pack2(fmaf(dv[0], st[e], nz[e]), fmaf(dv[1], st[e + 1], nz[e + 1]), KIND);
      if (m == 7) *place(stage, j) = make_uint4(dq[0], dq[1], dq[2], dq[3]);
    }
  }
};

template <int KIND, typename OutT, bool EVEN, int FN>
__device__ __forceinline__ void grouped_backward_tile(const GroupedArgs& a, const RowTile& t, int col0, char* lds,
                                                      float2 (*shared)[2][64]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k_steps = (a.d_out + 63) / 64;
  const bool cut = (a.d_out & 63) != 0;
  if (cut) {
    // the last block of the contraction, which comes first, is cut by d_out: its activations are loaded here,
    // zeros past d_out (what lies there in memory is not read)
    const int o0 = (k_steps - 1) * 64;
    for (int j = 0; j < 2 * FN; ++j) {
      const int r = (4 * j + wave) * 8 + (lane >> 3), o = o0 + 8 * ((lane & 7) ^ ColumnWeights<KIND, EVEN>::swizzle(r));
      uint32_t q[4] = {0, 0, 0, 0};
      if (r < t.rows) {
        const uint16_t* p = (const uint16_t*)a.x.p + (int64_t)(t.row0 + r) * a.x.ld + o;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (o + e < a.d_out) q[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
      }
      *reinterpret_cast<uint4*>(lds + (4 * j + wave) * 8 * kTileKB + lane * 16) = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  ColumnWeights<KIND, EVEN> weights(expert_buffers(a, t.expert), shared, a.d_in, col0);
  f32x16 acc[4][FN];
  w4a16_tile_loop<KIND, FN>(tile_tokens(a, t, a.d_out), weights, k_steps, cut, lds, acc);

  const int wm = wave / (8 / FN), wn = wave % (8 / FN), fr = lane & 31, fh = lane >> 5;
  OutT* y = (OutT*)a.y.p + (int64_t)t.row0 * a.y.ld;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int at = col0 + (wn * FN + j) * 32 + fr;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int r = wm * 128 + 32 * i + 8 * (e >> 2) + 4 * fh + (e & 3);
        if (r < t.rows && at < a.d_in) y[(int64_t)r * a.y.ld + at] = to_out<OutT>(acc[i][j][e], KIND);
      }
    }
}

template <int KIND, typename OutT, bool EVEN>
__global__ __launch_bounds__(kTileThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grouped_backward_tile_kernel(GroupedArgs a, int tiles_m, int tiles_n, int first) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kTileStage];
  __shared__ __attribute__((aligned(16))) float2 shared[2][2][64];
  int tm, tn;
  tile_of(first + (int)blockIdx.x, tiles_m, tiles_n, tm, tn);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, kTileTok, tm, t)) return;
  if (t.rows > 128) grouped_backward_tile<KIND, OutT, EVEN, 4>(a, t, tn * 256, lds, shared);
  else grouped_backward_tile<KIND, OutT, EVEN, 2>(a, t, tn * 256, lds, shared);
}

// Launches f(first, blocks) over all tiles; one launch holds at most 2^23 blocks of 256 threads.
template <typename F>
hipError_t over_tiles(int64_t tiles, F f) {
  constexpr int64_t kMost = 1 << 23;
  for (int64_t first = 0; first < tiles; first += kMost) {
    f((int)first, dim3((unsigned)(tiles - first < kMost ? tiles - first : kMost)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int KIND, typename OutT>
hipError_t launch_forward(const GroupedArgs& a, hipStream_t st) {
  const bool gate = a.mode != AWQ_GROUPED_PLAIN;
  const int width = gate ? a.d_out / 2 : a.d_out;
  if (a.n_rows >= kTileMinRows * a.n_experts) {
    const int tiles_m = (int)most_tiles(a.n_rows, a.n_experts, kTileTok);
    const int tiles_n = gate ? (width + 127) / 128 : (width + 255) / 256;
    return over_tiles((int64_t)tiles_m * tiles_n, [&](int first, dim3 grid) {
      if (gate)
        hipLaunchKernelGGL((grouped_tile_kernel<KIND, OutT, true>), grid, dim3(kTileThreads), 0, st, a, tiles_m, tiles_n,
                           first);
      else
        hipLaunchKernelGGL((grouped_tile_kernel<KIND, OutT, false>), grid, dim3(kTileThreads), 0, st, a, tiles_m,
                           tiles_n, first);
    });
  }
  const dim3 block(64 * kSmallWaves);
  const unsigned gy = (unsigned)most_tiles(a.n_rows, a.n_experts, 16);
  if (gate)
    hipLaunchKernelGGL((grouped_small_kernel<KIND, OutT, 2, 1, true>), dim3((width + 15) / 16, gy), block, 0, st, a);
  else
    hipLaunchKernelGGL((grouped_small_kernel<KIND, OutT, 2, 1, false>), dim3((width + 31) / 32, gy), block, 0, st, a);
  return hipGetLastError();
}

template <int KIND, typename OutT>
hipError_t launch_backward(const GroupedArgs& a, hipStream_t st) {
  if (a.n_rows >= kTileMinRows * a.n_experts) {
    const int tiles_m = (int)most_tiles(a.n_rows, a.n_experts, kTileTok), tiles_n = (a.d_in + 255) / 256;
    return over_tiles((int64_t)tiles_m * tiles_n, [&](int first, dim3 grid) {
      if ((a.d_out + 63) / 64 % 2 == 0)
        hipLaunchKernelGGL((grouped_backward_tile_kernel<KIND, OutT, true>), grid, dim3(kTileThreads), 0, st, a, tiles_m,
                           tiles_n, first);
      else
        hipLaunchKernelGGL((grouped_backward_tile_kernel<KIND, OutT, false>), grid, dim3(kTileThreads), 0, st, a,
                           tiles_m, tiles_n, first);
    });
  }
  const unsigned gy = (unsigned)most_tiles(a.n_rows, a.n_experts, 64);
  hipLaunchKernelGGL((grouped_backward_simple_kernel<KIND, OutT, 4>), dim3((a.d_in / kGroup + 3) / 4, gy), dim3(256),
                     0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4a16_grouped(const GroupedArgs& a, int kind, bool y_f32, hipStream_t st) {
  if (kind == 0) return y_f32 ? launch_forward<0, float>(a, st) : launch_forward<0, uint16_t>(a, st);
  return y_f32 ? launch_forward<1, float>(a, st) : launch_forward<1, uint16_t>(a, st);
}

hipError_t launch_w4a16_grouped_backward(const GroupedArgs& a, int kind, bool y_f32, hipStream_t st) {
  if (kind == 0) return y_f32 ? launch_backward<0, float>(a, st) : launch_backward<0, uint16_t>(a, st);
  return y_f32 ? launch_backward<1, float>(a, st) : launch_backward<1, uint16_t>(a, st);
}

}  // namespace awq
