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

template <int KIND, typename OutT>
hipError_t launch_forward(const GroupedArgs& a, hipStream_t st) {
  const bool gate = a.mode != AWQ_GROUPED_PLAIN;
  const int width = gate ? a.d_out / 2 : a.d_out;
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
