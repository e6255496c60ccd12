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

// act(g) * u in float32
__device__ __forceinline__ float gated(float g, float u, int mode) {
  const float a = mode == AWQ_GROUPED_GATED_SILU ? g / (1.0f + __expf(-g)) : (g <= 0.0f ? 0.0f : g);  // NaN stays
  return a * u;
}

// ---------------------------------------------------------------- a handful of rows per expert

// Up to 16 rows of one expert against all of its weights, read once at the memory's rate. The tile's rows lie in
// LDS whole, brought there by DMA. A wave multiplies 32 output rows (GATED: 16 of the gate and 16 of the up
// matrix) by every KS-th chunk of 8 groups: it keeps the codes of kRing groups in flight in registers, and one load
// brings a row's eight steps. With the rows in LDS the codes are the only loads that a wave waits for (the counter
// of outstanding loads completes in issue order, so a load of activations behind codes would wait for these too),
// and no load sits behind a branch, where the compiler would wait for it at once. The KS waves' partial products
// are added at the end, in wave order. Bound by the latency of its loads and the ramp of a short kernel: one token's gate
// and up products of 2 of 8 experts of 4096 x 22016 take 25 us (3.7 TB/s; one wave over the whole contraction 37) with the
// VALU 45 % busy, the matrix units 7 % and 1.01 times the bytes fetched past L2; 48 tokens' of 4 of 32 experts of
// 2048 x 2048 take 20 - 21 with 37 %, 6 % and 1.1 times.
constexpr int kRing = 2;
constexpr int kChunkGroups = 8;
constexpr int kStreamWaves = 4;
constexpr int kStreamLds = 64 << 10;  // bytes of rows in LDS: two blocks on a compute unit

// Rows of d_in inputs that a tile holds in LDS.
int stream_rows(int d_in) {
  const int rows = kStreamLds / (2 * d_in);
  return rows < 16 ? rows : 16;
}

struct __attribute__((packed, aligned(2))) Steps8 {
  uint32_t s[4];
};
struct __attribute__((packed, aligned(1))) Zeros8 {
  uint32_t z;
};

// A lane's place in one expert's export: its part (kq = lane / 16) of the codes of two output rows, one of each tile
// of 16, and their steps and zero points, eight groups at a time.
struct LaneRows {
  const uint8_t* codes;
  const uint16_t* steps;
  const uint8_t* zeros;
  int G, GZ, last_s, last_z;
  int row[2];
  uint32_t coff[2];
  struct Params {
    Steps8 s[2];
    Zeros8 z[2];
  };
  // col0: the first column of y; GATED: row 0 of the gate, row 1 of the up matrix
  template <bool GATED>
  __device__ __forceinline__ void init(const GroupedArgs& a, int expert, int col0) {
    const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
    const int width = GATED ? a.d_out / 2 : a.d_out;
    G = a.d_in / kGroup;
    GZ = (G + 1) / 2;
    const int64_t row_e = (int64_t)expert * a.d_out, rest = (int64_t)(a.n_experts - expert) * a.d_out;
    codes = a.codes + row_e * (a.d_in / 2);
    steps = a.steps + row_e * G;
    zeros = a.zeros + row_e * GZ;
    // the last places from which a load of eight does not pass the tensor's end
    last_s = (int)min(rest * G - 8, (int64_t)0x7FFFFFFF);
    last_z = (int)min(rest * GZ - 4, (int64_t)0x7FFFFFFF);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      row[j] = min(col0 + (GATED ? 0 : 16 * j) + n, width - 1) + (GATED ? j * width : 0);
      coff[j] = (uint32_t)row[j] * (uint32_t)(a.d_in / 2) + kq * 16;
    }
  }
  __device__ __forceinline__ void load_codes(int g, uint4 (&c)[2]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      c[j] = *reinterpret_cast<const uint4*>(codes + (int64_t)g * (kGroup / 2) + coff[j]);
  }
  // of groups g0 .. g0 + 7; what lies behind the row's last group is not used
  __device__ __forceinline__ void load_params(int g0, Params& p) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p.s[j] = *reinterpret_cast<const Steps8*>(steps + min(row[j] * G + g0, last_s));
      p.z[j] = *reinterpret_cast<const Zeros8*>(zeros + min(row[j] * GZ + (g0 >> 1), last_z));
    }
  }
  // moves the elements of a load that started early, at the tensor's end, to their places
  __device__ __forceinline__ void place_params(int g0, Params& p) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int ls = max(row[j] * G + g0 - last_s, 0), lz = max(row[j] * GZ + (g0 >> 1) - last_z, 0);
      if (__ballot(ls | lz)) {
        for (int k = 0; k < ls; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) p.s[j].s[i] = (p.s[j].s[i] >> 16) | (i < 3 ? p.s[j].s[i + 1] << 16 : 0u);
        }
        p.z[j].z >>= 8 * lz;
      }
    }
  }
  // the constants of group u of eight, row j
  static __device__ __forceinline__ MixParams mix(const Params& p, int j, int u) {
    const float st = (float)__builtin_bit_cast(_Float16, (uint16_t)(p.s[j].s[u / 2] >> (16 * (u & 1))));
    const int z = (p.z[j].z >> (4 * u)) & 15;
    return {st, -(float)(1024 + z) * st, st * 0.0625f, -(float)(64 + z) * st};
  }
};

// Stores a wave's 16 MT rows x 32 output rows (GATED: x 16 columns) from row r0 of the tile on.
template <int KIND, typename OutT, bool GATED, int MT>
__device__ __forceinline__ void store_rows(const GroupedArgs& a, const RowTile& t, int col0, const f32x4 (&acc)[MT][2]) {
  const int lane = threadIdx.x & 63, n = lane & 15, kq = lane >> 4;
  const int width = GATED ? a.d_out / 2 : a.d_out;
  OutT* y = (OutT*)a.y.p + (int64_t)t.row0 * a.y.ld;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < (GATED ? 1 : 2); ++j) {
      const int c = col0 + 16 * j + n;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * m + 4 * kq + i;
        const float v = GATED ? gated(acc[m][0][i], acc[m][1][i], a.mode) : acc[m][j][i];
        if (c < width && r < t.rows) y[(int64_t)r * a.y.ld + c] = to_out<OutT>(v, KIND);
      }
    }
}

template <int KIND, typename OutT, bool GATED, int KS>
__global__ __launch_bounds__(64 * kStreamWaves, 5) void grouped_stream_kernel(GroupedArgs a, int tile_rows) {
  constexpr int W = kStreamWaves, CI = W / KS;  // columns of 32 output rows per block
  constexpr int D = kRing, C = kChunkGroups;
  extern __shared__ __attribute__((aligned(1024))) char xs[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, tile_rows, blockIdx.y, t)) return;
  const int n = lane & 15, kq = lane >> 4;
  const int ks = wave % KS, item = blockIdx.x * CI + wave / KS;
  const int G = a.d_in / kGroup, col0 = item * (GATED ? 16 : 32);

  // the rows on their way to LDS, row after row in 16-byte chunks; the 16 chunks of a group's slice XOR-swizzled by
  // the row, so that 16 lanes that read one chunk of 16 rows find distinct banks
  {
    const int row_chunks = a.d_in / 8, all = t.rows * row_chunks, row_bytes = (int)a.x.ld * 2;
    const uint32_t inverse = ((1u << 24) + row_chunks - 1) / row_chunks;  // p / row_chunks for p < 4096, exactly
    const i32x4 xr = make_rsrc((const uint16_t*)a.x.p + (int64_t)t.row0 * a.x.ld,
                               (uint32_t)(t.rows - 1) * (uint32_t)row_bytes + (uint32_t)a.d_in * 2u);
    const uint32_t base = lds_address(xs);
    for (int p0 = wave * 64; p0 < all; p0 += 64 * W) {
      const int p = p0 + lane, r = (int)(__umul24(p, inverse) >> 24);  // r == rows past the last: out of range, zeros
      const int s = p - r * row_chunks;
      dma_load16(xr, __builtin_amdgcn_readfirstlane(base + p0 * 16),
                 r * row_bytes + ((s & ~15) | ((s ^ r) & 15)) * 16, 0);
    }
  }

  LaneRows w;
  w.init<GATED>(a, t.expert, col0);
  // this wave's groups: every KS-th chunk of C, the last chunk possibly short; a wave without any reads group 0
  const int chunks = (G + C - 1) / C;
  const int mine = chunks > ks ? (chunks - ks + KS - 1) / KS : 0;
  const bool has_last = mine > 0 && (chunks - 1) % KS == ks;
  const int n_groups = mine * C - (has_last ? chunks * C - G : 0);
  auto group_of = [&](int i) { return (ks + (i / C) * KS) * C + i % C; };
  uint4 cw[D][2];
  auto load_codes = [&](int u, int i) {  // past the last group it is read again, and not used
    w.load_codes(min(group_of(max(min(i, n_groups - 1), 0)), G - 1), cw[u]);
  };
  LaneRows::Params pr, pr_next;
  w.load_params(min(ks * C, G - 1), pr);
#pragma unroll
  for (int u = 0; u < D; ++u) load_codes(u, u);
  // the first codes are here: so are this wave's rows, whose loads went out before
  asm volatile("" : "+v"(cw[0][0].x), "+v"(cw[0][1].x)::"memory");
  __syncthreads();

  const uint32_t magic = 0x64006400u;  // float16 1024 in both halves
  const int xrow = min(n, t.rows - 1);
  const char* xl = xs + xrow * a.d_in * 2;
  int slot[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) slot[s] = ((4 * kq + s) ^ (xrow & 15)) << 4;
  f32x4 acc[1][2] = {{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}};
  for (int i0 = 0; i0 < n_groups; i0 += C) {
    const int g0 = (ks + (i0 / C) * KS) * C;
    w.load_params(min(g0 + KS * C, G - 1), pr_next);
    w.place_params(g0, pr);
    const char* xc = xl + g0 * (kGroup * 2);
#pragma unroll
    for (int u = 0; u < C; ++u) {
      if (i0 + u < n_groups) {  // wave-uniform
        uint4 x[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = *reinterpret_cast<const uint4*>(xc + u * (kGroup * 2) + slot[s]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const MixParams p = LaneRows::mix(pr, j, u);
          const uint32_t q[4] = {cw[u % D][j].x, cw[u % D][j].y, cw[u % D][j].z, cw[u % D][j].w};
#pragma unroll
          for (int s = 0; s < 4; ++s) acc[0][j] = mma<KIND>(x[s], dequant8_mix<KIND>(q[s], p, magic), acc[0][j]);
        }
      }
      load_codes(u % D, i0 + u + D);
    }
    pr = pr_next;
  }

  if constexpr (KS > 1) {
    __syncthreads();  // the rows have been read: their place takes the partial products
    f32x4* red = reinterpret_cast<f32x4*>(xs);
    red[(wave * 2) * 64 + lane] = acc[0][0];
    red[(wave * 2 + 1) * 64 + lane] = acc[0][1];
    __syncthreads();
    if (ks != 0) return;
#pragma unroll
    for (int k = 1; k < KS; ++k) {
      acc[0][0] += red[((wave + k) * 2) * 64 + lane];
      acc[0][1] += red[((wave + k) * 2 + 1) * 64 + lane];
    }
  }
  store_rows<KIND, OutT, GATED, 1>(a, t, col0, acc);
}

// ---------------------------------------------------------------- some tens of rows per expert

// 16 MT rows of one expert against its weights: each wave streams the codes of 32 output rows (GATED: 16 and 16)
// through registers as above, each dequantized fragment multiplying MT row tiles. The rows come through LDS a group
// (128 inputs) at a time, by DMA two groups ahead into a ring of four stages. Loads complete in issue order, and a
// group's codes are sent for right behind its rows: with the codes in hand, so is the wave's share of the rows. With many
// waves, bound by the memory and the dequantization in turn, then by the matrix instructions and LDS reads beside it: 8
// experts of 4096 x 22016 with 4 rows each take 97 us (4.6 TB/s fetched; VALU 62 % busy), with 32 rows 125 - 131 (3.0 TB/s of
// weights, 370 TFLOP/s; VALU 49 %, matrix units 30 %), with 128 rows 280 - 324. With few, by latency: a group waits for loads
// that were sent for two groups before, 0.8 us a group whatever the rows and columns are: one expert of 11008 x 4096 with 10
// rows takes 70 us (VALU 4 %), of 4096 x 512 with 100 rows 28.
template <int KIND, typename OutT, bool GATED, int W, int MT>
__global__ __launch_bounds__(64 * W) void grouped_mid_kernel(GroupedArgs a) {
  constexpr int C = kChunkGroups, kStages = 4, kStageBytes = 16 * MT * 256;
  __shared__ __attribute__((aligned(1024))) char xs[kStages * kStageBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, 16 * MT, blockIdx.y, t)) return;
  const int n = lane & 15, kq = lane >> 4;
  const int G = a.d_in / kGroup;
  const int col0 = (blockIdx.x * W + wave) * (GATED ? 16 : 32);

  // DMA: wave w brings the kilobytes w, w + W, ... of a stage, four rows each; the 16 chunks of a row's slice are
  // XOR-swizzled by the row. Rows past the tile's last read zeros.
  const int row_bytes = (int)a.x.ld * 2;
  const i32x4 xr = make_rsrc((const uint16_t*)a.x.p + (int64_t)t.row0 * a.x.ld,
                             (uint32_t)(t.rows - 1) * (uint32_t)row_bytes + (uint32_t)a.d_in * 2u);
  constexpr int kLoads = 4 * MT / W > 0 ? 4 * MT / W : 1;
  const bool brings = wave < 4 * MT;
  int voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = 4 * (wave + i * W) + (lane >> 4);
    voff[i] = r * row_bytes + (((lane & 15) ^ (r & 15)) << 4);
  }
  const uint32_t base = lds_address(xs);
  auto bring = [&](int g, int stage) {
    if (brings && g < G) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        dma_load16(xr, __builtin_amdgcn_readfirstlane(base + stage * kStageBytes + (wave + i * W) * 1024), voff[i],
                   g * (kGroup * 2));
    }
  };

  LaneRows w;
  w.init<GATED>(a, t.expert, col0);
  LaneRows::Params pr, pr_next;
  uint4 cw[2][2];
  w.load_params(0, pr);
  bring(0, 0);
  w.load_codes(0, cw[0]);
  bring(1, 1);
  w.load_codes(min(1, G - 1), cw[1]);

  const uint32_t magic = 0x64006400u;  // float16 1024 in both halves
  const char* xl = xs + n * 256;
  int slot[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) slot[s] = ((4 * kq + s) ^ n) << 4;
  f32x4 acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g0 = 0; g0 < G; g0 += C) {
    w.load_params(min(g0 + C, G - 1), pr_next);
    w.place_params(g0, pr);
#pragma unroll
    for (int u = 0; u < C; ++u) {
      if (g0 + u < G) {  // block-uniform
        // the codes of group g0 + u are here, and this wave's rows of it; then every wave's. The stage that the
        // next rows go to was last read two groups ago.
        asm volatile("" : "+v"(cw[u & 1][0].x), "+v"(cw[u & 1][1].x)::"memory");
        __syncthreads();
        uint4 c[2] = {cw[u & 1][0], cw[u & 1][1]};
        bring(g0 + u + 2, (u + 2) & 3);
        w.load_codes(min(g0 + u + 2, G - 1), cw[u & 1]);
        const MixParams p[2] = {LaneRows::mix(pr, 0, u), LaneRows::mix(pr, 1, u)};
        const char* xc = xl + (u & 3) * kStageBytes;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint4 x[MT];
#pragma unroll
          for (int m = 0; m < MT; ++m) x[m] = *reinterpret_cast<const uint4*>(xc + m * 4096 + slot[s]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t q = s == 0 ? c[j].x : s == 1 ? c[j].y : s == 2 ? c[j].z : c[j].w;
            const uint4 b = dequant8_mix<KIND>(q, p[j], magic);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m][j] = mma<KIND>(x[m], b, acc[m][j]);
          }
        }
      }
    }
    pr = pr_next;
  }
  store_rows<KIND, OutT, GATED, MT>(a, t, col0, acc);
}

// ---------------------------------------------------------------- the gradient with respect to the rows

// Lane e of each row of 16 lanes, in all of the row's lanes.
template <int E>
__device__ __forceinline__ float row_bcast(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + E, 0xF, 0xF, false));
}

// Up to some tens of rows per expert: 16 MT rows of d_x x one group's 128 columns per block, whose eight waves take
// every eighth block of 32 output rows o and add their products at the end, in a fixed order. Lane n = l mod 16 of
// lane group kq reads, for each of its eight k = 8 kq + e, the word of row o + k that holds columns 8 n .. 8 n + 7, so
// that its eight column tiles j (column 8 n + j in column place n) each find their eight consecutive k in the lane's
// own registers: the transposition costs no exchange. Lane n also brings the step and zero point of row o + 8 kq + n mod 8,
// which the lanes of its group take from it. Everything for the next block is loaded before this one is multiplied.
// Bound by what comes in past the L2s: 8 experts of 22016 x 4096 with 4 or 32 rows each take 167 - 174 us and fetch 2.3 - 2.5
// times the weights' bytes (870 - 960 MB, 5.1 - 5.7 TB/s), since a block reads 64 of the 128 bytes of a line of codes and 2 of
// one of steps, and the blocks that read the rest lie on other XCDs. The VALU is 37 - 43 % busy, the matrix units 5 - 22 %.
constexpr int kBackwardWaves = 8;

template <int KIND, typename OutT, int MT>
__global__ __launch_bounds__(64 * kBackwardWaves) void grouped_backward_mid_kernel(GroupedArgs a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTile t;
  if (!find_tile(a.offsets, a.n_experts, a.n_rows, 16 * MT, blockIdx.y, t)) return;
  const int G = a.d_in / kGroup, GZ = (G + 1) / 2, row_bytes = a.d_in / 2;
  const int g = blockIdx.x;
  const int n = lane & 15, kq = lane >> 4;
  const ExpertBuffers buf = expert_buffers(a, t.expert);
  const uint16_t* xrow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    xrow[m] = (const uint16_t*)a.x.p + (int64_t)(t.row0 + min(16 * m + n, t.rows - 1)) * a.x.ld + 8 * kq;
  f32x4 acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Block {
    uint32_t w[8], s, z;
    uint4 x[MT];
  };
  // weights of rows past d_out lie past the expert's buffers and read as zero
  auto load_weights = [&](int b, Block& v) {
    const uint32_t at = (uint32_t)(32 * b + 8 * kq) * (uint32_t)row_bytes + (uint32_t)(g * (kGroup / 2) + 4 * n);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v.w[e] = __builtin_amdgcn_raw_buffer_load_b32(buf.codes, (int)(at + (uint32_t)(e * row_bytes)), 0, 0);
    const int o = 32 * b + 8 * kq + (n & 7);
    v.s = __builtin_amdgcn_raw_buffer_load_b16(buf.steps, (o * G + g) * 2, 0, 0);
    v.z = __builtin_amdgcn_raw_buffer_load_b8(buf.zeros, o * GZ + (g >> 1), 0, 0);
  };
  auto load = [&](int b, Block& v) {
    load_weights(b, v);
#pragma unroll
    for (int m = 0; m < MT; ++m) v.x[m] = *reinterpret_cast<const uint4*>(xrow[m] + 32 * b);
  };
  const uint32_t magic = 0x64006400u;  // float16 1024 in both halves
  auto multiply = [&](const Block& v) {
    const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)v.s);
    const float c = -(float)(1024 + ((v.z >> (4 * (g & 1))) & 15)) * s;  // exact, as in MixParams
    const float st[8] = {row_bcast<0>(s), row_bcast<1>(s), row_bcast<2>(s), row_bcast<3>(s),
                         row_bcast<4>(s), row_bcast<5>(s), row_bcast<6>(s), row_bcast<7>(s)};
    const float c0[8] = {row_bcast<0>(c), row_bcast<1>(c), row_bcast<2>(c), row_bcast<3>(c),
                         row_bcast<4>(c), row_bcast<5>(c), row_bcast<6>(c), row_bcast<7>(c)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, and_or(v.w[e] >> (4 * q), 0x000F000Fu, magic));
        lo[e] = fmaf((float)h.x, st[e], c0[e]);
        hi[e] = fmaf((float)h.y, st[e], c0[e]);
      }
      const uint4 bl = make_uint4(pack2(lo[0], lo[1], KIND), pack2(lo[2], lo[3], KIND), pack2(lo[4], lo[5], KIND),
                                  pack2(lo[6], lo[7], KIND));
      const uint4 bh = make_uint4(pack2(hi[0], hi[1], KIND), pack2(hi[2], hi[3], KIND), pack2(hi[4], hi[5], KIND),
                                  pack2(hi[6], hi[7], KIND));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m][q] = mma<KIND>(v.x[m], bl, acc[m][q]);
        acc[m][q + 4] = mma<KIND>(v.x[m], bh, acc[m][q + 4]);
      }
    }
  };
  const int whole = a.d_out / 32;
  Block now, next;
  int b = wave;
  if (b < whole) load(b, now);
  for (; b < whole; b += kBackwardWaves) {
    load(min(b + kBackwardWaves, whole - 1), next);  // past the last one it is read again, and not used
    multiply(now);
    now = next;
  }
  if (b == whole && a.d_out % 32) {  // the block that d_out cuts: what lies behind it in x is not read
    load_weights(b, now);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t q[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (32 * b + 8 * kq + e < a.d_out) q[e >> 1] |= (uint32_t)xrow[m][32 * b + e] << (16 * (e & 1));
      now.x[m] = make_uint4(q[0], q[1], q[2], q[3]);
    }
    multiply(now);
  }
  // waves h .. 2 h - 1 hand their products to waves 0 .. h - 1
  f32x4* const red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int h = kBackwardWaves / 2; h >= 1; h /= 2) {
    if (h < kBackwardWaves / 2) __syncthreads();
    if (wave >= h && wave < 2 * h) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) red[(((wave - h) * MT + m) * 8 + j) * 64 + lane] = acc[m][j];
    }
    __syncthreads();
    if (wave < h) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[m][j] += red[((wave * MT + m) * 8 + j) * 64 + lane];
    }
  }
  if (wave != 0) return;
  OutT* y = (OutT*)a.y.p;
  struct __attribute__((packed, aligned(sizeof(OutT)))) Eight {
    OutT v[8];
  };
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * m + 4 * kq + i;
      Eight o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = to_out<OutT>(acc[m][j][i], KIND);
      if (r < t.rows) *reinterpret_cast<Eight*>(y + (int64_t)(t.row0 + r) * a.y.ld + g * kGroup + 8 * n) = o;
    }
}

// ---------------------------------------------------------------- many rows per expert

constexpr int kTileThreads = 256;

// The tile's rows of x.
__device__ __forceinline__ TileTokens tile_tokens(const GroupedArgs& a, const RowTile& t, int width) {
  const int row_bytes = (int)a.x.ld * 2;
  return {make_rsrc((const uint16_t*)a.x.p + (int64_t)t.row0 * a.x.ld,
                    (uint32_t)(t.rows - 1) * (uint32_t)row_bytes + (uint32_t)width * 2u),
          row_bytes};
}

// 256 rows x 256 output rows of one expert (the tile loop of w4a16_tile.h); a tile of at most 128 rows takes
// the 128-row form, which multiplies half as much. GATED: blocks of 32 output rows alternate between the gate
// and the up matrix (128 columns of y per tile), so that a lane holds both products of its elements. Bound by the
// matrix instructions and what issues beside them: 4096 tokens over 2 of 8 experts of 4096 x 22016, gated, 1.38 - 1.45
// ms (1.03 - 1.07 PFLOP/s).
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
// through LDS, double-buffered. The transposed codes cost more issue slots than the forward kernel's: 4096 tokens over 2
// of 8 experts of 4096 x 22016 take 1.57 - 1.62 ms (0.91 - 0.94 PFLOP/s).
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

// The forward kernels by the rows that an expert has on average (n_rows / n_experts; the split itself is known on
// the device alone, and any split is right with any of them). Measured with 8 experts of 4096 x 22016 (gate and up),
// all of them used, us:
//   rows per expert     1     4    16    32    64   128   256
//   stream             72   108   207   358
//   mid, 1 x 16 rows   72    95   125   192
//   mid, 2 x 16 rows   87   109   113   153
//   mid, 4 x 16 rows  103   122   127   131   192   324   558
//   tile              232   239   242   245   250   335   540
// Where tiles and columns make few waves, the stream kernel's split of the contraction counts more: one token's 2 of
// these 8 experts 26.7 against 32.4, of 11008 x 4096 down projections 15.9 against 50.
// The tile kernel's time is that of one tile's whole contraction as long as its 256 x 256 tiles do not fill the compute
// units; with so few the 64-row kernel's many more blocks are faster. By the outputs in tiles, us, mid 4 / tile:
//   1 expert of 4096 x 1024, 250 rows (4)  43 /  83      8 of 4096 x 4096, 160 rows (80)    79 /  95
//   2 of 4096 x 4096, 250 rows (32)        47 /  87      8 of 4096 x 4096, 250 rows (125)   85 /  94
//   2 of 4096 x 4096, 500 rows (64)        50 /  89      32 of 2048 x 2048, 160 rows (160)  69 /  68
//   8 of 11008 x 1024, 500 rows (64)      128 / 220      8 of 4096 x 4096, 500 rows (250)  158 / 118
constexpr int kTileMinRows = 144;   // tile kernels from here,
constexpr int kTileMinTiles = 128;  // with so many tiles' outputs
constexpr int kMid4MinRows = 24;    // 4 x 16 rows
constexpr int kMid2MinRows = 5;     // 2 x 16 rows
constexpr int64_t kFewWaves = 4096;
// Waves of a 64-row block, which share its rows' loads, by the waves there are (estimated from the average), us with
// 8 / 4 / 2 a block: 8 experts of 4096 x 4096, 250 rows (4096) 88 / 99 / 128, 120 rows (2048) 54 / 52 / 68, 60 rows
// (1024) 50 / 38 / 37; 2 of 4096 x 1024, 120 rows (128) 43 / 32 / 30; 32 of 4096 x 512, 60 rows (512) 46 / 36 / 34, 120
// rows (1024) 48 / 41 / 47.
constexpr int64_t kMidWaves8 = 2048, kMidWaves4 = 512;  // more waves than these: 8, 4 a block

template <int N>
using Int = std::integral_constant<int, N>;

template <int KIND, typename OutT, bool GATED>
hipError_t launch_forward(const GroupedArgs& a, hipStream_t st) {
  const int width = GATED ? a.d_out / 2 : a.d_out;
  const int items = GATED ? (width + 15) / 16 : (width + 31) / 32;  // columns of 32 output rows
  const int64_t used = a.n_rows < a.n_experts ? a.n_rows : a.n_experts;
  auto at_least = [&](int rows) { return a.n_rows >= (int64_t)rows * a.n_experts; };
  // (the small kernels load eight steps at a time: a smaller tensor of steps takes the tile kernel)
  const int tiles_n = GATED ? (width + 127) / 128 : (width + 255) / 256;
  const bool fill = (int64_t)a.n_rows * tiles_n >= (int64_t)kTileMinTiles * kTileTok;
  if ((at_least(kTileMinRows) && fill) || (int64_t)a.n_experts * a.d_out * (a.d_in / kGroup) < 8) {
    const int tiles_m = (int)most_tiles(a.n_rows, a.n_experts, kTileTok);
    return over_tiles((int64_t)tiles_m * tiles_n, [&](int first, dim3 grid) {
      hipLaunchKernelGGL((grouped_tile_kernel<KIND, OutT, GATED>), grid, dim3(kTileThreads), 0, st, a, tiles_m, tiles_n,
                         first);
    });
  }
  const int rows = stream_rows(a.d_in);
  if (rows >= 1 && !at_least(rows + 1) && used * items < kFewWaves) {
    const int chunks = (a.d_in / kGroup + kChunkGroups - 1) / kChunkGroups;
    const int64_t tiles = most_tiles(a.n_rows, a.n_experts, rows);
    const int lds = ((rows < a.n_rows ? rows : a.n_rows) * 2 * a.d_in + 1023) / 1024 * 1024;
    auto go = [&](auto split) {
      constexpr int W = kStreamWaves, KS = decltype(split)::value, CI = W / KS;
      hipLaunchKernelGGL((grouped_stream_kernel<KIND, OutT, GATED, KS>), dim3((items + CI - 1) / CI, (unsigned)tiles),
                         dim3(64 * W), lds > W * 2048 ? lds : W * 2048, st, a, rows);
    };
    if (chunks >= 4) go(Int<4>{});
    else if (chunks >= 2) go(Int<2>{});
    else go(Int<1>{});
    return hipGetLastError();
  }
  auto go = [&](auto waves, auto row_tiles) {
    constexpr int W = decltype(waves)::value, MT = decltype(row_tiles)::value;
    hipLaunchKernelGGL((grouped_mid_kernel<KIND, OutT, GATED, W, MT>),
                       dim3((items + W - 1) / W, (unsigned)most_tiles(a.n_rows, a.n_experts, 16 * MT)), dim3(64 * W), 0,
                       st, a);
  };
  const int64_t waves = used * ((a.n_rows + 64 * used - 1) / (64 * used)) * items;
  if (at_least(kMid4MinRows)) {
    if (waves > kMidWaves8) go(Int<8>{}, Int<4>{});
    else if (waves > kMidWaves4) go(Int<4>{}, Int<4>{});
    else go(Int<2>{}, Int<4>{});
  } else if (at_least(kMid2MinRows)) go(Int<4>{}, Int<2>{});
  else go(Int<4>{}, Int<1>{});
  return hipGetLastError();
}

// The gradient's kernels by the rows per expert. Measured with 8 experts of 22016 x 4096, all of them used, us:
//   rows per expert     4    16    32    64   128   256
//   mid, 1 x 16 rows  169   249   323   456
//   mid, 2 x 16 rows  171   167   277   356   540
//   mid, 4 x 16 rows  159   167   174   322   455   707
//   tile              382   382   383   386   478   522
// The tile kernel's time is a tile's whole contraction as long as its tiles do not fill the compute units; 64 experts
// of 2048 x 2048 with 64 rows each, which do, take it 95 against 124. By the outputs in tiles, us, mid 4 / tile:
//   1 expert of 4096 x 1024, 250 rows (4)  27 /  91      8 of 4096 x 4096, 160 rows (80)     85 / 103
//   2 of 4096 x 4096, 250 rows (32)        32 /  93      8 of 4096 x 4096, 250 rows (125)   113 / 100
//   2 of 4096 x 4096, 500 rows (64)        60 /  96      32 of 2048 x 2048, 160 rows (160)  103 /  69
constexpr int kBackwardTileMinRows = 144;
constexpr int kBackwardTileMinTiles = 96;  // outputs of so many tiles
constexpr int kBackwardTileMinRowsFull = 48;  // where the tiles fill the compute units
constexpr int64_t kFullTiles = 256;
constexpr int kBackwardMid4MinRows = 24;
constexpr int kBackwardMid2MinRows = 10;

template <int KIND, typename OutT>
hipError_t launch_backward(const GroupedArgs& a, hipStream_t st) {
  auto at_least = [&](int rows) { return a.n_rows >= (int64_t)rows * a.n_experts; };
  const int tiles_n = (a.d_in + 255) / 256;
  const int64_t used = a.n_rows < a.n_experts ? a.n_rows : a.n_experts;
  const bool fill = (int64_t)a.n_rows * tiles_n >= (int64_t)kBackwardTileMinTiles * kTileTok;
  if ((at_least(kBackwardTileMinRows) && fill) || (at_least(kBackwardTileMinRowsFull) && used * tiles_n >= kFullTiles)) {
    const int tiles_m = (int)most_tiles(a.n_rows, a.n_experts, kTileTok);
    return over_tiles((int64_t)tiles_m * tiles_n, [&](int first, dim3 grid) {
      if ((a.d_out + 63) / 64 % 2 == 0)
        hipLaunchKernelGGL((grouped_backward_tile_kernel<KIND, OutT, true>), grid, dim3(kTileThreads), 0, st, a, tiles_m,
                           tiles_n, first);
      else
        hipLaunchKernelGGL((grouped_backward_tile_kernel<KIND, OutT, false>), grid, dim3(kTileThreads), 0, st, a,
                           tiles_m, tiles_n, first);
    });
  }
  auto go = [&](auto row_tiles) {
    constexpr int MT = decltype(row_tiles)::value;
    hipLaunchKernelGGL((grouped_backward_mid_kernel<KIND, OutT, MT>),
                       dim3(a.d_in / kGroup, (unsigned)most_tiles(a.n_rows, a.n_experts, 16 * MT)),
                       dim3(64 * kBackwardWaves), MT * 32768, st, a);
  };
  if (at_least(kBackwardMid4MinRows)) go(Int<4>{});
  else if (at_least(kBackwardMid2MinRows)) go(Int<2>{});
  else go(Int<1>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4a16_grouped(const GroupedArgs& a, int kind, bool y_f32, hipStream_t st) {
  auto go = [&](auto k, auto out) {
    constexpr int KIND = decltype(k)::value;
    typedef decltype(out) OutT;
    return a.mode == AWQ_GROUPED_PLAIN ? launch_forward<KIND, OutT, false>(a, st) : launch_forward<KIND, OutT, true>(a, st);
  };
  if (kind == 0) return y_f32 ? go(Int<0>{}, 0.f) : go(Int<0>{}, (uint16_t)0);
  return y_f32 ? go(Int<1>{}, 0.f) : go(Int<1>{}, (uint16_t)0);
}

hipError_t launch_w4a16_grouped_backward(const GroupedArgs& a, int kind, bool y_f32, hipStream_t st) {
  if (kind == 0) return y_f32 ? launch_backward<0, float>(a, st) : launch_backward<0, uint16_t>(a, st);
  return y_f32 ? launch_backward<1, float>(a, st) : launch_backward<1, uint16_t>(a, st);
}

}  // namespace awq
