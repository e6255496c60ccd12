// The main loop of the W4A16 tile kernels (one weight matrix: w4a16.hip; one per expert:
// w4a16_grouped.hip): a tile of tokens x 256 outputs with the weight operand produced in LDS.
//
// The error GEMM's tiling: four waves, each 128 tokens x 32 FN outputs as 4 x FN accumulators of
// v_mfma_f32_32x32x16_{bf16,f16}; FN = 4: 2 x 2 waves, 256 tokens; FN = 2: 1 x 4 waves, 128 tokens. A K
// step is 64 values of the contraction: the activations (128 bytes of each token's row) move global -> LDS
// by buffer DMA, and the weights are dequantized by the block's threads into the same swizzled LDS layout
// (64 values each), so every weight is dequantized once per tile of tokens. Two LDS stages: the activations of
// step kt+2 are loaded into the stage step kt has just freed, and its weights dequantized there, spread over
// the four sub-steps that follow; each step's codes are requested a step before their dequantization begins.
#pragma once

#include <type_traits>

#include "w4a16_device.h"

namespace awq {

constexpr int kTileTok = 256, kTileRows = 256, kTileKB = 128;
constexpr int kTileStage = (kTileTok + kTileRows) * kTileKB;  // 64 KiB

// The activations of a tile: `rsrc` starts at its first token's row and ends with its last one's, so that
// tokens past the end read as zero (their rows are not stored).
struct TileTokens {
  i32x4 rsrc;
  int row_bytes;
};

// Weights of the forward product: thread t of the block dequantizes output row t of the tile, which lies at
// the byte offsets c_off, s_off and z_off of the descriptors (the offset is what their range check covers:
// a row past the end reads zeros). Sixteen-byte chunk c of an LDS row holds inputs 8 c .. 8 c + 7 of the step.
template <int KIND>
struct RowWeights {
  __amdgpu_buffer_rsrc_t cr, sr, zr;
  int c_off, s_off, z_off;
  uint4 cw[2][2];         // codes of two K steps (64 each) in flight / in use
  uint32_t sw[2], zw[2];  // their group's raw float16 step and zero-point byte
  float gst[2], gnzs[2];  // the group's step and -zero * step for the step whose codes are in set 0 / 1
  uint32_t dlo, dhi, dq[4];
  float dv[4];

  __device__ __forceinline__ RowWeights(__amdgpu_buffer_rsrc_t c, __amdgpu_buffer_rsrc_t s, __amdgpu_buffer_rsrc_t z,
                                        int co, int so, int zo)
      : cr(c), sr(s), zr(z), c_off(co), s_off(so), z_off(zo), dlo(0), dhi(0) {}
  static constexpr bool kEvenSteps = true;  // d_in is a multiple of 128
  static __device__ __forceinline__ int swizzle(int row) { return swz(row); }
  static __device__ __forceinline__ int block_of(int step, int) { return step; }
  __device__ __forceinline__ void load(int set, int step, int) {
    cw[set][0] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(cr, c_off, step * 32, 0));
    cw[set][1] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(cr, c_off + 16, step * 32, 0));
    sw[set] = __builtin_amdgcn_raw_buffer_load_b16(sr, s_off, (step >> 1) * 2, 0);
    zw[set] = __builtin_amdgcn_raw_buffer_load_b8(zr, z_off, step >> 2, 0);
  }
  __device__ __forceinline__ void publish(int) {}
  __device__ __forceinline__ void published() {}
  __device__ __forceinline__ void params(int set, int step) {
    tile_group_params(sw[set], zw[set], step >> 1, gst[set], gnzs[set]);
  }
  __device__ __forceinline__ uint32_t code_word(int set, int c) const {
    const uint4 u = cw[set][c >> 2];
    return (c & 3) == 0 ? u.x : (c & 3) == 1 ? u.y : (c & 3) == 2 ? u.z : u.w;
  }
  __device__ __forceinline__ uint4* place(char* stage, int c) const {
    return reinterpret_cast<uint4*>(stage + kTileTok * kTileKB + (int)threadIdx.x * kTileKB +
                                    ((c ^ swz((int)threadIdx.x)) << 4));
  }
  __device__ __forceinline__ void chunk(char* stage, int set, int c) const {
    *place(stage, c) = dequant8_bytes<KIND>(code_word(set, c), gst[set], gnzs[set]);
  }
  // a chunk as a pipeline of eight parts of at most four VALU instructions, one part after each MFMA: the parts'
  // dependency chains span several MFMAs instead of stalling the issue of the next one; part 7 writes the
  // chunk to LDS
  __device__ __forceinline__ void part(char* stage, int set, int c, int m) {
    const float st = gst[set], nzs = gnzs[set];
    if (m == 0) {
      const uint32_t wd = code_word(set, c);
      dlo = wd & 0x0F0F0F0Fu;
      dhi = (wd >> 4) & 0x0F0F0F0Fu;
    } else if (m == 1) {
      dv[0] = fmaf(ubyte_f32<0>(dlo), st, nzs);
      dv[1] = fmaf(ubyte_f32<0>(dhi), st, nzs);
    } else if (m == 2) {
      dq[0] = pack2(dv[0], dv[1], KIND);
      dv[2] = ubyte_f32<1>(dlo);
      dv[3] = ubyte_f32<1>(dhi);
    } else if (m == 3) {
      dq[1] = pack2(fmaf(dv[2], st, nzs), fmaf(dv[3], st, nzs), KIND);
    } else if (m == 4) {
      dv[0] = fmaf(ubyte_f32<2>(dlo), st, nzs);
      dv[1] = fmaf(ubyte_f32<2>(dhi), st, nzs);
    } else if (m == 5) {
      dq[2] = pack2(dv[0], dv[1], KIND);
      dv[2] = ubyte_f32<3>(dlo);
      dv[3] = ubyte_f32<3>(dhi);
    } else if (m == 6) {
      dq[3] = pack2(fmaf(dv[2], st, nzs), fmaf(dv[3], st, nzs), KIND);
    } else {
      *place(stage, c) = make_uint4(dq[0], dq[1], dq[2], dq[3]);
    }
  }
};

// acc[i][j], element e, in lane l: token 32 i + 8 (e / 4) + 4 (l / 32) + e % 4 of the wave's 128, output
// 32 j + l % 32 of its 32 FN. Wave w covers tokens from 128 (w / (8 / FN)) and outputs from
// 32 FN (w % (8 / FN)). Step s takes block W::block_of(s, k_steps) of the contraction; `first_by_hand`: the
// activations of step 0 are in stage 0 already (written by this block's threads).
template <int KIND, int FN, typename W>
__device__ __forceinline__ void w4a16_tile_loop(const TileTokens& tok, W& w, int k_steps, bool first_by_hand, char* lds,
                                                f32x16 (&acc)[4][FN]) {
  constexpr int FM = 4, NR = FM + FN, KB = kTileKB, BM = kTileTok, WN = 8 / FN, N = FM * FN;
  constexpr int kLoads = FN * 2;  // activation loads of a wave: 32 rows each over the four waves
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // activations: DMA load j of wave w covers token rows (4 j + w) * 8 .. + 7
  int voff_a[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int row = (4 * j + wave) * 8 + (lane >> 3);
    voff_a[j] = row * tok.row_bytes + (((lane & 7) ^ W::swizzle(row)) << 4);
  }
  const uint32_t lds_base = __builtin_amdgcn_readfirstlane(lds_address(lds));
  auto dma_a = [&](uint32_t stage, int j, int kstep) {
    dma_load16(tok.rsrc, __builtin_amdgcn_readfirstlane(stage + (4 * j + wave) * 8 * KB), voff_a[j], W::block_of(kstep, k_steps) * KB);
  };

  const int wm = wave / WN, wn = wave % WN;
  const int fr = lane & 31, fh = lane >> 5;
  const int ra_off = (wm * 128 + fr) * KB;
  const int rb_off = BM * KB + (wn * 32 * FN + fr) * KB;
  int slot[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) slot[q] = ((2 * q + fh) ^ W::swizzle(fr)) << 4;
  auto frag = [&](const char* stage, int sl, int r) -> uint4 {
    const int off = r < FM ? ra_off + r * 32 * KB : rb_off + (r - FM) * 32 * KB;
    return *reinterpret_cast<const uint4*>(stage + off + sl);
  };
  // one sub-step: N MFMAs on `use` while the next sub-step's fragments are read (if `reads`), and aux(0) ..
  // aux(15) spread behind them: each at most one load, one LDS write or a part of a chunk's dequantization
  auto substep = [&](auto zc, const uint4 (&use)[NR], uint4 (&nxt)[NR], const char* src, int sl, bool reads,
                     auto aux) {
    constexpr bool ZC = decltype(zc)::value;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      mma32<KIND, ZC>(use[i / FN], use[FM + i % FN], acc[i / FN][i % FN]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = i * 16 / N; s < (i + 1) * 16 / N; ++s) aux(s);
      if (reads && (N == 16 ? i % 2 == 0 : i < NR)) {
        constexpr int per = N == 16 ? 2 : 1;
        nxt[i / per] = frag(src, sl, i / per);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const std::false_type acc_in{};
  const std::true_type acc_zero{};
  auto none = [](int) {};

  // prologue: stage 0 (activations and weights) into buffer 0; stage 1's activations and the first
  // half of its weights into buffer 1 (the second half is done by step 0's first two sub-steps); the
  // codes of step 2 requested
  char* const buf[2] = {lds, lds + kTileStage};
  const uint32_t bufa[2] = {lds_base, lds_base + kTileStage};
  if (!first_by_hand) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) dma_a(bufa[0], j, 0);
  }
  w.load(0, 0, k_steps);
  w.load(1, min(1, k_steps - 1), k_steps);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  w.publish(0);
  w.publish(1);
  w.published();
  w.params(0, 0);
#pragma unroll
  for (int c = 0; c < 8; ++c) w.chunk(buf[0], 0, c);
#pragma unroll
  for (int j = 0; j < kLoads; ++j) dma_a(bufa[1], j, min(1, k_steps - 1));
  w.params(1, 1);
#pragma unroll
  for (int c = 0; c < 4; ++c) w.chunk(buf[1], 1, c);
  // (past the last step the last step's codes are loaded again and not used: the loads stay
  // unconditional, so no register is carried around the loop by a branch and copied while in flight)
  w.load(0, min(2, k_steps - 1), k_steps);
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  __syncthreads();
  uint4 f0[NR], f1[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) f0[r] = frag(buf[0], slot[0], r);
  substep(acc_zero, f0, f1, buf[0], slot[1], true, none);

  // step kt: B C | barrier | D A'. The weights of step kt+1 are finished (chunks 4..7) in B and C,
  // into its stage (read only after the barrier); D loads the activations of step kt+2 into the stage
  // of step kt (freed by the barrier), and D and A' dequantize chunks 0..3 of step kt+2's weights into
  // it; A' requests the codes of step kt+3 (into the register set B and C have just finished with).
  // Codes are thus requested before the barrier that precedes their first use, whose wait covers
  // them: the load counter completes in issue order, so a wait for codes requested after an
  // activation DMA would also wait for that DMA, long before its barrier needs it.
  // The parity of kt (buffer and codes register set) is a template argument: register arrays indexed
  // at run time would be placed in scratch memory.
  auto step = [&](int kt, auto parity) {
    constexpr int P = decltype(parity)::value;
    char* cur = buf[P];
    char* nxt = buf[P ^ 1];
    const bool pre2 = kt + 2 < k_steps;
    // B chunks 4, 5 and C chunks 6, 7 of step kt+1
    substep(acc_in, f1, f0, cur, slot[2], true, [&](int i) { w.part(nxt, P ^ 1, 4 + (i >> 3), i & 7); });
    substep(acc_in, f0, f1, cur, slot[3], true, [&](int i) { w.part(nxt, P ^ 1, 6 + (i >> 3), i & 7); });
    w.publish(P);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    // D: step kt+2's activations into the freed stage (a load per pair of MFMAs) and its weight
    // chunks 0, 1; A': the codes of step kt+3 and chunks 2, 3
    substep(acc_in, f1, f0, nxt, slot[0], true, [&](int i) {
      if (pre2 && (i & 1) == 0 && (i >> 1) < kLoads) dma_a(bufa[P], i >> 1, kt + 2);
      if (pre2 && i == 0) w.params(P, kt + 2);
      if (pre2) w.part(cur, P, i >> 3, i & 7);
    });
    substep(acc_in, f0, f1, nxt, slot[1], true, [&](int i) {
      if (i == 0) w.load(P ^ 1, min(kt + 3, k_steps - 1), k_steps);
      if (pre2) w.part(cur, P, 2 + (i >> 3), i & 7);
    });
  };
  const std::integral_constant<int, 0> even{};
  const std::integral_constant<int, 1> odd{};
  // steps 0 .. k_steps - 2 in pairs (and one), then the last one: B C D
  auto last = [&](const char* cur) {
    substep(acc_in, f1, f0, cur, slot[2], true, none);
    substep(acc_in, f0, f1, cur, slot[3], true, none);
    substep(acc_in, f1, f0, cur, slot[0], false, none);
  };
  int kt = 0;
  for (; kt + 2 < k_steps - 1; kt += 2) {
    step(kt, even);
    step(kt + 1, odd);
  }
  if constexpr (W::kEvenSteps) {
    step(kt, even);
    last(buf[1]);
  } else {
    if (k_steps > 1) {
      step(kt, even);
      step(kt + 1, odd);
    }
    last(buf[0]);
  }
}

}  // namespace awq
