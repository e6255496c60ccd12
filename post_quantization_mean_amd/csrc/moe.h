// Internal declarations of the mixture-of-experts block (block_norm.hip, moe_route.hip,
// w4a16_grouped.hip), shared with its host-side C ABI (moe_abi.hip). Not part of the public interface
// (include/awq_moe.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace awq {

constexpr int kMaxNormWidth = 32768;

// A matrix argument: a base pointer and a row pitch in elements.
struct Mat {
  void* p;
  int64_t ld;
};
struct CMat {
  const void* p;
  int64_t ld;
};

struct BlockNormArgs {
  CMat y, residual;
  int64_t n;
  int d;
  const void *w_post, *w_pre, *gate;
  int64_t ld_gate;  // 0: one gate row for all tokens
  float res_scale, eps;
};

hipError_t launch_block_norm(const BlockNormArgs& a, int dtype, Mat res_out, Mat h, hipStream_t stream);

// The workspace of the backward pass: row statistics (wide rows), and partial sums over tokens.
size_t block_norm_backward_stats_bytes(int64_t n_tokens, int64_t d);
size_t block_norm_backward_partial_floats(int64_t n_tokens, int64_t d);
hipError_t launch_block_norm_backward(const BlockNormArgs& a, int dtype, CMat d_res, CMat d_h, Mat d_y, Mat d_residual,
                                      float* d_w_post, float* d_w_pre, void* d_gate, int64_t ld_d_gate,
                                      void* stats_space, float* partial_space, hipStream_t stream);

// Blocks of the sort; 1: a single launch without workspace.
int moe_sort_blocks(int64_t n_slots);
hipError_t launch_moe_sort(const void* ids, bool ids64, int n_slots, int n_experts, int32_t* offsets, int32_t* order,
                           int32_t* position, int32_t* counts, hipStream_t stream);

struct RouteArgs {
  int64_t n_tokens;
  int d, top_k, n_rows;
  const int32_t* position;
  const void* ids;  // with scales
  bool ids64;
  const float* scales;
  int n_experts;
  bool stream_out;  // gather, combine's gradient: the rows written are too many for the second-level caches
};
hipError_t launch_moe_gather(const RouteArgs& a, int dtype, CMat x, Mat rows, hipStream_t stream);
// out[t] = sum_j (weights or 1) * (scales or 1) * rows[position]
hipError_t launch_moe_combine(const RouteArgs& a, int dtype, CMat rows, const float* weights, Mat out,
                              hipStream_t stream);
hipError_t launch_moe_combine_backward(const RouteArgs& a, int dtype, CMat d_out, CMat rows, const float* weights,
                                       Mat d_rows, float* d_weights, hipStream_t stream);

struct GroupedArgs {
  CMat x;
  const uint8_t* codes;
  const uint16_t* steps;
  const uint8_t* zeros;
  const int32_t* offsets;
  int n_experts, n_rows, d_in, d_out;
  int mode;  // awq_grouped_mode
  Mat y;
};
// kind 0: bfloat16 operands, 1: float16
hipError_t launch_w4a16_grouped(const GroupedArgs& a, int kind, bool y_f32, hipStream_t stream);
// x: d_y [n_rows, d_out], y: d_x [n_rows, d_in]
hipError_t launch_w4a16_grouped_backward(const GroupedArgs& a, int kind, bool y_f32, hipStream_t stream);

}  // namespace awq
