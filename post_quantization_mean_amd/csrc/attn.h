// Internal declarations of attention over the 4-bit cache (rope.hip, kv4_cache.hip, kv4_attention.hip, kv4_prompt.hip), shared with its
// host-side C ABI (attn_abi.hip). Not part of the public interface (include/awq_attn.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace awq {

// A [tokens, heads, channels] argument: pitches in elements.
struct Heads {
  void* p;
  int64_t ld, ld_head;
};
struct CHeads {
  const void* p;
  int64_t ld, ld_head;
};

// Division of 0 <= n < 2^31 by a number known on the host: one multiplication (the quotient of n and the divisor is that of
// n * (2^32 + mul) and 2^(32 + shift)).
struct Divisor {
  uint32_t mul, shift;
  Divisor(uint32_t d = 1) {
    shift = 0;
    while (((uint64_t)1 << shift) < d) ++shift;
    mul = (uint32_t)((((((uint64_t)1 << shift) - d) << 32) / d) + 1);
  }
#ifdef __HIPCC__
  __device__ __forceinline__ int of(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
#endif
};

struct RopeArgs {
  CHeads x;
  Heads out;
  int64_t n_tokens;
  int n_heads, head_dim, rot_dim;
  const void* positions;
  int64_t ld_positions;
  bool pos64;
  int n_axes;
  const float* inv_freq;
  const int32_t* axis;
  float cos_scale, sin_scale;  // sin_scale = -cos_scale: the gradient
  bool in_place;
  Divisor by_heads;  // by n_heads
};
hipError_t launch_rope(const RopeArgs& a, int dtype, bool pairs, hipStream_t stream);

// The cache: pitches from page to page in bytes of codes and in words of params (one word: step, offset).
struct Kv4Cache {
  uint8_t* codes;
  uint32_t* params;
  int64_t page_codes, page_params;
  int64_t n_pages;
  int page_log2, n_kv, head_dim, n_groups;
};

struct Kv4MoveArgs {
  Kv4Cache c;
  const void* slots;
  bool slots64;
  int64_t n_tokens;
};
hipError_t launch_kv4_write(const Kv4MoveArgs& a, int dtype, CHeads k, CHeads v, hipStream_t stream);
hipError_t launch_kv4_read(const Kv4MoveArgs& a, int dtype, Heads k, Heads v, hipStream_t stream);

constexpr int kUnit = 128;  // cached tokens that the split counts in

struct AttnArgs {
  Kv4Cache c;
  CHeads q;
  Heads out;
  bool out_f32;
  float* lse;
  const int32_t *table, *kv_len, *q_offsets;
  int64_t ld_table;
  int table_width, n_seqs, n_heads;
  int64_t n_tokens;
  int group;     // query heads of a key head
  int each;      // new tokens of each sequence where q_offsets is NULL
  float scale;   // times log2(e)
  int causal;
  int window;    // 0: none
  int max_kv;
  // how the work is split (plan_attention)
  int tile_rows;   // (token, head) rows of a key head that a block takes: a power of two
  int tile_log2;
  int n_tiles;     // tiles of rows over all sequences, at most
  int n_blocks;    // 0: a block for each tile and key head; else blocks that share the cached tokens evenly (kv4_device.h)
  Divisor by_group, by_tiles, by_kv;  // by group, by the tiles of each sequence (where q_offsets is NULL), by n_kv
  int* prefix;     // with n_blocks: [n_tiles + 1] (the workspace's start)
  float* part_o;     // [2 n_blocks][tile_rows][head_dim]
  float* part_ml;    // [2 n_blocks][tile_rows][2]: reference (NaN: see part_base) and sum of the numerators
  float* part_base;  // [2 n_blocks][tile_rows][2]: base and scale of the scores
};

// Fills the split from the sizes; returns the workspace's bytes.
size_t plan_attention(AttnArgs* a, bool ragged);
void place_workspace(AttnArgs* a, void* workspace);
// tile_rows of the kernel for prompts
constexpr int prompt_rows(int head_dim) { return head_dim <= 128 ? 256 : 128; }
hipError_t launch_kv4_prompt(const AttnArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_kv4_attention(const AttnArgs& a, bool bf16, hipStream_t stream);

}  // namespace awq
