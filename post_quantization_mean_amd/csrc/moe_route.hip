// Tokens into expert order and back.
//
// Sort: a stable counting sort of the slots by expert. Slots are split into contiguous ranges, one per
// block and within it one per wave; a wave walks its range 64 slots at a time and finds each slot's rank
// among the equal ids of the 64 by matching id bits with ballots, so that counts and places come out the
// same whatever the timing (no global atomics). One block does it all for few slots; more take a counting
// launch and a placing launch, whose blocks each add up the counts of the blocks before them.
//
// Gather and combine are bound by memory: gather reads a token's row once and writes it to its places,
// combine reads the places' rows and writes the token's row once, 16 bytes per lane.
#include "awq_moe.h"
#include "moe.h"
#include "moe_device.h"

namespace awq {
namespace {

// ---------------------------------------------------------------- sort

constexpr int kSortThreads = 256, kSortWaves = kSortThreads / 64;
constexpr int kSortMaxBlocks = 256;
constexpr int kSortSlots = 2048;  // slots of a block, until kSortMaxBlocks would be passed

__device__ __forceinline__ int load_id(const void* ids, bool ids64, int slot, int n_experts) {
  const int64_t v = ids64 ? ((const int64_t*)ids)[slot] : (int64_t)((const int32_t*)ids)[slot];
  return v >= 0 && v < n_experts ? (int)v : n_experts;  // n_experts: dropped
}

// The lanes of the wave whose id equals this lane's.
__device__ __forceinline__ uint64_t same_id(int id, int id_bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < id_bits; ++b) {
    const uint64_t set = __ballot((id >> b) & 1);
    m &= ((id >> b) & 1) ? set : ~set;
  }
  return m;
}

// One wave's slots [begin, end): calls f(slot, id, rank) for each lane's slot, where rank counts the wave's
// earlier slots of the same id, kept in cnt (LDS, one counter per id, this wave's own).
template <typename F>
__device__ __forceinline__ void walk(const void* ids, bool ids64, int begin, int end, int n_experts, int id_bits,
                                     int* cnt, F f) {
  const int lane = threadIdx.x & 63;
  for (int s0 = begin; s0 < end; s0 += 64) {
    const int slot = s0 + lane;
    const bool in = slot < end;
    const int id = in ? load_id(ids, ids64, slot, n_experts) : n_experts;
    const uint64_t same = same_id(id, id_bits);
    const int leader = __ffsll((unsigned long long)same) - 1;
    int base = 0;
    if (lane == leader && id < n_experts) base = atomicAdd(&cnt[id], __popcll(same));
    base = __shfl(base, leader, 64);
    if (in) f(slot, id, base + __popcll(same & ((1ull << lane) - 1)));
  }
}

// blocks == 1: the whole sort. Otherwise PLACE false counts (counts[block][expert]), PLACE true places.
template <bool PLACE>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(const void* ids, bool ids64, int n_slots, int n_experts,
                                                            int id_bits, int slots_per_block, int32_t* counts,
                                                            int32_t* offsets, int32_t* order, int32_t* position) {
  extern __shared__ int lds[];
  int* cnt = lds;                            // [kSortWaves][n_experts]: counts, then each wave's first place
  int* total = lds + kSortWaves * n_experts; // [n_experts]
  __shared__ int wave_total[kSortWaves + 1];
  const int tid = threadIdx.x, wave = tid >> 6, blocks = gridDim.x;
  const int b0 = (int)min((int64_t)blockIdx.x * slots_per_block, (int64_t)n_slots);
  const int b1 = (int)min((int64_t)b0 + slots_per_block, (int64_t)n_slots);
  const int per_wave = (slots_per_block + kSortWaves - 1) / kSortWaves;
  const int w0 = min(b0 + wave * per_wave, b1), w1 = min(w0 + per_wave, b1);
  for (int i = tid; i < kSortWaves * n_experts; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  walk(ids, ids64, w0, w1, n_experts, id_bits, cnt + wave * n_experts, [](int, int, int) {});
  __syncthreads();
  if constexpr (!PLACE) {
    for (int e = tid; e < n_experts; e += kSortThreads) {
      int s = 0;
      for (int w = 0; w < kSortWaves; ++w) s += cnt[w * n_experts + e];
      counts[(int64_t)blockIdx.x * n_experts + e] = s;
    }
    return;
  }
  // the expert's slots in all blocks, and in those before this one
  for (int e = tid; e < n_experts; e += kSortThreads) {
    int before = 0, all = 0;
    if (blocks > 1) {
      for (int b = 0; b < blocks; ++b) {
        const int c = counts[(int64_t)b * n_experts + e];
        before += b < (int)blockIdx.x ? c : 0;
        all += c;
      }
    }
    int run = before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = cnt[w * n_experts + e];
      cnt[w * n_experts + e] = run;
      run += c;
    }
    total[e] = blocks > 1 ? all : run;
  }
  __syncthreads();
  // exclusive scan of the totals: thread t holds experts t * per .. + per - 1
  const int per = (n_experts + kSortThreads - 1) / kSortThreads;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    mine += e < n_experts ? total[e] : 0;
  }
  int incl = mine;
  for (int m = 1; m < 64; m <<= 1) {
    const int o = __shfl_up(incl, m, 64);
    if ((tid & 63) >= m) incl += o;
  }
  if ((tid & 63) == 63) wave_total[wave] = incl;
  __syncthreads();
  int base = incl - mine, kept = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    base += w < wave ? wave_total[w] : 0;
    kept += wave_total[w];
  }
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < n_experts) {
      if (blockIdx.x == 0) offsets[e] = base;
      for (int w = 0; w < kSortWaves; ++w) cnt[w * n_experts + e] += base;
      base += total[e];
    }
  }
  if (blockIdx.x == 0 && tid == 0) offsets[n_experts] = kept;
  __syncthreads();
  walk(ids, ids64, w0, w1, n_experts, id_bits, cnt + wave * n_experts, [&](int slot, int id, int place) {
    position[slot] = id < n_experts ? place : -1;
    if (id < n_experts && place < n_slots) order[place] = slot;
  });
  for (int i = max(b0, kept) + tid; i < b1; i += kSortThreads) order[i] = -1;
}

// ---------------------------------------------------------------- gather, combine

// The multipliers of a slot's expert, or NULL when there are none; `skip`: the id is out of range.
__device__ __forceinline__ const float* slot_scales(const RouteArgs& a, int64_t slot, bool& skip) {
  if (!a.scales) return nullptr;
  const int64_t e = a.ids64 ? ((const int64_t*)a.ids)[slot] : (int64_t)((const int32_t*)a.ids)[slot];
  if (e < 0 || e >= a.n_experts) {
    skip = true;
    return nullptr;
  }
  return a.scales + e * a.d;
}

template <typename T>
__device__ __forceinline__ void load_scales(const float* p, int i, int d, float (&s)[kVec<T>]) {
#pragma unroll
  for (int k = 0; k < kVec<T>; k += 4) {
    float q[4];
    load_chunk(p, i + k, d, q);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[k + j] = q[j];
  }
}

template <typename T>
__global__ void gather_kernel(RouteArgs a, CMat x, Mat rows) {
  const int64_t t = blockIdx.x;
  const int i = ((int)blockIdx.y * (int)blockDim.x + (int)threadIdx.x) * kVec<T>;
  if (i >= a.d) return;
  float v[kVec<T>];
  load_chunk((const T*)x.p + t * x.ld, i, a.d, v);
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t slot = t * a.top_k + j;
    const int p = a.position[slot];
    bool skip = p < 0 || p >= a.n_rows;
    const float* sc = skip ? nullptr : slot_scales(a, slot, skip);
    if (skip) continue;
    float o[kVec<T>];
    if (sc) load_scales<T>(sc, i, a.d, o);
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) o[k] = sc ? v[k] * o[k] : v[k];
    store_chunk((T*)rows.p + (int64_t)p * rows.ld, i, a.d, o);
  }
}

template <typename T>
__global__ void combine_kernel(RouteArgs a, CMat rows, const float* weights, Mat out) {
  const int64_t t = blockIdx.x;
  const int i = ((int)blockIdx.y * (int)blockDim.x + (int)threadIdx.x) * kVec<T>;
  if (i >= a.d) return;
  float acc[kVec<T>];
#pragma unroll
  for (int k = 0; k < kVec<T>; ++k) acc[k] = 0.f;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t slot = t * a.top_k + j;
    const int p = a.position[slot];
    bool skip = p < 0 || p >= a.n_rows;
    const float* sc = skip ? nullptr : slot_scales(a, slot, skip);
    if (skip) continue;
    float v[kVec<T>], s[kVec<T>];
    load_chunk((const T*)rows.p + (int64_t)p * rows.ld, i, a.d, v);
    if (sc) load_scales<T>(sc, i, a.d, s);
    const float w = weights ? weights[slot] : 1.f;
#pragma unroll
    for (int k = 0; k < kVec<T>; ++k) acc[k] = fmaf(sc ? s[k] : w, v[k], acc[k]);
  }
  store_chunk((T*)out.p + t * out.ld, i, a.d, acc);
}

// One wave per slot.
template <typename T>
__global__ __launch_bounds__(256) void combine_backward_kernel(RouteArgs a, CMat d_out, CMat rows,
                                                               const float* weights, Mat d_rows, float* d_weights) {
  const int lane = threadIdx.x & 63;
  const int64_t slot = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (slot >= a.n_tokens * a.top_k) return;
  const int p = a.position[slot];
  if (p < 0 || p >= a.n_rows) {
    if (d_weights && lane == 0) d_weights[slot] = 0.f;
    return;
  }
  const T* gp = (const T*)d_out.p + slot / a.top_k * d_out.ld;
  const T* rp = (const T*)rows.p + (int64_t)p * rows.ld;
  T* op = d_rows.p ? (T*)d_rows.p + (int64_t)p * d_rows.ld : nullptr;
  const float w = weights[slot];
  float dot = 0.f;
  for (int i = lane * kVec<T>; i < a.d; i += 64 * kVec<T>) {
    float g[kVec<T>], r[kVec<T>];
    load_chunk(gp, i, a.d, g);
    if (d_weights) {
      load_chunk(rp, i, a.d, r);
#pragma unroll
      for (int k = 0; k < kVec<T>; ++k) dot = fmaf(g[k], r[k], dot);
    }
    if (op) {
#pragma unroll
      for (int k = 0; k < kVec<T>; ++k) g[k] *= w;
      store_chunk(op, i, a.d, g);
    }
  }
  dot = wave_sum(dot);
  if (d_weights && lane == 0) d_weights[slot] = dot;
}

template <typename F>
hipError_t with_dtype(int dtype, F f) {
  if (dtype == AWQ_DTYPE_BF16) f(Bf16{});
  else if (dtype == AWQ_DTYPE_F16) f(F16{});
  else f(0.f);
  return hipGetLastError();
}

// Threads per block along a row of `chunks` 16-byte chunks.
int row_threads(int chunks) { return chunks <= 64 ? 64 : chunks <= 128 ? 128 : 256; }

}  // namespace

int moe_sort_blocks(int64_t n_slots) {
  const int64_t b = (n_slots + kSortSlots - 1) / kSortSlots;
  return (int)(b < kSortMaxBlocks ? b : kSortMaxBlocks);
}

hipError_t launch_moe_sort(const void* ids, bool ids64, int n_slots, int n_experts, int32_t* offsets, int32_t* order,
                           int32_t* position, int32_t* counts, hipStream_t st) {
  const int blocks = moe_sort_blocks(n_slots);
  const int per = (n_slots + blocks - 1) / blocks;
  int id_bits = 0;
  while ((n_experts >> id_bits) != 0) ++id_bits;  // ids and n_experts itself, the dropped slots' id
  const size_t lds = (size_t)(kSortWaves + 1) * n_experts * sizeof(int);
  if (blocks > 1)
    hipLaunchKernelGGL((sort_kernel<false>), dim3(blocks), dim3(kSortThreads), lds, st, ids, ids64, n_slots,
                       n_experts, id_bits, per, counts, offsets, order, position);
  hipLaunchKernelGGL((sort_kernel<true>), dim3(blocks), dim3(kSortThreads), lds, st, ids, ids64, n_slots, n_experts,
                     id_bits, per, counts, offsets, order, position);
  return hipGetLastError();
}

hipError_t launch_moe_gather(const RouteArgs& a, int dtype, CMat x, Mat rows, hipStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int chunks = (a.d + kVec<T> - 1) / kVec<T>, threads = row_threads(chunks);
    hipLaunchKernelGGL((gather_kernel<T>), dim3((unsigned)a.n_tokens, (chunks + threads - 1) / threads),
                       dim3(threads), 0, st, a, x, rows);
  });
}

hipError_t launch_moe_combine(const RouteArgs& a, int dtype, CMat rows, const float* weights, Mat out,
                              hipStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int chunks = (a.d + kVec<T> - 1) / kVec<T>, threads = row_threads(chunks);
    hipLaunchKernelGGL((combine_kernel<T>), dim3((unsigned)a.n_tokens, (chunks + threads - 1) / threads),
                       dim3(threads), 0, st, a, rows, weights, out);
  });
}

hipError_t launch_moe_combine_backward(const RouteArgs& a, int dtype, CMat d_out, CMat rows, const float* weights,
                                       Mat d_rows, float* d_weights, hipStream_t st) {
  const int64_t slots = a.n_tokens * a.top_k;
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((combine_backward_kernel<T>), dim3((unsigned)((slots + 3) / 4)), dim3(256), 0, st, a, d_out,
                       rows, weights, d_rows, d_weights);
  });
}

}  // namespace awq
