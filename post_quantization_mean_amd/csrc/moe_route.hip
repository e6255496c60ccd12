// Tokens into expert order and back.
//
// Sort: a stable counting sort of the slots by expert. Slots are split into contiguous ranges, one per
// block and within it one per wave; a wave walks its range 64 slots at a time and finds each slot's rank
// among the equal ids of the 64 by matching id bits with ballots, so that counts and places come out the
// same whatever the timing (no global atomics). One block does it all for few slots; more take a counting
// launch and a placing launch, whose blocks each add up the counts of the blocks before them. Bound by latency:
// 32768 slots of 64 experts take 13 us, where 2048 slots a block beat 1024, 4096 and 8192.
//
// Gather and combine are bound by memory: gather reads a token's row once and writes it to its places,
// combine reads the places' rows and writes the token's row once, 16 bytes per lane. A wave takes 64 chunks of a
// token and starts the loads of up to four slots before it uses the first; blocks take the segments of a token
// before the next token, so that what is written and read at a time lies close. Measured with 4096 bf16 tokens of
// 2048 elements for 8 of 64 experts each: gather with multipliers 56 us (5.4 TB/s), without 54 (5.6), combine 53
// (5.6), gather's gradient 69 (4.4; the multipliers come from the caches), combine's 108 (5.3).
#include <type_traits>

#include "awq_moe.h"
#include "moe.h"
#include "moe_device.h"

namespace awq {
namespace {

// ---------------------------------------------------------------- sort

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortMaxBlocks = 256;
constexpr int kSortSlots = 2048;  // slots of a block (two steps of a wave), until kSortMaxBlocks would be passed

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
    // (counts that a caller's other work has overwritten must not lead out of `order`)
    if (id < n_experts && (unsigned)place < (unsigned)n_slots) order[place] = slot;
  });
  for (int i = max(b0, kept) + tid; i < b1; i += kSortThreads) order[i] = -1;
}

// ---------------------------------------------------------------- gather, combine

// How rows are moved: element by element (rows narrower than a chunk), or in whole loads without a branch, the last
// chunk moved back to end with the row (Place), and stored normally or past the caches.
enum RowMode { kRowSmall, kRowCached, kRowStreamed };

// A lane's chunk of kVec elements of every row it handles.
template <typename T, RowMode MODE>
struct RowChunk {
  static constexpr int V = kVec<T>;
  static constexpr bool SMALL = MODE == kRowSmall;
  Place<T> p;
  int i, d;
  __device__ __forceinline__ RowChunk(int first, int width) : p(first, width), i(first), d(width) {}
  __device__ __forceinline__ void load(const T* row, float (&v)[V]) const {
    if constexpr (SMALL) {
      load_chunk(row, i, d, v);
    } else {
      const uint4 u = load_raw(row, p);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = raw_f32<T>(u, k);
    }
  }
  __device__ __forceinline__ void store(T* row, const float (&v)[V]) const {
    if constexpr (SMALL) store_chunk(row, i, d, v);
    else store_own<T, MODE == kRowStreamed>(row, p, v);
  }
  // the chunk's elements of a float32 row
  __device__ __forceinline__ void load_f32(const float* row, float (&v)[V]) const {
    if constexpr (SMALL) {
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = i + k < d ? row[i + k] : 0.f;
    } else {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const Chunk<float> c = *reinterpret_cast<const Chunk<float>*>(row + p.at + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[k + q] = c.v[q];
      }
    }
  }
  // does element k of the chunk belong to it?
  __device__ __forceinline__ bool owns(int k) const { return SMALL ? i + k < d : k >= p.skip; }
};

// Tokens of a wave of the gather, for B slots a batch.
template <int B>
inline constexpr int kGatherTokens = B >= 4 ? 1 : 4 / B;

// B of a token's slots: which are kept, where their rows lie (row 0 where not, so that every load can go out
// before the first is used) and their experts' multipliers.
template <int B>
struct Slots {
  bool kept[B];
  int row[B];
  int64_t slot[B];
  const float* scales[B];
};
template <int B>
__device__ __forceinline__ void find_slots(const RouteArgs& a, int64_t t, int j, Slots<B>& s) {
#pragma unroll
  for (int q = 0; q < B; ++q) {
    s.slot[q] = t * a.top_k + min(j + q, a.top_k - 1);
    s.row[q] = a.position[s.slot[q]];
    s.kept[q] = j + q < a.top_k && s.row[q] >= 0 && s.row[q] < a.n_rows;
    if (a.scales) {
      int64_t e = a.ids64 ? ((const int64_t*)a.ids)[s.slot[q]] : (int64_t)((const int32_t*)a.ids)[s.slot[q]];
      const bool known = e >= 0 && e < a.n_experts;
      s.kept[q] = s.kept[q] && known;
      s.scales[q] = a.scales + (known ? e : 0) * a.d;
    }
    if (!s.kept[q]) s.row[q] = 0;
  }
}

// A wave's token and a lane's chunk of it in a token_grid.
template <typename T>
__device__ __forceinline__ void token_place(int64_t& t, int& i) {
  t = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  i = ((int)blockIdx.x * 64 + (int)(threadIdx.x & 63)) * kVec<T>;
}

// A wave takes 64 chunks of TB tokens' rows; TB B slots' loads go out together.
template <typename T, RowMode MODE, bool SCALED, int B>
__global__ __launch_bounds__(256) void gather_kernel(RouteArgs a, CMat x, Mat rows) {
  constexpr int TB = kGatherTokens<B>;
  int64_t t0;
  int i;
  token_place<T>(t0, i);
  t0 *= TB;
  if (t0 >= a.n_tokens || i >= a.d) return;
  const RowChunk<T, MODE> c(i, a.d);
  int64_t t[TB];
  float v[TB][kVec<T>];
#pragma unroll
  for (int u = 0; u < TB; ++u) {
    t[u] = min(t0 + u, a.n_tokens - 1);
    c.load((const T*)x.p + t[u] * x.ld, v[u]);
  }
  for (int j = 0; j < a.top_k; j += B) {
    Slots<B> s[TB];
    float m[TB][B][kVec<T>];
#pragma unroll
    for (int u = 0; u < TB; ++u) {
      find_slots(a, t[u], j, s[u]);
      if (SCALED) {
#pragma unroll
        for (int q = 0; q < B; ++q) c.load_f32(s[u].scales[q], m[u][q]);
      }
    }
#pragma unroll
    for (int u = 0; u < TB; ++u) {
#pragma unroll
      for (int q = 0; q < B; ++q) {
        if (s[u].kept[q] && t0 + u < a.n_tokens) {
#pragma unroll
          for (int k = 0; k < kVec<T>; ++k) m[u][q][k] = SCALED ? v[u][k] * m[u][q][k] : v[u][k];
          c.store((T*)rows.p + (int64_t)s[u].row[q] * rows.ld, m[u][q]);
        }
      }
    }
  }
}

template <typename T, RowMode MODE, bool SCALED, int B>
__global__ __launch_bounds__(256) void combine_kernel(RouteArgs a, CMat rows, const float* weights, Mat out) {
  int64_t t;
  int i;
  token_place<T>(t, i);
  if (t >= a.n_tokens || i >= a.d) return;
  const RowChunk<T, MODE> c(i, a.d);
  float acc[kVec<T>];
#pragma unroll
  for (int k = 0; k < kVec<T>; ++k) acc[k] = 0.f;
  for (int j = 0; j < a.top_k; j += B) {
    Slots<B> s;
    find_slots(a, t, j, s);
    float v[B][kVec<T>], m[B][kVec<T>], w[B];
#pragma unroll
    for (int q = 0; q < B; ++q) {
      c.load((const T*)rows.p + (int64_t)s.row[q] * rows.ld, v[q]);
      if (SCALED) c.load_f32(s.scales[q], m[q]);
      else w[q] = weights[s.slot[q]];
    }
#pragma unroll
    for (int q = 0; q < B; ++q) {
      if (s.kept[q]) {
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) acc[k] = fmaf(SCALED ? m[q][k] : w[q], v[q][k], acc[k]);
      }
    }
  }
  c.store((T*)out.p + t * out.ld, acc);
}

// The sum of a token's rows without multipliers: weights of one.
template <typename T, RowMode MODE, int B>
__global__ __launch_bounds__(256) void sum_kernel(RouteArgs a, CMat rows, Mat out) {
  int64_t t;
  int i;
  token_place<T>(t, i);
  if (t >= a.n_tokens || i >= a.d) return;
  const RowChunk<T, MODE> c(i, a.d);
  float acc[kVec<T>];
#pragma unroll
  for (int k = 0; k < kVec<T>; ++k) acc[k] = 0.f;
  for (int j = 0; j < a.top_k; j += B) {
    Slots<B> s;
    find_slots(a, t, j, s);
    float v[B][kVec<T>];
#pragma unroll
    for (int q = 0; q < B; ++q) c.load((const T*)rows.p + (int64_t)s.row[q] * rows.ld, v[q]);
#pragma unroll
    for (int q = 0; q < B; ++q) {
      if (s.kept[q]) {
#pragma unroll
        for (int k = 0; k < kVec<T>; ++k) acc[k] += v[q][k];
      }
    }
  }
  c.store((T*)out.p + t * out.ld, acc);
}

// One wave per slot, kDotChunks chunks of both rows in flight.
constexpr int kDotChunks = 4;
template <typename T, RowMode MODE>
__global__ __launch_bounds__(256) void combine_backward_kernel(RouteArgs a, CMat d_out, CMat rows,
                                                               const float* weights, Mat d_rows, float* d_weights) {
  const int lane = threadIdx.x & 63;
  const int64_t slot = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  for (int i0 = lane * kVec<T>; i0 < a.d; i0 += 64 * kVec<T> * kDotChunks) {
    float g[kDotChunks][kVec<T>], r[kDotChunks][kVec<T>];
#pragma unroll
    for (int q = 0; q < kDotChunks; ++q) {
      const RowChunk<T, MODE> c(i0 + q * 64 * kVec<T>, a.d);
      c.load(gp, g[q]);
      c.load(rp, r[q]);
    }
#pragma unroll
    for (int q = 0; q < kDotChunks; ++q) {
      const RowChunk<T, MODE> c(i0 + q * 64 * kVec<T>, a.d);
#pragma unroll
      for (int k = 0; k < kVec<T>; ++k) {
        if (c.owns(k)) dot = fmaf(g[q][k], r[q][k], dot);
        g[q][k] *= w;
      }
      if (op && c.i < a.d) c.store(op, g[q]);
    }
  }
  dot = wave_sum(dot);
  if (d_weights && lane == 0) d_weights[slot] = dot;
}

// f(element, mode, slots per batch) for the dtype, the width and the choices of a token
template <bool STREAM, typename F>
hipError_t with_rows(int dtype, const RouteArgs& a, F f) {
  auto batch = [&](auto t, auto mode) {
    if (a.top_k == 1) f(t, mode, std::integral_constant<int, 1>{});
    else if (a.top_k == 2) f(t, mode, std::integral_constant<int, 2>{});
    else f(t, mode, std::integral_constant<int, 4>{});
  };
  auto go = [&](auto t) {
    if (a.d < kVec<decltype(t)>) batch(t, std::integral_constant<RowMode, kRowSmall>{});
    else if (!STREAM || !a.stream_out) batch(t, std::integral_constant<RowMode, kRowCached>{});
    else if constexpr (STREAM) batch(t, std::integral_constant<RowMode, kRowStreamed>{});
  };
  if (dtype == AWQ_DTYPE_BF16) go(Bf16{});
  else if (dtype == AWQ_DTYPE_F16) go(F16{});
  else go(0.f);
  return hipGetLastError();
}

// Blocks of 64 chunks (fastest) by four units of tokens, which fill two dimensions: one holds 65535 blocks.
template <typename T>
dim3 token_grid(int d, int64_t units) {
  const int chunks = (d + kVec<T> - 1) / kVec<T>;
  const int64_t blocks = (units + 3) / 4, layers = (blocks + 65534) / 65535;
  return dim3((unsigned)((chunks + 63) / 64), (unsigned)((blocks + layers - 1) / layers), (unsigned)layers);
}

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
  return with_rows<true>(dtype, a, [&](auto t, auto mode, auto batch) {
    using T = decltype(t);
    constexpr RowMode M = decltype(mode)::value;
    constexpr int B = decltype(batch)::value;
    const dim3 grid = token_grid<T>(a.d, (a.n_tokens + kGatherTokens<B> - 1) / kGatherTokens<B>);
    if (a.scales) hipLaunchKernelGGL((gather_kernel<T, M, true, B>), grid, dim3(256), 0, st, a, x, rows);
    else hipLaunchKernelGGL((gather_kernel<T, M, false, B>), grid, dim3(256), 0, st, a, x, rows);
  });
}

hipError_t launch_moe_combine(const RouteArgs& a, int dtype, CMat rows, const float* weights, Mat out,
                              hipStream_t st) {
  return with_rows<false>(dtype, a, [&](auto t, auto mode, auto batch) {
    using T = decltype(t);
    constexpr RowMode M = decltype(mode)::value;
    constexpr int B = decltype(batch)::value;
    const dim3 grid = token_grid<T>(a.d, a.n_tokens);
    if (a.scales)
      hipLaunchKernelGGL((combine_kernel<T, M, true, B>), grid, dim3(256), 0, st, a, rows, weights, out);
    else if (weights)
      hipLaunchKernelGGL((combine_kernel<T, M, false, B>), grid, dim3(256), 0, st, a, rows, weights, out);
    else
      hipLaunchKernelGGL((sum_kernel<T, M, B>), grid, dim3(256), 0, st, a, rows, out);
  });
}

hipError_t launch_moe_combine_backward(const RouteArgs& a, int dtype, CMat d_out, CMat rows, const float* weights,
                                       Mat d_rows, float* d_weights, hipStream_t st) {
  const int64_t slots = a.n_tokens * a.top_k;
  return with_rows<true>(dtype, a, [&](auto t, auto mode, auto) {
    hipLaunchKernelGGL((combine_backward_kernel<decltype(t), decltype(mode)::value>),
                       dim3((unsigned)((slots + 3) / 4)), dim3(256), 0, st, a, d_out, rows, weights, d_rows, d_weights);
  });
}

}  // namespace awq
