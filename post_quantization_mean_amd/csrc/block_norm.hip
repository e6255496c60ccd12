// The RMS norms before and after a block, fused with the block's gate and residual scale, and their
// gradients:
//   z = y / sqrt(mean(y^2) + eps) * w_post,  r' = residual + res_scale * gate * z,
//   h = r' / sqrt(mean(r'^2) + eps) * w_pre.
// Both directions are bound by memory: a row is read once into registers, its sums are formed across the
// block, and each output is written once. One block handles a row (forward) or rows in a fixed stride
// (backward, whose [d] gradients gather in registers over the block's rows, then over blocks in a second
// kernel, in a fixed order: no atomics).
#include <type_traits>

#include "awq_moe.h"
#include "moe.h"
#include "moe_device.h"

namespace awq {
namespace {

constexpr int64_t kMaxBlocks = 1 << 20;

// mean of squares -> 1 / sqrt(. + eps)
__device__ __forceinline__ float rstd_of(float sum, int d, float eps) {
  return 1.0f / sqrtf(sum / (float)d + eps);
}

template <typename T, int THREADS, int ITEMS>
__global__ __launch_bounds__(THREADS) void block_norm_kernel(BlockNormArgs a, Mat res_out, Mat h) {
  constexpr int V = kVec<T>;
  __shared__ float red[2][THREADS / 64];
  const int d = a.d;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    __syncthreads();  // the previous row's sums have been read
    const T* yp = a.y.p ? (const T*)a.y.p + row * a.y.ld : nullptr;
    const T* rp = (const T*)a.residual.p + row * a.residual.ld;
    const T* gp = a.gate ? (const T*)a.gate + row * a.ld_gate : nullptr;

    float r[ITEMS][V];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) load_chunk(rp, (i * THREADS + (int)threadIdx.x) * V, d, r[i]);
    if (yp) {
      float y[ITEMS][V];
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        load_chunk(yp, (i * THREADS + (int)threadIdx.x) * V, d, y[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] = fmaf(y[i][k], y[i][k], s[0]);
      }
      float rs = 1.f;
      if (a.w_post) {
        block_sum<THREADS, 1>(s, red[0]);
        rs = rstd_of(s[0], d, a.eps);
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int at = (i * THREADS + (int)threadIdx.x) * V;
        float w[V];
        if (a.w_post) {
          load_chunk((const T*)a.w_post, at, d, w);
#pragma unroll
          for (int k = 0; k < V; ++k) y[i][k] = y[i][k] * rs * w[k];
        }
        if (gp) {
          load_chunk(gp, at, d, w);
#pragma unroll
          for (int k = 0; k < V; ++k) y[i][k] *= w[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) r[i][k] = fmaf(a.res_scale, y[i][k], r[i][k]);
        if (res_out.p) store_chunk((T*)res_out.p + row * res_out.ld, at, d, r[i]);
      }
    }
    if (h.p) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] = fmaf(r[i][k], r[i][k], s[0]);
      block_sum<THREADS, 1>(s, red[1]);
      const float rs = rstd_of(s[0], d, a.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int at = (i * THREADS + (int)threadIdx.x) * V;
        float w[V];
        load_chunk((const T*)a.w_pre, at, d, w);
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] *= r[i][k] * rs;
        store_chunk((T*)h.p + row * h.ld, at, d, w);
      }
    }
  }
}

struct BlockNormGrads {
  CMat d_res, d_h;
  Mat d_y, d_residual;
  void* d_gate;  // with a gate per token
  int64_t ld_d_gate;
  float* partial;  // [3][blocks][d]: d_w_post, d_w_pre, d_gate; or NULL
  bool sum_gate;
};

template <typename T, int THREADS, int ITEMS>
__global__ __launch_bounds__(THREADS) void block_norm_backward_kernel(BlockNormArgs a, BlockNormGrads g) {
  constexpr int V = kVec<T>, W = THREADS / 64;
  __shared__ float red[W * 4];
  const int d = a.d;
  const float inv_d = 1.0f / (float)d;
  float sw1[ITEMS][V], sw2[ITEMS][V], sg[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) sw1[i][k] = sw2[i][k] = sg[i][k] = 0.f;

  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* gp = a.gate ? (const T*)a.gate + row * a.ld_gate : nullptr;
    float y[ITEMS][V], r[ITEMS][V], D[ITEMS][V], dhw[ITEMS][V];
    float s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = (i * THREADS + (int)threadIdx.x) * V;
      load_chunk((const T*)a.residual.p + row * a.residual.ld, at, d, r[i]);
      if (a.y.p) load_chunk((const T*)a.y.p + row * a.y.ld, at, d, y[i]);
      else
#pragma unroll
        for (int k = 0; k < V; ++k) y[i][k] = 0.f;
      if (g.d_res.p) load_chunk((const T*)g.d_res.p + row * g.d_res.ld, at, d, D[i]);
      else
#pragma unroll
        for (int k = 0; k < V; ++k) D[i][k] = 0.f;
      if (g.d_h.p) load_chunk((const T*)g.d_h.p + row * g.d_h.ld, at, d, dhw[i]);
      else
#pragma unroll
        for (int k = 0; k < V; ++k) dhw[i][k] = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) s1[0] = fmaf(y[i][k], y[i][k], s1[0]);
    }
    float rs1 = 1.f;
    __syncthreads();  // the previous row's last sums have been read
    if (a.w_post) {
      block_sum<THREADS, 1>(s1, red);
      rs1 = rstd_of(s1[0], d, a.eps);
    }
    // u1 in y; r' in r; d_h w_pre stays in dhw
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = (i * THREADS + (int)threadIdx.x) * V;
      float w1[V], gt[V], w2[V];
      if (a.w_post) load_chunk((const T*)a.w_post, at, d, w1);
      if (gp) load_chunk(gp, at, d, gt);
      if (a.w_pre) load_chunk((const T*)a.w_pre, at, d, w2);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        y[i][k] *= rs1;
        float z = a.w_post ? y[i][k] * w1[k] : y[i][k];
        if (gp) z *= gt[k];
        r[i][k] = fmaf(a.res_scale, z, r[i][k]);
        s2[0] = fmaf(r[i][k], r[i][k], s2[0]);
        if (a.w_pre) s2[1] = fmaf(dhw[i][k] * w2[k], r[i][k], s2[1]);
      }
    }
    float rs2 = 0.f, m2 = 0.f;
    if (a.w_pre) {
      block_sum<THREADS, 2>(s2, red + W);
      rs2 = rstd_of(s2[0], d, a.eps);
      m2 = s2[1] * rs2 * inv_d;  // mean(d_h w_pre u2)
    }
    float s3[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = (i * THREADS + (int)threadIdx.x) * V;
      float w1[V], gt[V], w2[V], dg[V];
      if (a.w_post) load_chunk((const T*)a.w_post, at, d, w1);
      if (gp) load_chunk(gp, at, d, gt);
      if (a.w_pre) load_chunk((const T*)a.w_pre, at, d, w2);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (a.w_pre) {
          const float u2 = r[i][k] * rs2;
          sw2[i][k] = fmaf(dhw[i][k], u2, sw2[i][k]);
          D[i][k] = fmaf(rs2, dhw[i][k] * w2[k] - u2 * m2, D[i][k]);
        }
        r[i][k] = D[i][k];
        const float ad = a.res_scale * D[i][k];
        const float z = a.w_post ? y[i][k] * w1[k] : y[i][k];
        dg[k] = ad * z;
        sg[i][k] += dg[k];
        const float t = gp ? ad * gt[k] : ad;
        sw1[i][k] = fmaf(t, y[i][k], sw1[i][k]);
        D[i][k] = a.w_post ? t * w1[k] : t;
        s3[0] = fmaf(D[i][k], y[i][k], s3[0]);
      }
      if (g.d_residual.p) store_chunk((T*)g.d_residual.p + row * g.d_residual.ld, at, d, r[i]);
      if (g.d_gate && !g.sum_gate) store_chunk((T*)g.d_gate + row * g.ld_d_gate, at, d, dg);
    }
    if (g.d_y.p) {
      float m1 = 0.f;
      if (a.w_post) {
        block_sum<THREADS, 1>(s3, red + 3 * W);
        m1 = s3[0] * inv_d;
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int at = (i * THREADS + (int)threadIdx.x) * V;
        float o[V];
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = a.w_post ? rs1 * (D[i][k] - y[i][k] * m1) : D[i][k];
        store_chunk((T*)g.d_y.p + row * g.d_y.ld, at, d, o);
      }
    }
  }
  if (g.partial) {
    const int64_t plane = (int64_t)gridDim.x * d;
    float* p = g.partial + (int64_t)blockIdx.x * d;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = (i * THREADS + (int)threadIdx.x) * V;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (at + k < d) {
          p[at + k] = sw1[i][k];
          p[plane + at + k] = sw2[i][k];
          p[2 * plane + at + k] = sg[i][k];
        }
    }
  }
}

// out[c] = sum over the blocks' partial sums of column c, in block order within each of 16 interleaved
// runs, then over the runs.
struct ColumnSums {
  float* out[3];
};
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* partial, int blocks, int d, ColumnSums outs) {
  __shared__ float part[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), run = threadIdx.x >> 6;
  float* out = blockIdx.y == 0 ? outs.out[0] : blockIdx.y == 1 ? outs.out[1] : outs.out[2];
  if (!out) return;
  const float* p = partial + (int64_t)blockIdx.y * blocks * d;
  float s = 0.f;
  if (c < d)
    for (int b = run; b < blocks; b += 16) s += p[(int64_t)b * d + c];
  part[run][threadIdx.x & 63] = s;
  __syncthreads();
  if (run == 0 && c < d) {
    for (int w = 1; w < 16; ++w) s += part[w][threadIdx.x & 63];
    out[c] = s;
  }
}

template <typename T, typename F>
hipError_t with_shape(int d, F f) {
  const int chunks = (d + kVec<T> - 1) / kVec<T>;
  using std::integral_constant;
  if (chunks <= 64) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (chunks <= 256) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (chunks <= 512) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (chunks <= 1024) f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  else if (chunks <= 2048) f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
  else if (chunks <= 4096) f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  else f(integral_constant<int, 1024>{}, integral_constant<int, 8>{});
  return hipGetLastError();
}

template <typename F>
hipError_t with_dtype(int dtype, F f) {
  if (dtype == AWQ_DTYPE_BF16) return f(Bf16{});
  if (dtype == AWQ_DTYPE_F16) return f(F16{});
  return f(0.f);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, int dtype, Mat res_out, Mat h, hipStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return with_shape<T>(a.d, [&](auto threads, auto items) {
      hipLaunchKernelGGL((block_norm_kernel<T, decltype(threads)::value, decltype(items)::value>),
                         dim3((unsigned)(a.n < kMaxBlocks ? a.n : kMaxBlocks)), dim3(decltype(threads)::value), 0, st, a,
                         res_out, h);
    });
  });
}

int block_norm_backward_blocks(int64_t n_tokens, int64_t d) { return (int)(n_tokens < 512 ? n_tokens : 512); }

hipError_t launch_block_norm_backward(const BlockNormArgs& a, int dtype, CMat d_res, CMat d_h, Mat d_y, Mat d_residual,
                                      float* d_w_post, float* d_w_pre, void* d_gate, int64_t ld_d_gate,
                                      float* partial, hipStream_t st) {
  const int blocks = block_norm_backward_blocks(a.n, a.d);
  const bool sum_gate = a.ld_gate == 0;
  const BlockNormGrads g{d_res, d_h, d_y, d_residual, d_gate, ld_d_gate, partial, sum_gate};
  hipError_t e = with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return with_shape<T>(a.d, [&](auto threads, auto items) {
      hipLaunchKernelGGL((block_norm_backward_kernel<T, decltype(threads)::value, decltype(items)::value>),
                         dim3((unsigned)blocks), dim3(decltype(threads)::value), 0, st, a, g);
    });
  });
  if (e != hipSuccess || !partial) return e;
  const ColumnSums outs{{d_w_post, d_w_pre, sum_gate ? (float*)d_gate : nullptr}};
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((a.d + 63) / 64), 3), dim3(1024), 0, st, partial, blocks, a.d,
                     outs);
  return hipGetLastError();
}

}  // namespace awq
