// The RMS norms before and after a block, fused with the block's gate and residual scale, and their
// gradients:
//   z = y / sqrt(mean(y^2) + eps) * w_post,  r' = residual + res_scale * gate * z,
//   h = r' / sqrt(mean(r'^2) + eps) * w_pre.
// Both directions are bound by memory: a row is read once into registers (16 bytes per lane, kept packed),
// its sums are formed across the block, and each output is written once. A block takes rows in a fixed
// stride: the [d] weights stay in its registers, and the next row is loaded while the current one is
// summed, so that loads stay in flight across the sums' barriers. The gradients of the [d] weights gather in
// registers over the block's rows, then over blocks in a second kernel, in a fixed order: no atomics.
// Measured: forward 8192 x 8192 bf16 101 us (5.3 TB/s), 8192 x 4096 47 (5.7); gradients 8192 x 4096 bf16 97 (4.1: two
// blocks of 256 threads fill the registers of a compute unit), float32 155 (5.2). At 8192 x 4100 a row's last chunk needs a
// fifth wave and a compute unit holds one block: 143.
#include <type_traits>

#include "awq_moe.h"
#include "moe.h"
#include "moe_device.h"

namespace awq {
namespace {

// mean of squares -> 1 / sqrt(. + eps)
__device__ __forceinline__ float rstd_of(float sum, int d, float eps) {
  return 1.0f / sqrtf(sum / (float)d + eps);
}

// This thread's chunks of a row, packed.
template <typename T, int ITEMS>
struct Raw {
  uint4 u[ITEMS];
  __device__ __forceinline__ void load(const void* base, int64_t offset, const Place<T> (&p)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) u[i] = load_raw((const T*)base + offset, p[i]);
  }
  __device__ __forceinline__ void own(const Place<T> (&p)[ITEMS]) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) u[i] = own_raw<T>(u[i], p[i].skip);
  }
  __device__ __forceinline__ void fill(const uint4& v) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) u[i] = v;
  }
  __device__ __forceinline__ float at(int i, int k) const { return raw_f32<T>(u[i], k); }
  // Keeps the chunks packed past this point: without it the compiler unpacks once and holds the float32
  // values of weights across the loop and of the row across its sums, twice the registers.
  __device__ __forceinline__ void keep_packed() {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) asm volatile("" : "+v"(u[i].x), "+v"(u[i].y), "+v"(u[i].z), "+v"(u[i].w));
  }
};

template <int... I>
struct Seq {};
template <int N, int... I>
struct MakeSeq : MakeSeq<N - 1, N - 1, I...> {};
template <int... I>
struct MakeSeq<0, I...> {
  typedef Seq<I...> type;
};

// The places of a thread's chunks: chunk i starts at element (i * threads + thread) * kVec.
template <typename T, int ITEMS>
struct Places {
  Place<T> p[ITEMS];
  template <int... I>
  __device__ __forceinline__ Places(int d, Seq<I...>)
      : p{Place<T>((I * (int)blockDim.x + (int)threadIdx.x) * kVec<T>, d)...} {}
  __device__ __forceinline__ explicit Places(int d) : Places(d, typename MakeSeq<ITEMS>::type()) {}
};

// KEEP: the weights stay in registers and the next row is loaded ahead; otherwise (wide rows) neither, which
// the registers would not hold: weights and gate are loaded a chunk at a time. 1170 x 28672 bf16 57 - 60 us (4.5 - 4.7 TB/s;
// whole rows of weights spilled, 92), 2048 x 16384 float32 104 - 113 (4.8 - 5.2; 125), 1170 x 28672 float32, which still
// spills, 234 - 238 (2.3).
template <typename T, int ITEMS, int TMAX, bool KEEP>
__global__ __launch_bounds__(TMAX) void block_norm_kernel(BlockNormArgs a, Mat res_out, Mat h) {
  constexpr int V = kVec<T>;
  __shared__ float red[2][16];
  const int d = a.d;
  const bool block = a.y.p != nullptr, token_gate = a.ld_gate != 0;
  const bool ragged = d % (ITEMS * (int)blockDim.x * V) != 0;  // some lanes have less than whole chunks
  const Places<T, ITEMS> at(d);
  Raw<T, ITEMS> w1, w2, gt, y, r, yn, rn, gn;
  w1.fill(raw_ones<T>());
  gt.fill(raw_ones<T>());
  int64_t row = blockIdx.x;
  auto load_row = [&](int64_t n, Raw<T, ITEMS>& ly, Raw<T, ITEMS>& lr, Raw<T, ITEMS>& lg) {
    if (block) ly.load(a.y.p, n * a.y.ld, at.p);
    else ly.fill(make_uint4(0, 0, 0, 0));  // in every row: the row ahead has registers of its own
    lr.load(a.residual.p, n * a.residual.ld, at.p);
    if (KEEP && token_gate) lg.load(a.gate, n * a.ld_gate, at.p);
  };
  load_row(row, y, r, gt);
  if (KEEP) {
    if (a.w_post) w1.load(a.w_post, 0, at.p);
    if (a.gate && !token_gate) gt.load(a.gate, 0, at.p);
    if (a.w_pre) w2.load(a.w_pre, 0, at.p);
    if (ragged) {  // zero where a lane owns nothing, as y and r: the sum does not see the neighbours' infinities
      w1.own(at.p);
      gt.own(at.p);
    }
  }
  for (; row < a.n; row += gridDim.x) {
    const int64_t next = row + gridDim.x;
    if (KEEP && next < a.n) load_row(next, yn, rn, gn);
    if (ragged) {
      y.own(at.p);
      if (KEEP) r.own(at.p);
      if (KEEP && token_gate) gt.own(at.p);
    }
    if (KEEP) {
      w1.keep_packed();
      w2.keep_packed();
      gt.keep_packed();
    }
    float rs = a.res_scale;
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] = fmaf(y.at(i, k), y.at(i, k), s[0]);
      block_sum(s, red[0]);
      rs *= rstd_of(s[0], d, a.eps);
      y.keep_packed();
    }
    float v[ITEMS][V], s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!KEEP) {  // a chunk at a time: the registers do not hold the row and its weights
        if (a.w_post) w1.u[i] = load_raw((const T*)a.w_post, at.p[i]);
        if (a.gate) gt.u[i] = load_raw((const T*)a.gate + row * a.ld_gate, at.p[i]);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        v[i][k] = fmaf(y.at(i, k) * rs * w1.at(i, k), gt.at(i, k), r.at(i, k));
        // only a last chunk can be cut: a block has more threads than chunks too many
        if (!KEEP && i == ITEMS - 1) v[i][k] = k < at.p[i].skip ? 0.f : v[i][k];
        s[0] = fmaf(v[i][k], v[i][k], s[0]);
      }
      if (res_out.p) store_own((T*)res_out.p + row * res_out.ld, at.p[i], v[i]);
    }
    if (h.p) {
      block_sum(s, red[1]);
      const float rs2 = rstd_of(s[0], d, a.eps);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if (!KEEP) w2.u[i] = load_raw((const T*)a.w_pre, at.p[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] *= rs2 * w2.at(i, k);
        store_own((T*)h.p + row * h.ld, at.p[i], v[i]);
      }
    }
    if (!(a.w_post && h.p)) __syncthreads();  // one sum a row: the next one reuses its floats
    if (KEEP) {
      y = yn;
      r = rn;
      if (token_gate) gt = gn;
    } else
    if (next < a.n) {
      load_row(next, y, r, gt);
    }
  }
}

// Rows narrower than a chunk: one thread each.
template <typename T>
__global__ __launch_bounds__(256) void block_norm_narrow_kernel(BlockNormArgs a, Mat res_out, Mat h) {
  constexpr int V = kVec<T>;
  const int d = a.d;
  for (int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; row < a.n; row += (int64_t)gridDim.x * blockDim.x) {
    float y[V], v[V], s = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      y[c] = a.y.p && c < d ? to_f32(((const T*)a.y.p)[row * a.y.ld + c]) : 0.f;
      s = fmaf(y[c], y[c], s);
    }
    const float rs = a.w_post ? a.res_scale * rstd_of(s, d, a.eps) : a.res_scale;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if (c >= d) break;
      const float w1 = a.w_post ? to_f32(((const T*)a.w_post)[c]) : 1.f;
      const float gt = a.gate ? to_f32(((const T*)a.gate)[row * a.ld_gate + c]) : 1.f;
      v[c] = fmaf(y[c] * rs * w1, gt, to_f32(((const T*)a.residual.p)[row * a.residual.ld + c]));
      s2 = fmaf(v[c], v[c], s2);
      if (res_out.p) ((T*)res_out.p)[row * res_out.ld + c] = from_f32<T>(v[c]);
    }
    const float rs2 = rstd_of(s2, d, a.eps);
#pragma unroll
    for (int c = 0; c < V; ++c)
      if (h.p && c < d) ((T*)h.p)[row * h.ld + c] = from_f32<T>(v[c] * rs2 * to_f32(((const T*)a.w_pre)[c]));
  }
}

struct BlockNormGrads {
  CMat d_res, d_h;
  Mat d_y, d_residual, d_gate;  // d_gate: with a gate per token
  float* partial;               // [3][blocks][d]: d_w_post, d_w_pre, d_gate; or NULL
};

// PRE: with a norm behind r'. Without one the gradient does not see r', whatever it holds (0 * inf would). A template's
// choice: at run time it costs the others 5 % (8192 x 4100 bf16 143 -> 151 us).
template <typename T, int ITEMS, bool TOKEN, bool PRE>
__global__ __launch_bounds__(512) void block_norm_backward_kernel(BlockNormArgs a, BlockNormGrads g) {
  constexpr int V = kVec<T>;
  __shared__ float red[4][16];
  const int d = a.d;
  const float inv_d = 1.0f / (float)d;
  const bool block = a.y.p != nullptr;
  const bool ragged = d % (ITEMS * (int)blockDim.x * V) != 0;
  const Places<T, ITEMS> at(d);
  struct {
    Raw<T, ITEMS> y, r, dr, dh, gt;  // gt: with a gate per token
  } c;
  constexpr bool AHEAD = ITEMS <= 3;  // four chunks' registers do not hold the next row too
  auto ahead = c;
  auto load_into = [&](int64_t n, decltype(c)& c, Raw<T, ITEMS>& y) {
    if (block) y.load(a.y.p, n * a.y.ld, at.p);
    c.r.load(a.residual.p, n * a.residual.ld, at.p);
    if (g.d_res.p) c.dr.load(g.d_res.p, n * g.d_res.ld, at.p);
    if (g.d_h.p) c.dh.load(g.d_h.p, n * g.d_h.ld, at.p);
    if (TOKEN) c.gt.load(a.gate, n * a.ld_gate, at.p);
  };
  const uint4 zero = make_uint4(0, 0, 0, 0);
  c.y.fill(zero);
  c.dr.fill(zero);
  c.dh.fill(zero);
  ahead = c;
  Raw<T, ITEMS> w1, w2, wg;
  wg.fill(raw_ones<T>());
  w1.fill(raw_ones<T>());
  w2.fill(raw_ones<T>());
  float sw1[ITEMS][V], sw2[ITEMS][V], sg[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) sw1[i][k] = sw2[i][k] = sg[i][k] = 0.f;

  int64_t row = blockIdx.x;
  load_into(row, c, c.y);
  if (a.w_post) w1.load(a.w_post, 0, at.p);
  if (a.w_pre) w2.load(a.w_pre, 0, at.p);
  if (!TOKEN && a.gate) wg.load(a.gate, 0, at.p);
  if (ragged) {  // zero of every input where a lane owns nothing: the sums do not see the neighbours' weights
    w1.own(at.p);
    w2.own(at.p);
    wg.own(at.p);
  }
  for (; row < a.n; row += gridDim.x) {
    const int64_t next = row + gridDim.x;
    if (AHEAD && next < a.n) load_into(next, ahead, ahead.y);
    if (ragged) {
      c.y.own(at.p);
      c.r.own(at.p);
      c.dr.own(at.p);
      c.dh.own(at.p);
      if (TOKEN) c.gt.own(at.p);
    }
    auto keep_packed = [&]() {
      w1.keep_packed();
      w2.keep_packed();
      if (TOKEN) c.gt.keep_packed();
      else wg.keep_packed();
      c.y.keep_packed();
      c.r.keep_packed();
      c.dh.keep_packed();
    };
    keep_packed();
    float rs1 = 1.f;
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] = fmaf(c.y.at(i, k), c.y.at(i, k), s[0]);
      block_sum(s, red[0]);
      rs1 = rstd_of(s[0], d, a.eps);
      keep_packed();
    }
    // r' from the packed inputs, as often as it is needed
    const float ars = a.res_scale * rs1;
    auto gate = [&](int i, int k) { return TOKEN ? c.gt.at(i, k) : wg.at(i, k); };
    auto r_new = [&](int i, int k) { return fmaf(c.y.at(i, k) * ars * w1.at(i, k), gate(i, k), c.r.at(i, k)); };
    float rs2 = 0.f, m2 = 0.f;
    if (a.w_pre) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float r = r_new(i, k);
          s[0] = fmaf(r, r, s[0]);
          s[1] = fmaf(c.dh.at(i, k) * w2.at(i, k), r, s[1]);
        }
      block_sum(s, red[1]);
      rs2 = rstd_of(s[0], d, a.eps);
      m2 = s[1] * rs2 * inv_d;  // mean(d_h w_pre u2)
      keep_packed();
    }
    float t[ITEMS][V], s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float D[V], dg[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float u1 = c.y.at(i, k) * rs1, u2 = r_new(i, k) * rs2, dh = c.dh.at(i, k);
        sw2[i][k] = fmaf(dh, u2, sw2[i][k]);
        D[k] = fmaf(rs2, dh * w2.at(i, k) - u2 * m2, c.dr.at(i, k));
        if (!PRE) D[k] = c.dr.at(i, k);
        const float ad = a.res_scale * D[k];
        dg[k] = ad * u1 * w1.at(i, k);
        if (!TOKEN) sg[i][k] += dg[k];
        const float dz = ad * gate(i, k);
        sw1[i][k] = fmaf(dz, u1, sw1[i][k]);
        t[i][k] = dz * w1.at(i, k);
        s[0] = fmaf(t[i][k], u1, s[0]);
      }
      if (g.d_residual.p) store_own((T*)g.d_residual.p + row * g.d_residual.ld, at.p[i], D);
      if (TOKEN && g.d_gate.p) store_own((T*)g.d_gate.p + row * g.d_gate.ld, at.p[i], dg);
    }
    if (g.d_y.p) {
      float m1 = 0.f;
      if (a.w_post) {
        block_sum(s, red[3]);
        m1 = s[0] * inv_d * rs1;  // mean(t u1) / sqrt(.), times y below
        c.y.keep_packed();
      } else {
        c.y.fill(zero);  // d_y does not see y (0 * inf would)
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) t[i][k] = rs1 * (t[i][k] - c.y.at(i, k) * m1);
        store_own((T*)g.d_y.p + row * g.d_y.ld, at.p[i], t[i]);
      }
    }
    __syncthreads();  // the next row's sums reuse the floats of this one's
    if (AHEAD) c = ahead;
    else if (next < a.n) load_into(next, c, c.y);
  }
  if (g.partial) {
    const int64_t plane = (int64_t)gridDim.x * d;
    float* p = g.partial + (int64_t)blockIdx.x * d;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int e = at.p[i].at + k;
        if (k >= at.p[i].skip) {
          p[e] = sw1[i][k];
          p[plane + e] = sw2[i][k];
          p[2 * plane + e] = sg[i][k];
        }
      }
  }
}

// Rows too wide for the registers of a block, or narrower than a chunk, take two kernels: the first finds each
// row's norms and means (reading the row again in every pass, from the caches), with which the second is
// element-wise: its blocks walk down strips of columns, write the rows' gradients and keep the sums over tokens
// in registers. 14 passes instead of 6, of which the caches serve some: 1170 x 28672 bf16 183 - 193 us, 3048 x 11008 181,
// 1170 x 28672 float32 340 - 348 (with loads behind branches 458, 419, 391).
struct RowStats {
  float rs1, rs2, m2, m1;  // m1: mean(t u1) rs1, times y in d_y
};

// A chunk of every input at columns c .. c + kVec - 1 of a row, and what both kernels form of it. The loads have no
// branches, so that those of several chunks go out together: an input that is not given reads the residual's bytes
// instead, for a constant. (Rows narrower than a chunk are loaded element by element.)
template <typename T, bool SMALL>
struct WideChunk {
  static constexpr int V = kVec<T>;
  Place<T> at;
  int c, d;
  float y[V], r[V], dr[V], dh[V], w1[V], w2[V], gt[V];
  __device__ __forceinline__ WideChunk(int first, int width) : at(first, width), c(first), d(width) {}
  __device__ __forceinline__ bool owns(int k) const { return SMALL ? c + k < d : k >= at.skip; }
  __device__ __forceinline__ int column(int k) const { return SMALL ? c + k : at.at + k; }
  // `none` where the input is not given (elements of the chunk before hold the neighbour's values: owns())
  __device__ __forceinline__ void get(const void* p, const void* instead, int64_t offset, float none,
                                      float (&v)[V]) const {
    const T* row = p ? (const T*)p + offset : (const T*)instead;
    if constexpr (SMALL) {
      load_chunk(row, c, d, v);
    } else {
      const uint4 u = load_raw(row, at);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = raw_f32<T>(u, k);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = p ? v[k] : none;
  }
  __device__ __forceinline__ void load_y(const BlockNormArgs& a, int64_t row) {
    get(a.y.p, a.residual.p, row * a.y.ld, 0.f, y);
  }
  __device__ __forceinline__ void load_row(const BlockNormArgs& a, const BlockNormGrads& g, int64_t row) {
    const T* res = (const T*)a.residual.p + row * a.residual.ld;
    get(res, res, 0, 0.f, r);
    get(a.y.p, res, row * a.y.ld, 0.f, y);
    get(g.d_res.p, res, row * g.d_res.ld, 0.f, dr);
    get(g.d_h.p, res, row * g.d_h.ld, 0.f, dh);
    if (a.ld_gate != 0) get(a.gate, res, row * a.ld_gate, 1.f, gt);
  }
  __device__ __forceinline__ void load_weights(const BlockNormArgs& a) {
    get(a.w_post, a.residual.p, 0, 1.f, w1);
    get(a.w_pre, a.residual.p, 0, 1.f, w2);
    if (a.ld_gate == 0) get(a.gate, a.residual.p, 0, 1.f, gt);
  }
  __device__ __forceinline__ void store(T* row, const float (&v)[V]) const {
    if constexpr (SMALL) store_chunk(row, c, d, v);
    else store_own(row, at, v);
  }
  __device__ __forceinline__ float r_new(int k, float ars) const { return fmaf(y[k] * ars * w1[k], gt[k], r[k]); }
  // u2; without a norm behind r', what it holds does not matter (0 * inf would)
  __device__ __forceinline__ float unit(const BlockNormArgs& a, int k, float ars, float rs2) const {
    return a.w_pre ? r_new(k, ars) * rs2 : 0.f;
  }
  __device__ __forceinline__ float grad(int k, const RowStats& s, float u2) const {
    return fmaf(s.rs2, dh[k] * w2[k] - u2 * s.m2, dr[k]);
  }
};

template <typename T, bool SMALL>
__global__ __launch_bounds__(512) void block_norm_stats_kernel(BlockNormArgs a, BlockNormGrads g, RowStats* stats) {
  constexpr int V = kVec<T>;
  __shared__ float red[4][16];
  const int d = a.d, first = (int)threadIdx.x * V, step = (int)blockDim.x * V;
  const float inv_d = 1.0f / (float)d;
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    RowStats st = {1.f, 0.f, 0.f, 0.f};
    __syncthreads();  // the previous row's sums have been read
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll 4
      for (int c = first; c < d; c += step) {
        WideChunk<T, SMALL> x(c, d);
        x.load_y(a, row);
#pragma unroll
        for (int k = 0; k < V; ++k) s[0] = x.owns(k) ? fmaf(x.y[k], x.y[k], s[0]) : s[0];
      }
      block_sum(s, red[0]);
      st.rs1 = rstd_of(s[0], d, a.eps);
    }
    const float ars = a.res_scale * st.rs1;
    if (a.w_pre) {
      float s[2] = {0.f, 0.f};
      for (int c = first; c < d; c += step) {
        WideChunk<T, SMALL> x(c, d);
        x.load_row(a, g, row);
        x.load_weights(a);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float r = x.r_new(k, ars);
          s[0] = x.owns(k) ? fmaf(r, r, s[0]) : s[0];
          s[1] = x.owns(k) ? fmaf(x.dh[k] * x.w2[k], r, s[1]) : s[1];
        }
      }
      block_sum(s, red[1]);
      st.rs2 = rstd_of(s[0], d, a.eps);
      st.m2 = s[1] * st.rs2 * inv_d;
    }
    if (a.w_post) {
      float s[1] = {0.f};
      for (int c = first; c < d; c += step) {
        WideChunk<T, SMALL> x(c, d);
        x.load_row(a, g, row);
        x.load_weights(a);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float t = a.res_scale * x.grad(k, st, x.unit(a, k, ars, st.rs2)) * x.gt[k] * x.w1[k];
          s[0] = x.owns(k) ? fmaf(t, x.y[k] * st.rs1, s[0]) : s[0];
        }
      }
      block_sum(s, red[3]);
      st.m1 = s[0] * inv_d * st.rs1;
    }
    if (threadIdx.x == 0) stats[row] = st;
  }
}

template <typename T, bool SMALL>
__global__ __launch_bounds__(256) void block_norm_columns_kernel(BlockNormArgs a, BlockNormGrads g,
                                                                 const RowStats* stats) {
  constexpr int V = kVec<T>;
  const int d = a.d, c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * V;
  if (c >= d) return;
  float sw1[V], sw2[V], sg[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sw1[k] = sw2[k] = sg[k] = 0.f;
  WideChunk<T, SMALL> x(c, d);
  x.load_weights(a);
#pragma unroll 2
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    x.load_row(a, g, row);
    const RowStats st = stats[row];
    const float ars = a.res_scale * st.rs1;
    float D[V], dy[V], dg[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float u1 = x.y[k] * st.rs1, u2 = x.unit(a, k, ars, st.rs2);
      D[k] = x.grad(k, st, u2);
      const float ad = a.res_scale * D[k], dz = ad * x.gt[k];
      dg[k] = ad * u1 * x.w1[k];
      dy[k] = a.w_post ? st.rs1 * (dz * x.w1[k] - x.y[k] * st.m1) : dz;
      sw1[k] = fmaf(dz, u1, sw1[k]);
      sw2[k] = fmaf(x.dh[k], u2, sw2[k]);
      sg[k] += dg[k];
    }
    if (g.d_residual.p) x.store((T*)g.d_residual.p + row * g.d_residual.ld, D);
    if (g.d_gate.p) x.store((T*)g.d_gate.p + row * g.d_gate.ld, dg);
    if (g.d_y.p) x.store((T*)g.d_y.p + row * g.d_y.ld, dy);
  }
  if (g.partial) {
    const int64_t plane = (int64_t)gridDim.y * d;
    float* p = g.partial + (int64_t)blockIdx.y * d;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (x.owns(k)) {
        p[x.column(k)] = sw1[k];
        p[plane + x.column(k)] = sw2[k];
        p[2 * plane + x.column(k)] = sg[k];
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
  if (c < d) {
#pragma unroll 8
    for (int b = run; b < blocks; b += 16) s += p[(int64_t)b * d + c];
  }
  part[run][threadIdx.x & 63] = s;
  __syncthreads();
  if (run == 0 && c < d) {
    for (int w = 1; w < 16; ++w) s += part[w][threadIdx.x & 63];
    out[c] = s;
  }
}

template <typename F>
hipError_t with_dtype(int dtype, F f) {
  if (dtype == AWQ_DTYPE_BF16) f(Bf16{});
  else if (dtype == AWQ_DTYPE_F16) f(F16{});
  else f(0.f);
  return hipGetLastError();
}

// The block for a row of d elements: as few threads as hold it with `items` chunks each.
int row_threads(int d, int vec, int items) { return ((d + vec * items - 1) / (vec * items) + 63) / 64 * 64; }

// Blocks that keep about `per_cu` threads on each compute unit.
int64_t row_blocks(int64_t n, int threads, int per_cu) {
  const int64_t b = (int64_t)256 * (per_cu / threads > 0 ? per_cu / threads : 1);
  return n < b ? n : b;
}

template <int N>
using Int = std::integral_constant<int, N>;

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, int dtype, Mat res_out, Mat h, hipStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto items, auto keep) {
      constexpr int I = decltype(items)::value;
      const int threads = row_threads(a.d, kVec<T>, I);
      hipLaunchKernelGGL((block_norm_kernel<T, I, 1024, decltype(keep)::value>),
                         dim3((unsigned)row_blocks(a.n, threads, 1024)), dim3(threads), 0, st, a, res_out, h);
    };
    const int chunks = (a.d + kVec<T> - 1) / kVec<T>;
    if (a.d < kVec<T>)
      hipLaunchKernelGGL((block_norm_narrow_kernel<T>), dim3((unsigned)row_blocks((a.n + 255) / 256, 256, 2048)),
                         dim3(256), 0, st, a, res_out, h);
    else if (chunks <= 128) go(Int<1>{}, std::true_type{});
    else if (chunks <= 2048) go(Int<2>{}, std::true_type{});
    else if (chunks <= 4096) go(Int<4>{}, std::false_type{});
    else if constexpr (sizeof(T) == 4) go(Int<8>{}, std::false_type{});
  });
}

// Rows whose gradient is held in registers; the others take the two kernels.
constexpr int kBackwardWidth = 8192;
bool wide_backward(int64_t d) { return d > kBackwardWidth || d < 8; }

// Blocks of partial sums. In registers: two blocks on a compute unit, which is what these allow. Wide: strips
// of at least 1024 columns (float32) by so many rows' strides that about 1024 blocks walk down the strips.
int block_norm_backward_blocks(int64_t n_tokens, int64_t d) {
  if (wide_backward(d)) {
    const int64_t strips = (d + 1023) / 1024, b = (1024 + strips - 1) / strips;
    return (int)(n_tokens < b ? n_tokens : b);
  }
  return (int)row_blocks(n_tokens, row_threads((int)d, 8, 1), 1024);
}

size_t block_norm_backward_partial_floats(int64_t n_tokens, int64_t d) {
  return (size_t)3 * (size_t)block_norm_backward_blocks(n_tokens, d) * (size_t)d;
}

size_t block_norm_backward_stats_bytes(int64_t n_tokens, int64_t d) {
  return wide_backward(d) ? (size_t)n_tokens * sizeof(RowStats) : 0;
}

hipError_t launch_block_norm_backward(const BlockNormArgs& a, int dtype, CMat d_res, CMat d_h, Mat d_y, Mat d_residual,
                                      float* d_w_post, float* d_w_pre, void* d_gate, int64_t ld_d_gate,
                                      void* stats_space, float* partial_space, hipStream_t st) {
  const bool sum_gate = a.ld_gate == 0;
  float* const partial = d_w_post || d_w_pre || (d_gate && sum_gate) ? partial_space : nullptr;
  int blocks = block_norm_backward_blocks(a.n, a.d);
  const BlockNormGrads g{d_res, d_h, d_y, d_residual, {sum_gate ? nullptr : d_gate, ld_d_gate}, partial};
  hipError_t e = with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    constexpr int V = kVec<T>;
    if (wide_backward(a.d)) {
      RowStats* stats = static_cast<RowStats*>(stats_space);
      auto go = [&](auto small) {
        constexpr bool SMALL = decltype(small)::value;
        const int threads = SMALL ? 64 : 512;
        hipLaunchKernelGGL((block_norm_stats_kernel<T, SMALL>), dim3((unsigned)row_blocks(a.n, threads, 2048)),
                           dim3(threads), 0, st, a, g, stats);
        hipLaunchKernelGGL((block_norm_columns_kernel<T, SMALL>),
                           dim3((unsigned)((a.d + 256 * V - 1) / (256 * V)), blocks), dim3(256), 0, st, a, g, stats);
      };
      if (a.d < V || a.d < 8) go(std::true_type{});
      else go(std::false_type{});
      return;
    }
    // float32 rows keep the memory busy with one block on a compute unit, and have half the partial sums to add
    if (sizeof(T) == 4) blocks = (int)row_blocks(a.n, row_threads(a.d, 8, 1), 512);
    auto go = [&](auto items) {
      constexpr int I = decltype(items)::value;
      const dim3 grid((unsigned)blocks), block(row_threads(a.d, V, I));
      auto launch = [&](auto pre) {
        constexpr bool PRE = decltype(pre)::value;
        if (sum_gate) hipLaunchKernelGGL((block_norm_backward_kernel<T, I, false, PRE>), grid, block, 0, st, a, g);
        else hipLaunchKernelGGL((block_norm_backward_kernel<T, I, true, PRE>), grid, block, 0, st, a, g);
      };
      if (a.w_pre) launch(std::true_type{});
      else launch(std::false_type{});
    };
    const int chunks = (a.d + V - 1) / V;
    if (chunks <= 64) go(Int<1>{});
    else if (chunks <= 1024) go(Int<2>{});
    else if constexpr (sizeof(T) == 4) {
      if (chunks <= 1536) go(Int<3>{});
      else go(Int<4>{});
    }
  });
  if (e != hipSuccess || !partial) return e;
  const ColumnSums outs{{d_w_post, d_w_pre, sum_gate ? (float*)d_gate : nullptr}};
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((a.d + 63) / 64), 3), dim3(1024), 0, st, partial, blocks, a.d,
                     outs);
  return hipGetLastError();
}

}  // namespace awq
