// Host side of the C ABI declared in include/awq_moe.h: argument checks, all before any HIP call, and the
// launches. No allocation happens here; every buffer belongs to the caller.
#include <math.h>

#include "abi_status.h"
#include "awq_moe.h"
#include "moe.h"

static_assert(AWQ_MAX_NORM_WIDTH == awq::kMaxNormWidth, "one bound for the header and the kernels");

namespace {

using awq::CMat;
using awq::fail;
using awq::hip_fail;
using awq::Mat;
using awq::ok;

typedef long long ll;

#define TRY(expr)                \
  do {                           \
    int _s = (expr);             \
    if (_s != AWQ_OK) return _s; \
  } while (0)

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
size_t esize(int dtype) { return dtype == AWQ_DTYPE_F32 ? 4 : 2; }

int check_dtype(int dtype) {
  if (dtype != AWQ_DTYPE_F32 && dtype != AWQ_DTYPE_BF16 && dtype != AWQ_DTYPE_F16)
    return fail(AWQ_ERR_UNSUPPORTED, "dtype %d is not an awq_dtype", dtype);
  return AWQ_OK;
}

// A required matrix argument of rows of `width` elements.
int check_mat(const char* name, const void* p, int64_t ld, int64_t width, int dtype) {
  if (!p) return fail(AWQ_ERR_NULL, "%s is NULL", name);
  if (ld < width) return fail(AWQ_ERR_ARG, "the pitch %lld of %s is below its width %lld", (ll)ld, name, (ll)width);
  if (ld > ((int64_t)1 << 40)) return fail(AWQ_ERR_UNSUPPORTED, "the pitch %lld of %s is too large", (ll)ld, name);
  if (!aligned(p, esize(dtype))) return fail(AWQ_ERR_UNSUPPORTED, "%s is not element-aligned", name);
  return AWQ_OK;
}

// An output that may lie where an input does has to lie there row by row: with another pitch a row's output would cover
// rows that other blocks still read.
int check_in_place(const char* name, const void* out, int64_t ld_out, const char* over, const void* in, int64_t ld_in,
                   int64_t rows) {
  if (out && out == in && ld_out != ld_in && rows > 1)
    return fail(AWQ_ERR_ARG, "%s over %s with another pitch (%lld, %lld)", name, over, (ll)ld_out, (ll)ld_in);
  return AWQ_OK;
}

int check_vec(const char* name, const void* p, size_t align) {
  if (!p) return fail(AWQ_ERR_NULL, "%s is NULL", name);
  if (!aligned(p, align)) return fail(AWQ_ERR_UNSUPPORTED, "%s is not %zu-byte aligned", name, align);
  return AWQ_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return AWQ_OK;
  if (!ws || have < need) return fail(AWQ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? have : 0, need);
  if (!aligned(ws, 256)) return fail(AWQ_ERR_UNSUPPORTED, "the workspace is not 256-byte aligned");
  return AWQ_OK;
}

// ---- norms

bool norm_sizes_ok(int64_t n, int64_t d) { return n > 0 && n <= 0x7FFFFFFF && d > 0 && d <= AWQ_MAX_NORM_WIDTH; }

int check_norm(const void* y, int64_t ld_y, const void* residual, int64_t ld_residual, int dtype, int64_t n, int64_t d,
               const void* w_post, const void* gate, int64_t ld_gate, float res_scale, const void* w_pre, float eps,
               awq::BlockNormArgs* a) {
  TRY(check_dtype(dtype));
  if (n < 0 || d <= 0) return fail(AWQ_ERR_SHAPE, "n_tokens %lld must be >= 0 and d %lld > 0", (ll)n, (ll)d);
  if (n == 0) return fail(AWQ_ERR_NO_TOKENS, "n_tokens == 0");
  if (n > 0x7FFFFFFF) return fail(AWQ_ERR_UNSUPPORTED, "n_tokens %lld is too large", (ll)n);
  if (d > AWQ_MAX_NORM_WIDTH)
    return fail(AWQ_ERR_UNSUPPORTED, "d %lld: norms up to %d wide are implemented", (ll)d, AWQ_MAX_NORM_WIDTH);
  if (!(eps >= 0.0f) || isinf(eps)) return fail(AWQ_ERR_ARG, "eps %g is not a finite number >= 0", eps);
  if (!y && (w_post || gate)) return fail(AWQ_ERR_NULL, "w_post and gate need y");
  if (y) TRY(check_mat("y", y, ld_y, d, dtype));
  TRY(check_mat("residual", residual, ld_residual, d, dtype));
  if (w_post) TRY(check_vec("w_post", w_post, esize(dtype)));
  if (w_pre) TRY(check_vec("w_pre", w_pre, esize(dtype)));
  if (gate) TRY(check_mat("gate", gate, ld_gate == 0 ? d : ld_gate, d, dtype));
  // The kernels take a pitch for a gate of each token's own, and zeros times the scale for a y that is not there: neither
  // is passed on without its matrix.
  *a = awq::BlockNormArgs{{y, ld_y}, {residual, ld_residual}, n, (int)d, w_post, w_pre, gate, gate ? ld_gate : 0,
                          y ? res_scale : 1.0f, eps};
  return AWQ_OK;
}

// ---- routes

int check_slots(int64_t n_tokens, int top_k) {
  if (n_tokens < 0) return fail(AWQ_ERR_SHAPE, "n_tokens %lld < 0", (ll)n_tokens);
  if (top_k < 1 || top_k > AWQ_MAX_TOP_K) return fail(AWQ_ERR_ARG, "top_k %d outside [1, %d]", top_k, AWQ_MAX_TOP_K);
  if (n_tokens == 0) return fail(AWQ_ERR_NO_TOKENS, "n_tokens == 0");
  if (n_tokens > AWQ_MAX_SLOTS / top_k)
    return fail(AWQ_ERR_UNSUPPORTED, "%lld tokens x %d choices: more than %lld slots", (ll)n_tokens, top_k,
                (ll)AWQ_MAX_SLOTS);
  return AWQ_OK;
}

int check_experts(int n_experts) {
  if (n_experts < 1 || n_experts > AWQ_MAX_EXPERTS)
    return fail(AWQ_ERR_ARG, "n_experts %d outside [1, %d]", n_experts, AWQ_MAX_EXPERTS);
  return AWQ_OK;
}

int check_ids(const void* ids, int id_bytes) {
  if (id_bytes != 4 && id_bytes != 8) return fail(AWQ_ERR_UNSUPPORTED, "id_bytes %d is neither 4 nor 8", id_bytes);
  return check_vec("expert_ids", ids, (size_t)id_bytes);
}

int check_rows(int64_t n_rows) {
  if (n_rows < 0) return fail(AWQ_ERR_SHAPE, "n_rows %lld < 0", (ll)n_rows);
  if (n_rows > AWQ_MAX_SLOTS)
    return fail(AWQ_ERR_UNSUPPORTED, "%lld rows: more than %lld", (ll)n_rows, (ll)AWQ_MAX_SLOTS);
  if (n_rows == 0) return fail(AWQ_ERR_NO_TOKENS, "n_rows == 0");
  return AWQ_OK;
}

// Rows of 32 MiB and more, the second-level caches together, are stored past these: they would not hold them for
// their reader, and stores that scatter rows leave less room for what is read. Gathering 134 MB with multipliers
// 90 -> 56 us, 67 MB 53 -> 31, without them 60 -> 54; the gradient of combining 134 MB 112 -> 111 us.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

int check_route(int dtype, int64_t n_tokens, int top_k, int64_t d, int64_t n_rows, const int32_t* position,
                const void* ids, int id_bytes, const float* scales, int n_experts, awq::RouteArgs* a) {
  TRY(check_dtype(dtype));
  TRY(check_slots(n_tokens, top_k));
  if (d <= 0) return fail(AWQ_ERR_SHAPE, "d %lld must be > 0", (ll)d);
  if (d > AWQ_MAX_ROW_WIDTH) return fail(AWQ_ERR_UNSUPPORTED, "d %lld is too large", (ll)d);
  TRY(check_rows(n_rows));
  TRY(check_vec("position", position, 4));
  if (scales) {
    TRY(check_experts(n_experts));
    TRY(check_ids(ids, id_bytes));
    TRY(check_vec("in_scales", scales, 4));
  }
  *a = awq::RouteArgs{n_tokens, (int)d, top_k, (int)n_rows, position, ids, id_bytes == 8, scales, n_experts,
                      n_rows * d * (int64_t)esize(dtype) >= kStreamBytes};
  return AWQ_OK;
}

// ---- the experts' products

// `x` is [n_rows, x_width], `y` [n_rows, y_width]. The pitch of a single row means nothing: *ld_x becomes one that the
// kernels take.
int check_grouped(const char* x_name, const void* x, int64_t* ld_x, int64_t x_width, int x_dtype, const uint8_t* codes,
                  const uint16_t* steps, const uint8_t* zeros, const int32_t* offsets, int n_experts, int64_t n_rows,
                  int64_t d_in, int64_t d_out, const char* y_name, void* y, int64_t ld_y, int64_t y_width,
                  int y_dtype) {
  if (x_dtype != AWQ_DTYPE_BF16 && x_dtype != AWQ_DTYPE_F16)
    return fail(AWQ_ERR_UNSUPPORTED, "dtype %d of %s: AWQ_DTYPE_BF16 or AWQ_DTYPE_F16", x_dtype, x_name);
  if (y_dtype != AWQ_DTYPE_F32 && y_dtype != x_dtype)
    return fail(AWQ_ERR_UNSUPPORTED, "dtype %d of %s: AWQ_DTYPE_F32 or that of %s", y_dtype, y_name, x_name);
  if (d_out <= 0) return fail(AWQ_ERR_SHAPE, "d_out %lld must be > 0", (ll)d_out);
  if (d_in <= 0 || d_in % AWQ_GROUP_SIZE)
    return fail(AWQ_ERR_SHAPE, "d_in %lld is not a positive multiple of %d", (ll)d_in, AWQ_GROUP_SIZE);
  TRY(check_rows(n_rows));
  TRY(check_experts(n_experts));
  TRY(check_vec("codes", codes, 16));
  TRY(check_vec("steps_f16", steps, 2));
  TRY(check_vec("zeros_u4", zeros, 1));
  TRY(check_vec("offsets", offsets, 4));
  TRY(check_mat(x_name, x, *ld_x, x_width, x_dtype));
  TRY(check_mat(y_name, y, ld_y, y_width, y_dtype));
  if (n_rows == 1) *ld_x = (x_width + 7) / 8 * 8;
  if (*ld_x % 8 || !aligned(x, 16))
    return fail(AWQ_ERR_UNSUPPORTED, "%s must be 16-byte aligned with a pitch of a multiple of 8", x_name);
  // byte offsets inside a tile of 256 rows of x, or of 256 rows of codes, are signed 32-bit
  if (*ld_x > 0x3FFFFF || d_in > 0x3FFF80 || d_out > 0x3FFFFF)
    return fail(AWQ_ERR_UNSUPPORTED, "%s pitch %lld, d_in %lld or d_out %lld too large for 32-bit tile offsets", x_name,
                (ll)*ld_x, (ll)d_in, (ll)d_out);
  if (d_out > 0x7FFFFFFF / (d_in / 2))
    return fail(AWQ_ERR_UNSUPPORTED, "an expert of %lld x %lld weights is too large for 32-bit offsets", (ll)d_out,
                (ll)d_in);
  return AWQ_OK;
}

}  // namespace

extern "C" {

int awq_block_norm(const void* y, int64_t ld_y, const void* residual, int64_t ld_residual, int dtype, int64_t n_tokens,
                   int64_t d, const void* w_post, const void* gate, int64_t ld_gate, float res_scale,
                   const void* w_pre, float eps, void* res_out, int64_t ld_res_out, void* h, int64_t ld_h,
                   void* stream) {
  awq::BlockNormArgs a;
  TRY(check_norm(y, ld_y, residual, ld_residual, dtype, n_tokens, d, w_post, gate, ld_gate, res_scale, w_pre, eps, &a));
  if ((w_pre == nullptr) != (h == nullptr)) return fail(AWQ_ERR_NULL, "w_pre and h go together");
  if (!y && res_out) return fail(AWQ_ERR_NULL, "res_out needs y");
  if (!res_out && !h) return fail(AWQ_ERR_NULL, "neither res_out nor h is given");
  if (res_out) TRY(check_mat("res_out", res_out, ld_res_out, d, dtype));
  if (h) TRY(check_mat("h", h, ld_h, d, dtype));
  if (h && h == res_out) return fail(AWQ_ERR_ARG, "h and res_out are the same buffer");
  TRY(check_in_place("res_out", res_out, ld_res_out, "y", y, ld_y, n_tokens));
  TRY(check_in_place("res_out", res_out, ld_res_out, "residual", residual, ld_residual, n_tokens));
  TRY(check_in_place("h", h, ld_h, "y", y, ld_y, n_tokens));
  TRY(check_in_place("h", h, ld_h, "residual", residual, ld_residual, n_tokens));
  hipError_t e = awq::launch_block_norm(a, dtype, {res_out, ld_res_out}, {h, ld_h}, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "block_norm launch");
  return ok();
}

size_t awq_block_norm_backward_workspace_bytes(int64_t n_tokens, int64_t d) {
  if (!norm_sizes_ok(n_tokens, d)) return 0;
  return round_up(awq::block_norm_backward_stats_bytes(n_tokens, d), 256) +
         round_up(awq::block_norm_backward_partial_floats(n_tokens, d) * sizeof(float), 256);
}

int awq_block_norm_backward(const void* y, int64_t ld_y, const void* residual, int64_t ld_residual, int dtype,
                            int64_t n_tokens, int64_t d, const void* w_post, const void* gate, int64_t ld_gate,
                            float res_scale, const void* w_pre, float eps, const void* d_res_out,
                            int64_t ld_d_res_out, const void* d_h, int64_t ld_d_h, void* d_y, int64_t ld_d_y,
                            void* d_residual, int64_t ld_d_residual, float* d_w_post, float* d_w_pre, void* d_gate,
                            int64_t ld_d_gate, void* workspace, size_t workspace_bytes, void* stream) {
  awq::BlockNormArgs a;
  TRY(check_norm(y, ld_y, residual, ld_residual, dtype, n_tokens, d, w_post, gate, ld_gate, res_scale, w_pre, eps, &a));
  if ((w_pre == nullptr) != (d_h == nullptr)) return fail(AWQ_ERR_NULL, "w_pre and d_h go together");
  if (!d_res_out && !d_h) return fail(AWQ_ERR_NULL, "neither d_res_out nor d_h is given");
  if (d_res_out) TRY(check_mat("d_res_out", d_res_out, ld_d_res_out, d, dtype));
  if (d_h) TRY(check_mat("d_h", d_h, ld_d_h, d, dtype));
  if (!d_y && !d_residual && !d_w_post && !d_w_pre && !d_gate) return fail(AWQ_ERR_NULL, "no output is given");
  if (d_y && !y) return fail(AWQ_ERR_NULL, "d_y needs y");
  if (d_w_post && !w_post) return fail(AWQ_ERR_NULL, "d_w_post needs w_post");
  if (d_w_pre && !w_pre) return fail(AWQ_ERR_NULL, "d_w_pre needs w_pre");
  if (d_gate && !gate) return fail(AWQ_ERR_NULL, "d_gate needs gate");
  if (d_y) TRY(check_mat("d_y", d_y, ld_d_y, d, dtype));
  if (d_residual) TRY(check_mat("d_residual", d_residual, ld_d_residual, d, dtype));
  TRY(check_in_place("d_residual", d_residual, ld_d_residual, "d_res_out", d_res_out, ld_d_res_out, n_tokens));
  TRY(check_in_place("d_y", d_y, ld_d_y, "d_h", d_h, ld_d_h, n_tokens));
  if (d_w_post) TRY(check_vec("d_w_post", d_w_post, 4));
  if (d_w_pre) TRY(check_vec("d_w_pre", d_w_pre, 4));
  const bool sum_gate = d_gate && ld_gate == 0;
  if (sum_gate) TRY(check_vec("d_gate", d_gate, 4));
  else if (d_gate) TRY(check_mat("d_gate", d_gate, ld_d_gate, d, dtype));
  TRY(check_workspace(workspace, workspace_bytes, awq_block_norm_backward_workspace_bytes(n_tokens, d)));
  const size_t stats = round_up(awq::block_norm_backward_stats_bytes(n_tokens, d), 256);
  hipError_t e = awq::launch_block_norm_backward(a, dtype, {d_res_out, ld_d_res_out}, {d_h, ld_d_h}, {d_y, ld_d_y},
                                                 {d_residual, ld_d_residual}, d_w_post, d_w_pre, d_gate, ld_d_gate,
                                                 workspace, (float*)((char*)workspace + stats), (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "block_norm_backward launch");
  return ok();
}

size_t awq_moe_sort_workspace_bytes(int64_t n_tokens, int top_k, int n_experts) {
  if (n_tokens <= 0 || top_k < 1 || top_k > AWQ_MAX_TOP_K || n_experts < 1 || n_experts > AWQ_MAX_EXPERTS ||
      n_tokens > AWQ_MAX_SLOTS / top_k)
    return 0;
  const int blocks = awq::moe_sort_blocks(n_tokens * top_k);
  return blocks == 1 ? 0 : round_up((size_t)blocks * (size_t)n_experts * sizeof(int32_t), 256);
}

int awq_moe_sort(const void* expert_ids, int id_bytes, int64_t n_tokens, int top_k, int n_experts, int32_t* offsets,
                 int32_t* order, int32_t* position, void* workspace, size_t workspace_bytes, void* stream) {
  TRY(check_slots(n_tokens, top_k));
  TRY(check_experts(n_experts));
  TRY(check_ids(expert_ids, id_bytes));
  TRY(check_vec("offsets", offsets, 4));
  TRY(check_vec("order", order, 4));
  TRY(check_vec("position", position, 4));
  TRY(check_workspace(workspace, workspace_bytes, awq_moe_sort_workspace_bytes(n_tokens, top_k, n_experts)));
  hipError_t e = awq::launch_moe_sort(expert_ids, id_bytes == 8, (int)(n_tokens * top_k), n_experts, offsets, order,
                                      position, (int32_t*)workspace, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_sort launch");
  return ok();
}

int awq_moe_gather(const void* x, int64_t ld_x, int dtype, int64_t n_tokens, int64_t d, const int32_t* position,
                   int top_k, const void* expert_ids, int id_bytes, const float* in_scales, int n_experts, void* rows,
                   int64_t ld_rows, int64_t n_rows, void* stream) {
  awq::RouteArgs a;
  TRY(check_route(dtype, n_tokens, top_k, d, n_rows, position, expert_ids, id_bytes, in_scales, n_experts, &a));
  TRY(check_mat("x", x, ld_x, d, dtype));
  TRY(check_mat("rows", rows, ld_rows, d, dtype));
  hipError_t e = awq::launch_moe_gather(a, dtype, {x, ld_x}, {rows, ld_rows}, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_gather launch");
  return ok();
}

int awq_moe_gather_backward(const void* d_rows, int64_t ld_d_rows, int dtype, int64_t n_rows, int64_t d,
                            const int32_t* position, int64_t n_tokens, int top_k, const void* expert_ids, int id_bytes,
                            const float* in_scales, int n_experts, void* d_x, int64_t ld_d_x, void* stream) {
  awq::RouteArgs a;
  TRY(check_route(dtype, n_tokens, top_k, d, n_rows, position, expert_ids, id_bytes, in_scales, n_experts, &a));
  TRY(check_mat("d_rows", d_rows, ld_d_rows, d, dtype));
  TRY(check_mat("d_x", d_x, ld_d_x, d, dtype));
  hipError_t e = awq::launch_moe_combine(a, dtype, {d_rows, ld_d_rows}, nullptr, {d_x, ld_d_x}, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_gather_backward launch");
  return ok();
}

int awq_moe_combine(const void* rows, int64_t ld_rows, int dtype, int64_t n_rows, int64_t d, const int32_t* position,
                    const float* weights, int64_t n_tokens, int top_k, void* out, int64_t ld_out, void* stream) {
  awq::RouteArgs a;
  TRY(check_route(dtype, n_tokens, top_k, d, n_rows, position, nullptr, 4, nullptr, 1, &a));
  TRY(check_vec("weights", weights, 4));
  TRY(check_mat("rows", rows, ld_rows, d, dtype));
  TRY(check_mat("out", out, ld_out, d, dtype));
  hipError_t e = awq::launch_moe_combine(a, dtype, {rows, ld_rows}, weights, {out, ld_out}, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_combine launch");
  return ok();
}

int awq_moe_combine_backward(const void* d_out, int64_t ld_d_out, const void* rows, int64_t ld_rows, int dtype,
                             int64_t n_rows, int64_t d, const int32_t* position, const float* weights,
                             int64_t n_tokens, int top_k, void* d_rows, int64_t ld_d_rows, float* d_weights,
                             void* stream) {
  awq::RouteArgs a;
  TRY(check_route(dtype, n_tokens, top_k, d, n_rows, position, nullptr, 4, nullptr, 1, &a));
  if (!d_rows && !d_weights) return fail(AWQ_ERR_NULL, "neither d_rows nor d_weights is given");
  TRY(check_vec("weights", weights, 4));
  TRY(check_mat("d_out", d_out, ld_d_out, d, dtype));
  TRY(check_mat("rows", rows, ld_rows, d, dtype));
  if (d_rows) TRY(check_mat("d_rows", d_rows, ld_d_rows, d, dtype));
  TRY(check_in_place("d_rows", d_rows, ld_d_rows, "rows", rows, ld_rows, n_rows));
  if (d_weights) TRY(check_vec("d_weights", d_weights, 4));
  hipError_t e = awq::launch_moe_combine_backward(a, dtype, {d_out, ld_d_out}, {rows, ld_rows}, weights,
                                                  {d_rows, ld_d_rows}, d_weights, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "moe_combine_backward launch");
  return ok();
}

int awq_w4a16_grouped_gemm(const void* x, int64_t ld_x, int x_dtype, const uint8_t* codes, const uint16_t* steps_f16,
                           const uint8_t* zeros_u4, const int32_t* offsets, int n_experts, int64_t n_rows,
                           int64_t d_in, int64_t d_out, int mode, void* y, int64_t ld_y, int y_dtype, void* stream) {
  if (mode != AWQ_GROUPED_PLAIN && mode != AWQ_GROUPED_GATED_SILU && mode != AWQ_GROUPED_GATED_RELU)
    return fail(AWQ_ERR_ARG, "mode %d is not an awq_grouped_mode", mode);
  const bool gate = mode != AWQ_GROUPED_PLAIN;
  if (gate && d_out % 2) return fail(AWQ_ERR_SHAPE, "d_out %lld of a gate/up pair is odd", (ll)d_out);
  TRY(check_grouped("x", x, &ld_x, d_in, x_dtype, codes, steps_f16, zeros_u4, offsets, n_experts, n_rows, d_in, d_out,
                    "y", y, ld_y, gate ? d_out / 2 : d_out, y_dtype));
  const awq::GroupedArgs a{{x, ld_x}, codes, steps_f16, zeros_u4, offsets, n_experts, (int)n_rows, (int)d_in,
                           (int)d_out, mode, {y, ld_y}};
  hipError_t e = awq::launch_w4a16_grouped(a, x_dtype == AWQ_DTYPE_F16 ? 1 : 0, y_dtype == AWQ_DTYPE_F32,
                                           (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "w4a16_grouped_gemm launch");
  return ok();
}

int awq_w4a16_grouped_gemm_backward(const void* d_y, int64_t ld_d_y, int dy_dtype, const uint8_t* codes,
                                    const uint16_t* steps_f16, const uint8_t* zeros_u4, const int32_t* offsets,
                                    int n_experts, int64_t n_rows, int64_t d_in, int64_t d_out, void* d_x,
                                    int64_t ld_d_x, int dx_dtype, void* stream) {
  TRY(check_grouped("d_y", d_y, &ld_d_y, d_out, dy_dtype, codes, steps_f16, zeros_u4, offsets, n_experts, n_rows, d_in,
                    d_out, "d_x", d_x, ld_d_x, d_in, dx_dtype));
  const awq::GroupedArgs a{{d_y, ld_d_y}, codes, steps_f16, zeros_u4, offsets, n_experts, (int)n_rows, (int)d_in,
                           (int)d_out, AWQ_GROUPED_PLAIN, {d_x, ld_d_x}};
  hipError_t e = awq::launch_w4a16_grouped_backward(a, dy_dtype == AWQ_DTYPE_F16 ? 1 : 0, dx_dtype == AWQ_DTYPE_F32,
                                                    (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "w4a16_grouped_gemm_backward launch");
  return ok();
}

}  // extern "C"
