// Host side of the C ABI declared in include/awq_attn.h: argument checks, all before any HIP call, and the
// launches. No allocation happens here; every buffer belongs to the caller.
#include <float.h>
#include <math.h>

#include "abi_status.h"
#include "attn.h"
#include "awq_attn.h"

namespace {

using awq::fail;
using awq::hip_fail;
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

int check_tokens(int64_t n_tokens) {
  if (n_tokens < 0) return fail(AWQ_ERR_SHAPE, "n_tokens %lld < 0", (ll)n_tokens);
  if (n_tokens == 0) return fail(AWQ_ERR_NO_TOKENS, "n_tokens == 0");
  if (n_tokens > AWQ_MAX_ATTN_TOKENS)
    return fail(AWQ_ERR_UNSUPPORTED, "%lld tokens: more than %lld", (ll)n_tokens, (ll)AWQ_MAX_ATTN_TOKENS);
  return AWQ_OK;
}

int check_heads(const char* name, int64_t heads) {
  if (heads < 1 || heads > AWQ_MAX_HEADS)
    return fail(AWQ_ERR_SHAPE, "%s %lld outside [1, %d]", name, (ll)heads, AWQ_MAX_HEADS);
  return AWQ_OK;
}

int check_vec(const char* name, const void* p, size_t align) {
  if (!p) return fail(AWQ_ERR_NULL, "%s is NULL", name);
  if (!aligned(p, align)) return fail(AWQ_ERR_UNSUPPORTED, "%s is not %zu-byte aligned", name, align);
  return AWQ_OK;
}

// A required [tokens, heads, width] argument whose elements do not overlap. (The pitch of one token or head means nothing.)
int check_tensor(const char* name, const void* p, int64_t ld, int64_t ld_head, int64_t tokens, int64_t heads, int64_t width,
                 int dtype) {
  TRY(check_vec(name, p, esize(dtype)));
  const int64_t most = (int64_t)1 << 32;
  if (tokens == 1) ld = width * heads > ld_head * heads ? width * heads : ld_head * heads;
  if (heads == 1) ld_head = width;
  if (ld < width || ld_head < width)
    return fail(AWQ_ERR_ARG, "a pitch of %s (%lld, %lld) is below its width %lld", name, (ll)ld, (ll)ld_head, (ll)width);
  if (ld > most || ld_head > most)
    return fail(AWQ_ERR_UNSUPPORTED, "a pitch of %s (%lld, %lld) is too large", name, (ll)ld, (ll)ld_head);
  const bool tokens_outside = ld >= (heads - 1) * ld_head + width, heads_outside = ld_head >= (tokens - 1) * ld + width;
  if (tokens > 1 && heads > 1 && !tokens_outside && !heads_outside)
    return fail(AWQ_ERR_ARG, "the rows of %s overlap (pitches %lld, %lld)", name, (ll)ld, (ll)ld_head);
  return AWQ_OK;
}

// An output that may lie where an input does has to lie there element by element.
int check_in_place(const char* name, const void* out, int64_t ld_out, int64_t ld_out_head, const char* over, const void* in,
                   int64_t ld_in, int64_t ld_in_head, int64_t tokens, int64_t heads) {
  if (out == in && ((tokens > 1 && ld_out != ld_in) || (heads > 1 && ld_out_head != ld_in_head)))
    return fail(AWQ_ERR_ARG, "%s over %s with other pitches", name, over);
  return AWQ_OK;
}

// ---- rotary positions

int rope(const char* x_name, const void* x, int64_t ld_x, int64_t ld_x_head, int dtype, int64_t n_tokens, int64_t n_heads,
         int64_t head_dim, const void* positions, int64_t ld_positions, int position_bytes, int n_axes, const float* inv_freq,
         const int32_t* axis, int64_t rot_dim, int style, float scale, bool backward, const char* out_name, void* out,
         int64_t ld_out, int64_t ld_out_head, void* stream) {
  TRY(check_dtype(dtype));
  TRY(check_tokens(n_tokens));
  TRY(check_heads("n_heads", n_heads));
  if (head_dim < 2 || head_dim > AWQ_MAX_ROPE_DIM)
    return fail(AWQ_ERR_SHAPE, "head_dim %lld outside [2, %d]", (ll)head_dim, AWQ_MAX_ROPE_DIM);
  if (rot_dim < 2 || rot_dim > head_dim || rot_dim % 2)
    return fail(AWQ_ERR_SHAPE, "rot_dim %lld is not even, in [2, %lld]", (ll)rot_dim, (ll)head_dim);
  if (style != AWQ_ROPE_HALF && style != AWQ_ROPE_PAIRS) return fail(AWQ_ERR_ARG, "style %d is not an awq_rope_style", style);
  if (n_axes < 1 || n_axes > AWQ_MAX_ROPE_AXES)
    return fail(AWQ_ERR_ARG, "n_axes %d outside [1, %d]", n_axes, AWQ_MAX_ROPE_AXES);
  if (position_bytes != 4 && position_bytes != 8)
    return fail(AWQ_ERR_UNSUPPORTED, "position_bytes %d is neither 4 nor 8", position_bytes);
  if (!isfinite(scale)) return fail(AWQ_ERR_ARG, "scale %g is not finite", scale);
  TRY(check_vec("positions", positions, (size_t)position_bytes));
  if (n_axes > 1 && (ld_positions < n_tokens || ld_positions > (int64_t)1 << 40))
    return fail(AWQ_ERR_ARG, "the pitch %lld of positions is not in [n_tokens, 2^40]", (ll)ld_positions);
  TRY(check_vec("inv_freq", inv_freq, 4));
  if (axis) TRY(check_vec("axis", axis, 4));
  TRY(check_tensor(x_name, x, ld_x, ld_x_head, n_tokens, n_heads, head_dim, dtype));
  TRY(check_tensor(out_name, out, ld_out, ld_out_head, n_tokens, n_heads, head_dim, dtype));
  TRY(check_in_place(out_name, out, ld_out, ld_out_head, x_name, x, ld_x, ld_x_head, n_tokens, n_heads));
  const awq::RopeArgs a{{x, ld_x, ld_x_head}, {out, ld_out, ld_out_head}, n_tokens, (int)n_heads, (int)head_dim, (int)rot_dim,
                        positions, ld_positions, position_bytes == 8, n_axes, inv_freq, axis, scale,
                        backward ? -scale : scale, out == x, awq::Divisor((uint32_t)n_heads)};
  hipError_t e = awq::launch_rope(a, dtype, style == AWQ_ROPE_PAIRS, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, backward ? "rope_backward launch" : "rope launch");
  return ok();
}

// ---- the cache

int check_head_dim(int64_t d) {
  if (d < 32 || d > AWQ_KV4_MAX_HEAD_DIM || d % 32)
    return fail(AWQ_ERR_SHAPE, "head_dim %lld is not a multiple of 32 up to %d", (ll)d, AWQ_KV4_MAX_HEAD_DIM);
  return AWQ_OK;
}

int check_cache(const uint8_t* codes, int64_t page_codes, const void* params, int64_t page_params, int64_t n_pages,
                int page_size, int64_t n_kv, int64_t head_dim, awq::Kv4Cache* c) {
  TRY(check_heads("n_kv", n_kv));
  TRY(check_head_dim(head_dim));
  if (page_size < AWQ_KV4_MIN_PAGE || page_size > AWQ_KV4_MAX_PAGE || (page_size & (page_size - 1)))
    return fail(AWQ_ERR_SHAPE, "page_size %d is not a power of two from %d to %d", page_size, AWQ_KV4_MIN_PAGE,
                AWQ_KV4_MAX_PAGE);
  if (n_pages < 1 || n_pages > 0x7FFFFFFF) return fail(AWQ_ERR_SHAPE, "n_pages %lld outside [1, 2^31)", (ll)n_pages);
  TRY(check_vec("codes", codes, 16));
  TRY(check_vec("params", params, 16));
  const int64_t groups = (head_dim + AWQ_GROUP_SIZE - 1) / AWQ_GROUP_SIZE;
  const int64_t rows = 2 * n_kv * page_size;
  if (page_codes < rows * (head_dim / 2) || page_params < rows * groups)
    return fail(AWQ_ERR_ARG, "page_codes %lld or page_params %lld is below a page's size (%lld, %lld)", (ll)page_codes,
                (ll)page_params, (ll)(rows * (head_dim / 2)), (ll)(rows * groups));
  if (page_codes % 16 || page_params % 4)
    return fail(AWQ_ERR_UNSUPPORTED, "page_codes %lld is no multiple of 16, or page_params %lld none of 4", (ll)page_codes,
                (ll)page_params);
  if (page_codes > (int64_t)1 << 32 || page_params > (int64_t)1 << 32)
    return fail(AWQ_ERR_UNSUPPORTED, "page_codes %lld or page_params %lld is too large", (ll)page_codes, (ll)page_params);
  *c = awq::Kv4Cache{const_cast<uint8_t*>(codes), (uint32_t*)const_cast<void*>(params), page_codes, page_params, n_pages,
                     __builtin_ctz((unsigned)page_size), (int)n_kv, (int)head_dim, (int)groups};
  return AWQ_OK;
}

int check_slots(const void* slots, int slot_bytes) {
  if (slot_bytes != 4 && slot_bytes != 8)
    return fail(AWQ_ERR_UNSUPPORTED, "slot_bytes %d is neither 4 nor 8", slot_bytes);
  return check_vec("slots", slots, (size_t)slot_bytes);
}

// ---- attention

constexpr int64_t kMostKv = (int64_t)1 << 30;

int check_attention_sizes(int64_t n_tokens, int64_t n_seqs, bool ragged, int64_t n_heads, int64_t n_kv, int64_t head_dim,
                          int64_t window, int64_t max_kv) {
  TRY(check_tokens(n_tokens));
  TRY(check_heads("n_heads", n_heads));
  TRY(check_heads("n_kv", n_kv));
  if (n_heads % n_kv) return fail(AWQ_ERR_SHAPE, "n_heads %lld is no multiple of n_kv %lld", (ll)n_heads, (ll)n_kv);
  TRY(check_head_dim(head_dim));
  if (n_seqs < 1 || n_seqs > AWQ_MAX_ATTN_SEQS)
    return fail(AWQ_ERR_SHAPE, "n_seqs %lld outside [1, %d]", (ll)n_seqs, AWQ_MAX_ATTN_SEQS);
  if (!ragged && n_tokens % n_seqs)
    return fail(AWQ_ERR_SHAPE, "n_tokens %lld is no multiple of n_seqs %lld, and q_offsets is NULL", (ll)n_tokens, (ll)n_seqs);
  if (n_tokens > ((int64_t)1 << 27) / n_heads)  // blocks are numbered in 32 bits of threads
    return fail(AWQ_ERR_UNSUPPORTED, "%lld tokens of %lld heads: too many", (ll)n_tokens, (ll)n_heads);
  if (window < 0) return fail(AWQ_ERR_ARG, "window %lld < 0", (ll)window);
  if (max_kv < 0) return fail(AWQ_ERR_ARG, "max_kv %lld < 0", (ll)max_kv);
  return AWQ_OK;
}

awq::AttnArgs attention_plan(int64_t n_tokens, int64_t n_seqs, bool ragged, int64_t n_heads, int64_t n_kv, int64_t head_dim,
                             int causal, int64_t window, int64_t max_kv, size_t* bytes) {
  awq::AttnArgs a = {};
  a.c.n_kv = (int)n_kv;
  a.c.head_dim = (int)head_dim;
  a.n_tokens = n_tokens;
  a.n_seqs = (int)n_seqs;
  a.n_heads = (int)n_heads;
  a.group = (int)(n_heads / n_kv);
  a.each = (int)(n_tokens / n_seqs);
  a.causal = causal;
  a.window = (int)(window < kMostKv ? window : kMostKv);
  a.max_kv = (int)(max_kv < 1 ? 1 : max_kv < kMostKv ? max_kv : kMostKv);
  *bytes = round_up(awq::plan_attention(&a, ragged), 256);
  return a;
}

}  // namespace

extern "C" {

int awq_rope(const void* x, int64_t ld_x, int64_t ld_x_head, int dtype, int64_t n_tokens, int64_t n_heads, int64_t head_dim,
             const void* positions, int64_t ld_positions, int position_bytes, int n_axes, const float* inv_freq,
             const int32_t* axis, int64_t rot_dim, int style, float scale, void* out, int64_t ld_out, int64_t ld_out_head,
             void* stream) {
  return rope("x", x, ld_x, ld_x_head, dtype, n_tokens, n_heads, head_dim, positions, ld_positions, position_bytes, n_axes,
              inv_freq, axis, rot_dim, style, scale, false, "out", out, ld_out, ld_out_head, stream);
}

int awq_rope_backward(const void* d_out, int64_t ld_d_out, int64_t ld_d_out_head, int dtype, int64_t n_tokens,
                      int64_t n_heads, int64_t head_dim, const void* positions, int64_t ld_positions, int position_bytes,
                      int n_axes, const float* inv_freq, const int32_t* axis, int64_t rot_dim, int style, float scale,
                      void* d_x, int64_t ld_d_x, int64_t ld_d_x_head, void* stream) {
  return rope("d_out", d_out, ld_d_out, ld_d_out_head, dtype, n_tokens, n_heads, head_dim, positions, ld_positions,
              position_bytes, n_axes, inv_freq, axis, rot_dim, style, scale, true, "d_x", d_x, ld_d_x, ld_d_x_head, stream);
}

int awq_kv4_write(const void* k, int64_t ld_k, int64_t ld_k_head, const void* v, int64_t ld_v, int64_t ld_v_head, int dtype,
                  int64_t n_tokens, int64_t n_kv, int64_t head_dim, const void* slots, int slot_bytes, uint8_t* codes,
                  int64_t page_codes, void* params, int64_t page_params, int64_t n_pages, int page_size, void* stream) {
  awq::Kv4MoveArgs a = {};
  TRY(check_dtype(dtype));
  TRY(check_tokens(n_tokens));
  TRY(check_cache(codes, page_codes, params, page_params, n_pages, page_size, n_kv, head_dim, &a.c));
  TRY(check_slots(slots, slot_bytes));
  TRY(check_tensor("k", k, ld_k, ld_k_head, n_tokens, n_kv, head_dim, dtype));
  TRY(check_tensor("v", v, ld_v, ld_v_head, n_tokens, n_kv, head_dim, dtype));
  a.slots = slots;
  a.slots64 = slot_bytes == 8;
  a.n_tokens = n_tokens;
  hipError_t e = awq::launch_kv4_write(a, dtype, {k, ld_k, ld_k_head}, {v, ld_v, ld_v_head}, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv4_write launch");
  return ok();
}

int awq_kv4_read(const uint8_t* codes, int64_t page_codes, const void* params, int64_t page_params, int64_t n_pages,
                 int page_size, int64_t n_kv, int64_t head_dim, const void* slots, int slot_bytes, int64_t n_tokens,
                 int dtype, void* k, int64_t ld_k, int64_t ld_k_head, void* v, int64_t ld_v, int64_t ld_v_head,
                 void* stream) {
  awq::Kv4MoveArgs a = {};
  TRY(check_dtype(dtype));
  TRY(check_tokens(n_tokens));
  TRY(check_cache(codes, page_codes, params, page_params, n_pages, page_size, n_kv, head_dim, &a.c));
  TRY(check_slots(slots, slot_bytes));
  if (!k && !v) return fail(AWQ_ERR_NULL, "neither k nor v is given");
  if (k) TRY(check_tensor("k", k, ld_k, ld_k_head, n_tokens, n_kv, head_dim, dtype));
  if (v) TRY(check_tensor("v", v, ld_v, ld_v_head, n_tokens, n_kv, head_dim, dtype));
  if (k == v) return fail(AWQ_ERR_ARG, "k and v are the same buffer");
  a.slots = slots;
  a.slots64 = slot_bytes == 8;
  a.n_tokens = n_tokens;
  hipError_t e = awq::launch_kv4_read(a, dtype, {k, ld_k, ld_k_head}, {v, ld_v, ld_v_head}, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv4_read launch");
  return ok();
}

size_t awq_kv4_attention_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int ragged, int64_t n_heads, int64_t n_kv,
                                         int64_t head_dim, int causal, int64_t window, int64_t max_kv) {
  if (check_attention_sizes(n_tokens, n_seqs, ragged != 0, n_heads, n_kv, head_dim, window, max_kv) != AWQ_OK) {
    ok();  // a query leaves no error behind
    return 0;
  }
  size_t bytes;  // (of max_kv 0: enough for any table)
  attention_plan(n_tokens, n_seqs, ragged != 0, n_heads, n_kv, head_dim, causal, window, max_kv ? max_kv : kMostKv, &bytes);
  return bytes;
}

int awq_kv4_attention(const void* q, int64_t ld_q, int64_t ld_q_head, int q_dtype, int64_t n_tokens, int64_t n_heads,
                      int64_t n_kv, int64_t head_dim, const uint8_t* codes, int64_t page_codes, const void* params,
                      int64_t page_params, int64_t n_pages, int page_size, const int32_t* table, int64_t ld_table,
                      int64_t table_width, const int32_t* kv_len, const int32_t* q_offsets, int64_t n_seqs, float scale,
                      int causal, int64_t window, int64_t max_kv, void* out, int64_t ld_out, int64_t ld_out_head,
                      int out_dtype, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (q_dtype != AWQ_DTYPE_BF16 && q_dtype != AWQ_DTYPE_F16)
    return fail(AWQ_ERR_UNSUPPORTED, "q_dtype %d: AWQ_DTYPE_BF16 or AWQ_DTYPE_F16", q_dtype);
  if (out_dtype != AWQ_DTYPE_F32 && out_dtype != q_dtype)
    return fail(AWQ_ERR_UNSUPPORTED, "out_dtype %d: AWQ_DTYPE_F32 or that of q", out_dtype);
  TRY(check_attention_sizes(n_tokens, n_seqs, q_offsets != nullptr, n_heads, n_kv, head_dim, window, max_kv));
  awq::Kv4Cache c;
  TRY(check_cache(codes, page_codes, params, page_params, n_pages, page_size, n_kv, head_dim, &c));
  TRY(check_vec("table", table, 4));
  TRY(check_vec("kv_len", kv_len, 4));
  if (q_offsets) TRY(check_vec("q_offsets", q_offsets, 4));
  if (table_width < 1 || (n_seqs > 1 && ld_table < table_width))
    return fail(AWQ_ERR_ARG, "table_width %lld is below 1 or above the pitch %lld of table", (ll)table_width, (ll)ld_table);
  if (table_width > kMostKv / page_size || ld_table > (int64_t)1 << 40)
    return fail(AWQ_ERR_UNSUPPORTED, "%lld pages of %d tokens, or a pitch of %lld: too many", (ll)table_width, page_size,
                (ll)ld_table);
  if (!isfinite(scale)) return fail(AWQ_ERR_ARG, "scale %g is not finite", scale);
  TRY(check_tensor("q", q, ld_q, ld_q_head, n_tokens, n_heads, head_dim, q_dtype));
  TRY(check_tensor("out", out, ld_out, ld_out_head, n_tokens, n_heads, head_dim, out_dtype));
  if (out == q && out_dtype != q_dtype) return fail(AWQ_ERR_ARG, "out over q of another type");
  TRY(check_in_place("out", out, ld_out, ld_out_head, "q", q, ld_q, ld_q_head, n_tokens, n_heads));
  if (lse) TRY(check_vec("lse", lse, 4));
  size_t need;
  awq::AttnArgs a = attention_plan(n_tokens, n_seqs, q_offsets != nullptr, n_heads, n_kv, head_dim, causal, window,
                                   max_kv ? max_kv : table_width * page_size, &need);
  // units of the split are counted in 32 bits; tables that could hold more are not split
  if ((int64_t)a.n_tiles * n_kv * (table_width * page_size / awq::kUnit + 1) > 0x7FFFFFFF) a.n_blocks = 0, need = 0;
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(AWQ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (!aligned(workspace, 256)) return fail(AWQ_ERR_UNSUPPORTED, "the workspace is not 256-byte aligned");
    awq::place_workspace(&a, workspace);
  }
  a.c = c;
  a.q = {q, ld_q, ld_q_head};
  a.out = {out, ld_out, ld_out_head};
  a.out_f32 = out_dtype == AWQ_DTYPE_F32;
  a.lse = lse;
  a.table = table;
  a.kv_len = kv_len;
  a.q_offsets = q_offsets;
  a.ld_table = ld_table;
  a.table_width = (int)table_width;
  const double in_base_2 = (double)scale * 1.44269504088896340736;  // float32's largest at most
  a.scale = (float)fmin(fmax(in_base_2, -(double)FLT_MAX), (double)FLT_MAX);
  hipError_t e = awq::launch_kv4_attention(a, q_dtype == AWQ_DTYPE_BF16, (hipStream_t)stream);
  if (e != hipSuccess) return hip_fail(e, "kv4_attention launch");
  return ok();
}

}  // extern "C"
