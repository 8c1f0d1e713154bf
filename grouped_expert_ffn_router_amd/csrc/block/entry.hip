// C ABI of the operators around the experts' products.
//
// One translation unit with ops/entry.hip and api.hip, whose argument checks,
// error message and kernel timing these entry points share; their kernels are
// in the other files of this directory.

#include "../ops/entry.hip"

#include "block.h"

namespace {

int act_ok(int32_t act_dtype) {
  if (act_dtype != MOE_ACT_BF16 && act_dtype != MOE_ACT_F32)
    return fail(MOE_EDTYPE, "act_dtype %d is not MOE_ACT_BF16 (0) or MOE_ACT_F32 (1)", act_dtype);
  return MOE_OK;
}

// Rows of `cols` values of `size` bytes at p: address and stride multiples of `unit`, the stride at least a row.
int rows_ok(const void* p, int64_t stride, int64_t cols, int64_t size, int64_t unit, const char* what) {
  if (!p) return fail(MOE_EINVAL, "%s is NULL", what);
  if ((uintptr_t)p % unit || stride % unit || stride < cols * size)
    return fail(MOE_EALIGN, "%s: address and stride must be multiples of %lld bytes, the stride at least a row", what,
                (long long)unit);
  return MOE_OK;
}

int mx8_strides_ok(int64_t cols, int64_t code_stride, int64_t scale_stride, const char* what) {
  if (code_stride % 16 || code_stride < cols)
    return fail(MOE_EALIGN, "%s: code_stride_bytes must be a multiple of 16 and >= cols", what);
  if (scale_stride % 16 || scale_stride < mx_scale_bytes(cols))
    return fail(MOE_EALIGN, "%s: scale_stride_bytes must be a multiple of 16 and >= cols / 32 rounded up to 16", what);
  return MOE_OK;
}

int mx8_rows_ok(const moe_mx_rows* r, int64_t cols, const char* what) {
  if (!r) return fail(MOE_EINVAL, "%s is NULL", what);
  NEED(r->codes, what);
  NEED(r->scales, what);
  return mx8_strides_ok(cols, r->code_stride_bytes, r->scale_stride_bytes, what);
}

Rows8 rows8(const moe_mx_rows* r) {
  return {(uint8_t*)r->codes, (uint8_t*)r->scales, r->code_stride_bytes, r->scale_stride_bytes};
}

// rows * cols within 2^40, without overflow.
int size_ok(int64_t rows, int64_t cols) {
  if (rows < 0) return fail(MOE_EINVAL, "rows < 0");
  if (rows > (1ll << 40) / cols) return fail(MOE_EINVAL, "rows * cols exceeds 2^40");
  return MOE_OK;
}

int norm_ok(int32_t act_dtype, int64_t rows, int64_t cols, int32_t weight_dtype, float eps) {
  int rc = act_ok(act_dtype);
  if (rc) return rc;
  if (weight_dtype != MOE_ACT_BF16 && weight_dtype != MOE_ACT_F32)
    return fail(MOE_EDTYPE, "weight_dtype %d is not MOE_ACT_BF16 (0) or MOE_ACT_F32 (1)", weight_dtype);
  if (cols <= 0 || cols > MOE_NORM_COLS_MAX)
    return fail(MOE_EINVAL, "cols (%lld) out of range [1, %d]", (long long)cols, MOE_NORM_COLS_MAX);
  if (!(eps >= 0.f) || eps > 3e38f) return fail(MOE_EINVAL, "eps must be finite and not negative");
  return size_ok(rows, cols);
}

int weight_ok(const void* weight, int32_t weight_dtype) {
  if (!weight) return fail(MOE_EINVAL, "weight is NULL");
  if ((uintptr_t)weight % (weight_dtype == MOE_ACT_BF16 ? 2 : 4))
    return fail(MOE_EALIGN, "weight is not aligned to its values");
  return MOE_OK;
}

int rule_ok(const moe_router_rule* r, int64_t tokens, int32_t n_experts, int32_t top_k, SelectRule* q) {
  if (!r) return fail(MOE_EINVAL, "rule is NULL");
  if (tokens < 0 || tokens > (1ll << 30)) return fail(MOE_EINVAL, "tokens out of range [0, 2^30]");
  if (n_experts <= 0 || n_experts > 2048) return fail(MOE_EINVAL, "n_experts out of range [1, 2048]");
  if (top_k <= 0 || top_k > 32 || top_k > n_experts) return fail(MOE_EINVAL, "top_k must be <= min(32, n_experts)");
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
    return fail(MOE_EINVAL, "score %d is not MOE_SCORE_SOFTMAX (0) or MOE_SCORE_SIGMOID (1)", r->score);
  if (r->groups <= 0 || r->groups > 64 || n_experts % r->groups)
    return fail(MOE_EINVAL, "groups must divide n_experts, at most 64");
  if (r->top_groups <= 0 || r->top_groups > r->groups) return fail(MOE_EINVAL, "top_groups out of range [1, groups]");
  if ((int64_t)r->top_groups * (n_experts / r->groups) < top_k)
    return fail(MOE_EINVAL, "top_groups hold fewer than top_k experts");
  if (r->group_best != 1 && r->group_best != 2) return fail(MOE_EINVAL, "group_best is 1 or 2");
  if (r->renormalise != 0 && r->renormalise != 1) return fail(MOE_EINVAL, "renormalise is 0 or 1");
  if (!(r->scale > 0.f) || r->scale > 3e38f) return fail(MOE_EINVAL, "scale must be positive and finite");
  *q = SelectRule{r->score, r->groups, r->top_groups, r->group_best, r->renormalise, r->scale};
  return MOE_OK;
}

int logits_ok(const float* p, int64_t stride, int32_t n_experts, const char* what) {
  NEED4(p, what);
  if (stride < n_experts || stride > (1ll << 40)) return fail(MOE_EALIGN, "%s: the stride must be at least n_experts values", what);
  return MOE_OK;
}

int swiglu_ok(int32_t act_dtype, int32_t groups, int64_t max_rows, int64_t hidden, const int32_t* counts) {
  int rc = act_ok(act_dtype);
  if (rc) return rc;
  if (groups < 0 || max_rows < 0) return fail(MOE_EINVAL, "groups and max_rows must not be negative");
  if (groups > 4096 || max_rows > (1ll << 30)) return fail(MOE_EINVAL, "groups or max_rows exceed the kernels' range");
  if (hidden <= 0 || hidden % MX_BLOCK || hidden > (1 << 23))
    return fail(MOE_EINVAL, "hidden (%lld) must be a positive multiple of 32, at most 2^23", (long long)hidden);
  if (counts && ((uintptr_t)counts & 3)) return fail(MOE_EALIGN, "counts is not 4-byte aligned");
  return size_ok(groups * max_rows, 2 * hidden);
}

}  // namespace

extern "C" {

int moe_mxb_strides(int64_t cols, int64_t* code_stride_bytes, int64_t* scale_stride_bytes) {
  const int rc = mx_cols(cols, "cols");
  if (rc) return rc;
  if (code_stride_bytes) *code_stride_bytes = cols;
  if (scale_stride_bytes) *scale_stride_bytes = mx_scale_bytes(cols);
  return MOE_OK;
}

int moe_mxb_quantize(int32_t act_dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride_bytes,
                     const moe_mx_rows* out, void* stream) {
  int rc = act_ok(act_dtype);
  if (rc || (rc = mx_cols(cols, "cols")) || (rc = size_ok(rows, cols))) return rc;
  if (rows == 0) return MOE_OK;
  if ((rc = rows_ok(x, x_stride_bytes, cols, act_dtype == MOE_ACT_BF16 ? 2 : 4, 16, "x")) || (rc = mx8_rows_ok(out, cols, "out")))
    return rc;
  LAUNCH("mx8_quantize", launch_mx8_quantize(act_dtype == MOE_ACT_BF16, rows, cols, x, x_stride_bytes, rows8(out),
                                             (hipStream_t)stream), "moe_mxb_quantize");
  return MOE_OK;
}

int moe_mxb_dequantize(int32_t act_dtype, int64_t rows, int64_t cols, const moe_mx_rows* q, void* out,
                       int64_t out_stride_bytes, void* stream) {
  int rc = act_ok(act_dtype);
  if (rc || (rc = mx_cols(cols, "cols")) || (rc = size_ok(rows, cols))) return rc;
  if (rows == 0) return MOE_OK;
  if ((rc = mx8_rows_ok(q, cols, "q")) ||
      (rc = rows_ok(out, out_stride_bytes, cols, act_dtype == MOE_ACT_BF16 ? 2 : 4, 16, "out")))
    return rc;
  LAUNCH("mx8_dequantize", launch_mx8_dequantize(act_dtype == MOE_ACT_BF16, rows, cols, rows8(q), out, out_stride_bytes,
                                                 (hipStream_t)stream), "moe_mxb_dequantize");
  return MOE_OK;
}

int moe_mxb_gemm(int32_t out_dtype, int32_t groups, int64_t max_rows, int64_t n, int64_t k, const moe_mx_rows* a,
                 const int32_t* counts, const moe_mx_rows* b, void* out, int64_t out_stride_bytes, void* stream) {
  int rc = act_ok(out_dtype);
  if (rc) return rc;
  if (groups < 0 || max_rows < 0) return fail(MOE_EINVAL, "groups and max_rows must not be negative");
  if (n <= 0 || n > (1 << 24)) return fail(MOE_EINVAL, "n must be positive, at most 2^24");
  if ((rc = mx_cols(k, "k"))) return rc;
  if (groups > 4096 || max_rows > (1 << 24) || groups * max_rows > (1ll << 30) || groups * n > (1ll << 30) ||
      groups * ceil_div(max_rows, 256) * ceil_div(n, 256) > (1ll << 21))  // a launch has fewer than 2^32 threads
    return fail(MOE_EINVAL, "groups, max_rows or n exceed the kernels' index range");
  if (groups == 0 || max_rows == 0) return MOE_OK;
  if ((rc = mx8_rows_ok(a, k, "a")) || (rc = mx_rows_ok(b, k, "b"))) return rc;
  const int64_t size = out_dtype == MOE_ACT_BF16 ? 2 : 4;
  if ((rc = rows_ok(out, out_stride_bytes, n, size, size, "out"))) return rc;
  if (counts && ((uintptr_t)counts & 3)) return fail(MOE_EALIGN, "counts is not 4-byte aligned");
  const MxGemmArgs q{mx_view(a), mx_view(b), counts, groups, (int)max_rows, (int)n, (int)k, out_stride_bytes, out, size == 2};
  LAUNCH("mx8_gemm", launch_mx8_gemm(q, cu_count(), (hipStream_t)stream), "moe_mxb_gemm");
  return MOE_OK;
}

int moe_rms_norm(int32_t act_dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride_bytes,
                 const void* residual, int64_t residual_stride_bytes, const void* weight, int32_t weight_dtype, float eps,
                 void* sum, int64_t sum_stride_bytes, void* y, int64_t y_stride_bytes, const moe_mx_rows* y8, void* stream) {
  int rc = norm_ok(act_dtype, rows, cols, weight_dtype, eps);
  if (rc) return rc;
  if (!y && !y8) return fail(MOE_EINVAL, "y and y8 are both NULL");
  if (y8 && cols % MX_BLOCK) return fail(MOE_EINVAL, "MX-FP8 rows need cols to be a multiple of 32");
  if (rows == 0) return MOE_OK;
  const bool bf16 = act_dtype == MOE_ACT_BF16;
  const int64_t size = bf16 ? 2 : 4, unit = y8 ? 16 : size;
  if ((rc = rows_ok(x, x_stride_bytes, cols, size, unit, "x")) || (rc = weight_ok(weight, weight_dtype))) return rc;
  if (y8 && (uintptr_t)weight % 16) return fail(MOE_EALIGN, "weight is not 16-byte aligned, as MX-FP8 rows need");
  if (residual && (rc = rows_ok(residual, residual_stride_bytes, cols, size, unit, "residual"))) return rc;
  if (sum && (rc = rows_ok(sum, sum_stride_bytes, cols, size, unit, "sum"))) return rc;
  if (y && (rc = rows_ok(y, y_stride_bytes, cols, size, unit, "y"))) return rc;
  if (y8 && (rc = mx8_rows_ok(y8, cols, "y8"))) return rc;
  const NormArgs a{rows, cols, x, residual, weight, x_stride_bytes, residual_stride_bytes, sum_stride_bytes, y_stride_bytes,
                   sum, y, y8 ? rows8(y8) : Rows8{}, eps, bf16, weight_dtype == MOE_ACT_F32};
  LAUNCH("rms_norm", launch_rms_norm(a, (hipStream_t)stream), "moe_rms_norm");
  return MOE_OK;
}

int moe_rms_norm_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
  const int rc = norm_ok(MOE_ACT_BF16, rows, cols, MOE_ACT_BF16, 0.f);
  if (rc) return rc;
  if (!bytes) return fail(MOE_EINVAL, "bytes is NULL");
  *bytes = (size_t)norm_parts(rows, cols) * cols * sizeof(float);
  return MOE_OK;
}

int moe_rms_norm_backward(int32_t act_dtype, int64_t rows, int64_t cols, const void* dy, int64_t dy_stride_bytes,
                          const void* sum, int64_t sum_stride_bytes, const void* weight, int32_t weight_dtype, float eps,
                          const void* dsum, int64_t dsum_stride_bytes, void* dx, int64_t dx_stride_bytes, float* dweight,
                          void* ws, void* stream) {
  int rc = norm_ok(act_dtype, rows, cols, weight_dtype, eps);
  if (rc) return rc;
  NEED4(dweight, "dweight");
  const bool bf16 = act_dtype == MOE_ACT_BF16;
  const int64_t size = bf16 ? 2 : 4;
  if (rows > 0) {
    if ((rc = rows_ok(dy, dy_stride_bytes, cols, size, size, "dy")) || (rc = rows_ok(sum, sum_stride_bytes, cols, size, size, "sum")) ||
        (rc = rows_ok(dx, dx_stride_bytes, cols, size, size, "dx")) || (rc = weight_ok(weight, weight_dtype)))
      return rc;
    if (dsum && (rc = rows_ok(dsum, dsum_stride_bytes, cols, size, size, "dsum"))) return rc;
    NEED(ws, "ws");
  }
  NormBackArgs a{rows, cols, dy, sum, dsum, weight, dy_stride_bytes, sum_stride_bytes, dsum_stride_bytes, dx_stride_bytes,
                 dx, dweight, (float*)ws, 0, eps, bf16, weight_dtype == MOE_ACT_F32};
  if (rows > 0)
    LAUNCH("rms_norm_backward", launch_rms_norm_backward(a, (hipStream_t)stream), "moe_rms_norm_backward");
  LAUNCH("norm_dweight", launch_norm_dweight(a, (hipStream_t)stream), "moe_rms_norm_backward dweight");
  return MOE_OK;
}

int moe_select(const moe_router_rule* rule, int64_t tokens, int32_t n_experts, int32_t top_k, const float* logits,
               int64_t logits_stride, const float* balance, int32_t* topk_idx, float* topk_w, void* stream) {
  SelectRule r;
  int rc = rule_ok(rule, tokens, n_experts, top_k, &r);
  if (rc || tokens == 0) return rc;
  if ((rc = logits_ok(logits, logits_stride, n_experts, "logits"))) return rc;
  if (balance) NEED4(balance, "balance");
  NEED4(topk_idx, "topk_idx");
  NEED4(topk_w, "topk_w");
  LAUNCH("select", launch_select_rule(r, logits, logits_stride, balance, tokens, n_experts, top_k, topk_idx, topk_w,
                                      (hipStream_t)stream), "moe_select");
  return MOE_OK;
}

int moe_select_backward(const moe_router_rule* rule, int64_t tokens, int32_t n_experts, int32_t top_k, const float* dtopk_w,
                        const float* topk_w, const int32_t* topk_idx, const float* logits, int64_t logits_stride,
                        float* dlogits, int64_t dlogits_stride, void* stream) {
  SelectRule r;
  int rc = rule_ok(rule, tokens, n_experts, top_k, &r);
  if (rc || tokens == 0) return rc;
  NEED4(dtopk_w, "dtopk_w");
  NEED4(topk_w, "topk_w");
  NEED4(topk_idx, "topk_idx");
  if ((rc = logits_ok(logits, logits_stride, n_experts, "logits")) || (rc = logits_ok(dlogits, dlogits_stride, n_experts, "dlogits")))
    return rc;
  LAUNCH("select_backward", launch_select_backward(r, dtopk_w, topk_w, topk_idx, logits, logits_stride, tokens, n_experts, top_k,
                                                   dlogits, dlogits_stride, (hipStream_t)stream), "moe_select_backward");
  return MOE_OK;
}

int moe_swiglu_checkpoint(int32_t act_dtype, int32_t groups, int64_t max_rows, int64_t hidden, const void* gate_up,
                          int64_t gate_up_stride_bytes, const int32_t* counts, void* h, int64_t h_stride_bytes,
                          const moe_mx_rows* saved, void* stream) {
  int rc = swiglu_ok(act_dtype, groups, max_rows, hidden, counts);
  if (rc || groups == 0 || max_rows == 0) return rc;
  const int64_t size = act_dtype == MOE_ACT_BF16 ? 2 : 4;
  if ((rc = rows_ok(gate_up, gate_up_stride_bytes, 2 * hidden, size, 16, "gate_up")) ||
      (rc = rows_ok(h, h_stride_bytes, hidden, size, 16, "h")) || (rc = mx8_rows_ok(saved, 2 * hidden, "saved")))
    return rc;
  SwigluArgs a{};
  a.groups = groups; a.max_rows = max_rows; a.hidden = hidden; a.counts = counts;
  a.gate_up = gate_up; a.ldg = gate_up_stride_bytes; a.h = h; a.ldh = h_stride_bytes; a.q = rows8(saved);
  a.bf16 = size == 2;
  LAUNCH("swiglu_checkpoint", launch_swiglu_checkpoint(a, (hipStream_t)stream), "moe_swiglu_checkpoint");
  return MOE_OK;
}

int moe_swiglu_backward(int32_t act_dtype, int32_t groups, int64_t max_rows, int64_t hidden, const void* dh,
                        int64_t dh_stride_bytes, const moe_mx_rows* saved, const int32_t* counts, void* dgate_up,
                        int64_t dgate_up_stride_bytes, void* h, int64_t h_stride_bytes, void* stream) {
  int rc = swiglu_ok(act_dtype, groups, max_rows, hidden, counts);
  if (rc || groups == 0 || max_rows == 0) return rc;
  const int64_t size = act_dtype == MOE_ACT_BF16 ? 2 : 4;
  if ((rc = rows_ok(dh, dh_stride_bytes, hidden, size, 16, "dh")) || (rc = mx8_rows_ok(saved, 2 * hidden, "saved")) ||
      (rc = rows_ok(dgate_up, dgate_up_stride_bytes, 2 * hidden, size, 16, "dgate_up")))
    return rc;
  if (h && (rc = rows_ok(h, h_stride_bytes, hidden, size, 16, "h"))) return rc;
  SwigluArgs a{};
  a.groups = groups; a.max_rows = max_rows; a.hidden = hidden; a.counts = counts;
  a.dh = dh; a.ldd = dh_stride_bytes; a.q = rows8(saved); a.dgate_up = dgate_up; a.ldg = dgate_up_stride_bytes;
  a.h = h; a.ldh = h_stride_bytes;
  a.bf16 = size == 2;
  LAUNCH("swiglu_backward", launch_swiglu_backward(a, (hipStream_t)stream), "moe_swiglu_backward");
  return MOE_OK;
}

}  // extern "C"
