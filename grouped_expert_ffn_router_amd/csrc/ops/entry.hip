// C ABI of the MX-FP4 operators and of the few-token layer.
//
// One translation unit with api.hip, whose argument checks, dims derivation,
// error message and kernel timing these entry points share; their kernels are
// in ops/mx.hip and ops/few.hip.

#include "../api.hip"

#include "few.h"
#include "mx.h"

namespace {

// ------------------------------------------------------------ MX-FP4 arguments

int mx_cols(int64_t cols, const char* what) {
  if (cols <= 0 || cols % MX_BLOCK || cols > (1 << 24))
    return fail(MOE_EINVAL, "%s (%lld) must be a positive multiple of 32, at most 2^24", what, (long long)cols);
  return MOE_OK;
}

int mx_strides_ok(int64_t cols, int64_t code_stride, int64_t scale_stride, const char* what) {
  if (code_stride % 16 || code_stride < cols / 2)
    return fail(MOE_EALIGN, "%s: code_stride_bytes must be a multiple of 16 and >= cols / 2", what);
  if (scale_stride % 16 || scale_stride < mx_scale_bytes(cols))
    return fail(MOE_EALIGN, "%s: scale_stride_bytes must be a multiple of 16 and >= cols / 32 rounded up to 16", what);
  return MOE_OK;
}

int mx_rows_ok(const moe_mx_rows* r, int64_t cols, const char* what) {
  if (!r) return fail(MOE_EINVAL, "%s is NULL", what);
  NEED(r->codes, what);
  NEED(r->scales, what);
  return mx_strides_ok(cols, r->code_stride_bytes, r->scale_stride_bytes, what);
}

MxView mx_view(const moe_mx_rows* r) {
  return {(const uint8_t*)r->codes, (const uint8_t*)r->scales, r->code_stride_bytes, r->scale_stride_bytes};
}

// The arguments moe_mx_quantize and moe_mx_dequantize share.
int mx_convert_ok(int32_t act_dtype, int64_t rows, int64_t cols, const void* act, int64_t act_stride,
                  const void* codes, int64_t code_stride, const void* scales, int64_t scale_stride,
                  const char* act_name) {
  if (act_dtype != MOE_ACT_BF16 && act_dtype != MOE_ACT_F32)
    return fail(MOE_EDTYPE, "act_dtype %d is not MOE_ACT_BF16 (0) or MOE_ACT_F32 (1)", act_dtype);
  if (rows < 0) return fail(MOE_EINVAL, "rows < 0");
  int rc = mx_cols(cols, "cols");
  if (rc) return rc;
  if (rows > (1ll << 40) / cols) return fail(MOE_EINVAL, "rows * cols exceeds 2^40");
  if (rows == 0) return MOE_OK;
  NEED(act, act_name);
  NEED(codes, "codes");
  NEED(scales, "scales");
  if (act_stride % 16 || act_stride < cols * (act_dtype == MOE_ACT_BF16 ? 2 : 4))
    return fail(MOE_EALIGN, "%s: its stride must be a multiple of 16 and hold cols values", act_name);
  return mx_strides_ok(cols, code_stride, scale_stride, "rows");
}

// Scratch of moe_mx_expert_gemm: per live wave, the wave's quantised rows and
// its hidden rows (a recv_cap block per expert, or one ragged bank).
struct MxLayout {
  size_t x, x_scales, h, h_scales, wave, total;
};

int mx_layout(const Q& q, MxLayout* w) {
  if (q.L % MX_BLOCK || q.H % MX_BLOCK)
    return fail(MOE_EINVAL, "MX-FP4 experts need latent and expert_hidden to be multiples of 32");
  if (q.WX * ceil_div(q.rcap, 256) * ceil_div(2 * q.H > q.L ? 2 * q.H : q.L, 256) > (1ll << 21))
    return fail(MOE_EINVAL, "a wave's products exceed 2^21 tiles of 256 x 256, what a launch takes");
  const size_t rows = (size_t)(q.WR > 0 ? q.WR : q.WX * q.rcap);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  w->x = take(rows * (q.L / 2));
  w->x_scales = take(rows * mx_scale_bytes(q.L));
  w->h = take(rows * (q.H / 2));
  w->h_scales = take(rows * mx_scale_bytes(q.H));
  w->wave = off;
  w->total = off * q.LW;
  return MOE_OK;
}

// ------------------------------------------------------------ few tokens

int few_dims(const moe_dims* d, FewDims* f) {
  if (!d) return fail(MOE_EINVAL, "dims is NULL");
  if (d->act_dtype != MOE_ACT_BF16 && d->act_dtype != MOE_ACT_F32)
    return fail(MOE_EDTYPE, "act_dtype %d is not MOE_ACT_BF16 (0) or MOE_ACT_F32 (1)", d->act_dtype);
  if (d->tokens < 0 || d->tokens > MOE_FEW_TOKENS_MAX)
    return fail(MOE_EINVAL, "tokens %d out of range [0, %d]", d->tokens, MOE_FEW_TOKENS_MAX);
  if (d->d_model <= 0 || d->latent <= 0 || d->n_experts <= 0 || d->top_k <= 0 || d->n_ranks <= 0 ||
      d->expert_hidden <= 0 || d->shared_experts < 0 || d->shared_hidden <= 0)
    return fail(MOE_EINVAL, "dims must be positive (tokens and shared_experts may be 0)");
  if (d->n_experts > 2048) return fail(MOE_EINVAL, "n_experts > 2048");
  if (d->n_experts % d->n_ranks) return fail(MOE_EINVAL, "n_experts %% n_ranks != 0");
  if (d->my_rank < 0 || d->my_rank >= d->n_ranks) return fail(MOE_EINVAL, "my_rank out of range");
  if (d->top_k > 32 || d->top_k > d->n_experts) return fail(MOE_EINVAL, "top_k must be <= min(32, n_experts)");
  const int64_t shared = (int64_t)d->shared_experts * d->shared_hidden;
  if (d->d_model > (1 << 24) || d->expert_hidden > (1 << 24) || d->latent + shared >= (1 << 24) ||
      d->shared_hidden > (1 << 24))
    return fail(MOE_EINVAL, "d_model, expert_hidden and latent + shared_experts * shared_hidden must be below 2^24");
  const bool bf16 = d->act_dtype == MOE_ACT_BF16;
  if (bf16 && (d->d_model % 64 || d->latent % 64 || d->expert_hidden % 64 || d->shared_hidden % 64))
    return fail(MOE_EINVAL, "bf16 layers need d_model, latent, expert_hidden, shared_hidden multiples of 64");
  const int X = d->n_experts / d->n_ranks;
  if ((int64_t)d->tokens * d->top_k * ceil_div(d->expert_hidden, 16) > (1ll << 25) ||
      d->shared_experts * ceil_div(d->shared_hidden, 16) > (1ll << 20))
    return fail(MOE_EINVAL, "tokens * top_k * expert_hidden or shared_experts exceed what a launch takes");
  *f = FewDims{d->tokens, d->d_model, d->latent, d->n_experts, d->top_k, d->expert_hidden, d->shared_experts,
               d->shared_hidden, X, d->my_rank * X, bf16, false};
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_mx_strides(int64_t cols, int64_t* code_stride_bytes, int64_t* scale_stride_bytes) {
  const int rc = mx_cols(cols, "cols");
  if (rc) return rc;
  if (code_stride_bytes) *code_stride_bytes = cols / 2;
  if (scale_stride_bytes) *scale_stride_bytes = mx_scale_bytes(cols);
  return MOE_OK;
}

int moe_mx_quantize(int32_t act_dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride_bytes, void* codes,
                    int64_t code_stride_bytes, void* scales, int64_t scale_stride_bytes, void* stream) {
  const int rc = mx_convert_ok(act_dtype, rows, cols, x, x_stride_bytes, codes, code_stride_bytes, scales,
                               scale_stride_bytes, "x");
  if (rc || rows == 0) return rc;
  LAUNCH("mx_quantize", launch_mx_quantize(act_dtype == MOE_ACT_BF16, rows, cols, x, x_stride_bytes, (uint8_t*)codes,
                                           code_stride_bytes, (uint8_t*)scales, scale_stride_bytes,
                                           (hipStream_t)stream), "moe_mx_quantize");
  return MOE_OK;
}

int moe_mx_dequantize(int32_t act_dtype, int64_t rows, int64_t cols, const void* codes, int64_t code_stride_bytes,
                      const void* scales, int64_t scale_stride_bytes, void* out, int64_t out_stride_bytes,
                      void* stream) {
  const int rc = mx_convert_ok(act_dtype, rows, cols, out, out_stride_bytes, codes, code_stride_bytes, scales,
                               scale_stride_bytes, "out");
  if (rc || rows == 0) return rc;
  LAUNCH("mx_dequantize", launch_mx_dequantize(act_dtype == MOE_ACT_BF16, rows, cols, (const uint8_t*)codes,
                                               code_stride_bytes, (const uint8_t*)scales, scale_stride_bytes, out,
                                               out_stride_bytes, (hipStream_t)stream), "moe_mx_dequantize");
  return MOE_OK;
}

int moe_mx_gemm(int32_t out_dtype, int32_t groups, int64_t max_rows, int64_t n, int64_t k, const moe_mx_rows* a,
                const int32_t* counts, const moe_mx_rows* b, void* out, int64_t out_stride_bytes, void* stream) {
  if (out_dtype != MOE_ACT_BF16 && out_dtype != MOE_ACT_F32)
    return fail(MOE_EDTYPE, "out_dtype %d is not MOE_ACT_BF16 (0) or MOE_ACT_F32 (1)", out_dtype);
  if (groups < 0 || max_rows < 0) return fail(MOE_EINVAL, "groups and max_rows must not be negative");
  if (n <= 0 || n > (1 << 24)) return fail(MOE_EINVAL, "n must be positive, at most 2^24");
  int rc = mx_cols(k, "k");
  if (rc) return rc;
  if (groups > 4096 || max_rows > (1 << 24) || groups * max_rows > (1ll << 30) || groups * n > (1ll << 30) ||
      groups * ceil_div(max_rows, 256) * ceil_div(n, 256) > (1ll << 21))  // a launch has fewer than 2^32 threads
    return fail(MOE_EINVAL, "groups, max_rows or n exceed the kernels' index range");
  if (groups == 0 || max_rows == 0) return MOE_OK;
  if ((rc = mx_rows_ok(a, k, "a")) || (rc = mx_rows_ok(b, k, "b"))) return rc;
  const int64_t size = out_dtype == MOE_ACT_BF16 ? 2 : 4;
  if (!out) return fail(MOE_EINVAL, "out is NULL");
  if ((uintptr_t)out % size || out_stride_bytes % size || out_stride_bytes < n * size)
    return fail(MOE_EALIGN, "out: address and stride must be multiples of the value size, the stride at least n values");
  if (counts && ((uintptr_t)counts & 3)) return fail(MOE_EALIGN, "counts is not 4-byte aligned");
  const MxGemmArgs q{mx_view(a), mx_view(b), counts, groups, (int)max_rows, (int)n, (int)k, out_stride_bytes, out,
                     out_dtype == MOE_ACT_BF16};
  LAUNCH("mx_gemm", launch_mx_gemm(q, cu_count(), (hipStream_t)stream), "moe_mx_gemm");
  return MOE_OK;
}

int moe_mx_workspace_size(const moe_dims* dims, size_t* bytes) {
  Q q;
  int rc = derive(dims, &q);
  if (rc) return rc;
  MxLayout w;
  if ((rc = mx_layout(q, &w))) return rc;
  if (!bytes) return fail(MOE_EINVAL, "bytes is NULL");
  *bytes = w.total;
  return MOE_OK;
}

int moe_mx_expert_gemm(const moe_dims* dims, int32_t wave, const void* wave_buf, const void* recv_pools,
                       int64_t src_stride_bytes, const int32_t* row_src, const int32_t* wave_count,
                       const moe_mx_rows* w13, const moe_mx_rows* w2, void* ret_pools, int64_t ret_src_stride_bytes,
                       void* ws, void* ws_mx, void* stream) {
  Q q;
  int rc = derive(dims, &q);
  if (rc) return rc;
  MxLayout m;
  if ((rc = mx_layout(q, &m))) return rc;
  NEED4_IF(q.rcap > 0, row_src, "row_src"); NEED4(wave_count, "wave_count");
  if ((rc = mx_rows_ok(w13, q.L, "w13")) || (rc = mx_rows_ok(w2, q.H, "w2"))) return rc;
  NEED_IF(q.scap > 0, ret_pools, "ret_pools"); NEED(ws, "ws"); NEED_IF(m.total > 0, ws_mx, "ws_mx");
  if (wave < 0 || wave >= q.W) return fail(MOE_EINVAL, "wave %d out of range [0, %d)", wave, (int)q.W);
  if (ret_src_stride_bytes % 16 || ret_src_stride_bytes < q.scap * q.row_bytes)
    return fail(MOE_EALIGN, "ret_src_stride_bytes must be a multiple of 16 and >= send_cap * L * sizeof(act)");
  if (wave_buf) {
    if (!aligned16(wave_buf)) return fail(MOE_EALIGN, "wave_buf is not 16-byte aligned");
  } else {
    NEED_IF(q.scap > 0, recv_pools, "recv_pools (wave_buf is NULL)");
    if (src_stride_bytes % 16 || src_stride_bytes < q.scap * q.prow)
      return fail(MOE_EALIGN, "src_stride_bytes must be a multiple of 16 and >= send_cap * pool_stride_bytes");
  }
  const WsLayout w = layout(q);
  hipStream_t st = (hipStream_t)stream;
  char* base = (char*)ws_mx + (size_t)(wave % q.LW) * m.wave;
  const MxView x{(uint8_t*)base + m.x, (uint8_t*)base + m.x_scales, q.L / 2, mx_scale_bytes(q.L)};
  const MxView h{(uint8_t*)base + m.h, (uint8_t*)base + m.h_scales, q.H / 2, mx_scale_bytes(q.H)};
  MxView v13 = mx_view(w13), v2 = mx_view(w2);
  const int64_t x0 = (int64_t)wave * q.WX;  // the wave's first local expert
  v13.codes += x0 * 2 * q.H * v13.ldc; v13.scales += x0 * 2 * q.H * v13.lds;
  v2.codes += x0 * q.L * v2.ldc; v2.scales += x0 * q.L * v2.lds;
  const MxGather gather{(const char*)wave_buf, (const char*)recv_pools, src_stride_bytes, q.prow, (int)q.scap, row_src,
                        wave_count, (int)q.WX, (int)q.rcap, q.WR};
  const MxExpertArgs e{x, h, v13, v2, wave_count, (int)q.WX, (int)q.rcap, (int)q.L, (int)q.H, q.WR, q.bf16,
                       (char*)ret_pools, ret_src_stride_bytes, q.row_bytes, (int)q.scap, row_src};
  LAUNCH("mx_gather", launch_mx_gather(q.bf16, gather, q.L, (uint8_t*)base + m.x, (uint8_t*)base + m.x_scales, st),
         "moe_mx_expert_gemm gather");
  LAUNCH("mx_gate_up", launch_mx_gate_up(e, cu_count(), st), "moe_mx_expert_gemm gate/up");
  LAUNCH("mx_down", launch_mx_down(e, cu_count(), st), "moe_mx_expert_gemm down");
  LAUNCH("zero_dropped", launch_zero_dropped(at<int32_t>(ws, w.r_j), at<int32_t>(ws, w.r_rank), (int)(q.R * q.scap), (int)q.scap,
                              (int)q.rcap, wave * (int)q.WX, (int)q.WX, ret_pools, ret_src_stride_bytes, q.row_bytes,
                              st), "moe_mx_expert_gemm zero rows");
  return MOE_OK;
}

int moe_few_workspace_size(const moe_dims* dims, size_t* bytes) {
  FewDims f;
  const int rc = few_dims(dims, &f);
  if (rc) return rc;
  if (!bytes) return fail(MOE_EINVAL, "bytes is NULL");
  // enough for every smaller batch and for experts of either form (the shares of the down product depend on both)
  size_t most = 0;
  for (; f.T > 0; --f.T)
    for (int mx = 0; mx <= (f.bf16 ? 1 : 0); ++mx) {
      f.mx = mx != 0;
      const size_t n = few_layout(f).total;
      if (n > most) most = n;
    }
  *bytes = most;
  return MOE_OK;
}

int moe_few_tokens(const moe_dims* dims, const void* x, const void* w_router, const void* w_down, const float* bias,
                   int32_t bias_row_tokens, const void* w13, const void* w13_scales, const void* w2,
                   const void* w2_scales, const void* w_up, const void* ws13, const void* ws2, int32_t* topk_idx,
                   float* topk_w, void* out, void* ws, void* stream) {
  FewArgs a{};
  const int rc = few_dims(dims, &a.d);
  if (rc) return rc;
  if (a.d.T == 0) return MOE_OK;
  NEED(x, "x"); NEED(w_router, "w_router"); NEED(w_down, "w_down"); NEED(w13, "w13"); NEED(w2, "w2");
  NEED(w_up, "w_up"); NEED(out, "out"); NEED(ws, "ws");
  NEED4(topk_idx, "topk_idx"); NEED4(topk_w, "topk_w");
  if (bias) NEED4(bias, "bias");
  if (bias_row_tokens < 0) return fail(MOE_EINVAL, "bias_row_tokens < 0");
  if (a.d.S > 0) { NEED(ws13, "ws13"); NEED(ws2, "ws2"); }
  if (!w13_scales != !w2_scales) return fail(MOE_EINVAL, "w13_scales and w2_scales go together");
  if (w13_scales) {
    if (!a.d.bf16) return fail(MOE_EDTYPE, "MX-FP4 experts need a bf16 layer");
    NEED(w13_scales, "w13_scales"); NEED(w2_scales, "w2_scales");
    a.d.mx = true;
  }
  const FewWs w = few_layout(a.d);
  a.x = x; a.w_router = w_router; a.w_down = w_down; a.w13 = w13; a.w2 = w2; a.w_up = w_up; a.ws13 = ws13; a.ws2 = ws2;
  a.w13_scales = (const uint8_t*)w13_scales; a.w2_scales = (const uint8_t*)w2_scales;
  a.bias = bias; a.bias_row_tokens = bias_row_tokens;
  a.topk_idx = topk_idx; a.topk_w = topk_w; a.out = out;
  a.logits = at<float>(ws, w.logits);
  a.mask = at<uint64_t>(ws, w.mask);
  a.active = at<int32_t>(ws, w.active);
  a.first = at<int32_t>(ws, w.first);
  a.count = at<int32_t>(ws, w.count);
  a.gate = at<float>(ws, w.gate);
  a.z = {at<char>(ws, w.z), at<char>(ws, w.z_lo)};
  a.hs = {at<char>(ws, w.hs), at<char>(ws, w.hs_lo)};
  a.h = {at<char>(ws, w.h), at<char>(ws, w.h_lo)};
  a.c = {at<char>(ws, w.c), at<char>(ws, w.c_lo)};
  a.part = at<float>(ws, w.part);
  a.arrived = at<int32_t>(ws, w.arrived);
  a.parts = w.parts; a.tiles = w.tiles; a.down_rt = w.down_rt;
  hipStream_t st = (hipStream_t)stream;
  LAUNCH("few_project", launch_few_project(a, st), "moe_few_tokens project");
  LAUNCH("few_select_shared", launch_few_select(a, st), "moe_few_tokens select");
  LAUNCH("few_gate_up", launch_few_gate_up(a, st), "moe_few_tokens gate/up");
  LAUNCH("few_down", launch_few_down(a, st), "moe_few_tokens down");
  LAUNCH("few_up", launch_few_up(a, st), "moe_few_tokens up");
  return MOE_OK;
}

}  // extern "C"
