/* The entry points around the experts' products (MX-FP8 rows, norm, choice of
 * experts, SwiGLU) from plain C: sizes on the host, and refusals before any
 * HIP call.  Every call that could launch gets a NULL pointer or a size that is
 * refused, so nothing here needs a GPU.  Prints "ok" and exits 0 on success;
 * the first failure is printed. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe.h"

static int fail(const char* what) {
  printf("FAIL: %s (last error: %s)\n", what, moe_last_error());
  return 1;
}

static uint64_t lcg = 0x853c49e6748fea9bull;
static uint64_t next_bits(void) {
  lcg = lcg * 6364136223846793005ull + 1442695040888963407ull;
  return lcg >> 20;
}

/* extremes, sizes that fit and any other value */
static int64_t any64(void) {
  static const int64_t special[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 2, 8, 16, 31, 32, 64, 384, 1024, 4096, 16384, 16385,
                                    1 << 24, (1 << 24) + 32, 1ll << 30, 1ll << 31, 1ll << 40, 1ll << 62, INT64_MAX - 1, INT64_MAX};
  const int n = (int)(sizeof(special) / sizeof(special[0]));
  const uint64_t r = next_bits();
  return r % 3 ? special[(r >> 8) % (uint64_t)n] : (int64_t)((r >> 8) % 100000) - 50;
}
static int32_t any32(void) { return (int32_t)any64(); }

static int refused(int rc) { return rc == MOE_EINVAL || rc == MOE_EALIGN || rc == MOE_EDTYPE; }

int main(void) {
  char buf[4096 + 16];
  char* at = buf + (16 - (uintptr_t)buf % 16) % 16; /* 16-byte aligned, never read */
  int64_t c = 0, s = 0;
  size_t ws = 0;
  const moe_mx_rows ok = {at, at, 512, 16}, odd = {at + 8, at, 512, 16}, tight = {at, at, 480, 16}, scales = {at, at, 512, 8};

  if (moe_mxb_strides(2080, &c, &s) != MOE_OK || c != 2080 || s != 80) return fail("moe_mxb_strides of 2080 values");
  if (moe_mxb_strides(32, NULL, NULL) != MOE_OK || moe_mxb_strides(48, &c, &s) != MOE_EINVAL) return fail("moe_mxb_strides");

  /* rows of 512 values */
  if (moe_mxb_quantize(MOE_ACT_BF16, 0, 512, NULL, 0, NULL, NULL) != MOE_OK) return fail("no rows");
  if (moe_mxb_quantize(2, 1, 512, at, 1024, &ok, NULL) != MOE_EDTYPE) return fail("a type accepted");
  if (moe_mxb_quantize(MOE_ACT_BF16, 1, 512, at, 1024, NULL, NULL) != MOE_EINVAL) return fail("NULL rows accepted");
  if (moe_mxb_quantize(MOE_ACT_BF16, 1, 512, at + 2, 1024, &ok, NULL) != MOE_EALIGN) return fail("unaligned x accepted");
  if (moe_mxb_quantize(MOE_ACT_BF16, 2, 512, at, 1008, &ok, NULL) != MOE_EALIGN) return fail("overlapping rows accepted");
  if (moe_mxb_quantize(MOE_ACT_BF16, 1, 512, at, 1024, &odd, NULL) != MOE_EALIGN) return fail("unaligned codes accepted");
  if (moe_mxb_quantize(MOE_ACT_BF16, 1, 512, at, 1024, &tight, NULL) != MOE_EALIGN) return fail("a short code stride accepted");
  if (moe_mxb_dequantize(MOE_ACT_F32, 1, 512, &scales, at, 2048, NULL) != MOE_EALIGN) return fail("a short scale stride accepted");

  /* the product: a is 8-bit rows, b 4-bit ones */
  if (moe_mxb_gemm(MOE_ACT_BF16, 1, 4, 8, 512, &tight, NULL, &ok, at, 16, NULL) != MOE_EALIGN) return fail("4-bit rows as a");
  if (moe_mxb_gemm(MOE_ACT_BF16, 1, 4, 8, 512, &ok, NULL, &ok, at, 14, NULL) != MOE_EALIGN) return fail("a short output stride");
  if (moe_mxb_gemm(MOE_ACT_F32, 1, 4, 8, 512, &ok, NULL, &ok, at + 2, 32, NULL) != MOE_EALIGN) return fail("an unaligned output");
  if (moe_mxb_gemm(MOE_ACT_F32, 1, 4, 8, 512, &ok, (const int32_t*)(at + 1), &ok, at, 32, NULL) != MOE_EALIGN) return fail("counts");
  if (moe_mxb_gemm(MOE_ACT_F32, 0, 4, 8, 512, NULL, NULL, NULL, NULL, 0, NULL) != MOE_OK) return fail("no groups");
  if (moe_mxb_gemm(MOE_ACT_F32, 4097, 4, 8, 512, &ok, NULL, &ok, at, 32, NULL) != MOE_EINVAL) return fail("4097 groups");

  /* norm */
  if (moe_rms_norm_workspace_size(8192, 6144, &ws) != MOE_OK || ws != (size_t)1024 * 6144 * 4) return fail("workspace of 8192 rows");
  if (moe_rms_norm_workspace_size(0, 6144, &ws) != MOE_OK || ws != 0) return fail("workspace of no rows");
  if (moe_rms_norm_workspace_size(1, MOE_NORM_COLS_MAX + 1, &ws) != MOE_EINVAL) return fail("too wide a row");
  if (moe_rms_norm_workspace_size(1, 64, NULL) != MOE_EINVAL) return fail("NULL bytes");
  if (moe_rms_norm(MOE_ACT_BF16, 1, 64, at, 128, NULL, 0, at, MOE_ACT_BF16, 1e-6f, NULL, 0, NULL, 0, NULL, NULL) != MOE_EINVAL)
    return fail("no output accepted");
  if (moe_rms_norm(MOE_ACT_BF16, 1, 40, at, 80, NULL, 0, at, MOE_ACT_BF16, 1e-6f, NULL, 0, NULL, 0, &ok, NULL) != MOE_EINVAL)
    return fail("8-bit rows of 40 values accepted");
  if (moe_rms_norm(MOE_ACT_BF16, 2, 64, at, 136, NULL, 0, at, MOE_ACT_BF16, 1e-6f, NULL, 0, NULL, 0, &ok, NULL) != MOE_EALIGN)
    return fail("8-bit rows of unaligned ones accepted");
  if (moe_rms_norm(MOE_ACT_BF16, 2, 64, at, 128, NULL, 0, at + 2, MOE_ACT_BF16, 1e-6f, NULL, 0, NULL, 0, &ok, NULL) != MOE_EALIGN)
    return fail("8-bit rows with an unaligned weight accepted");
  if (moe_rms_norm(MOE_ACT_F32, 2, 64, at, 258, NULL, 0, at, MOE_ACT_F32, 1e-6f, NULL, 0, at, 256, NULL, NULL) != MOE_EALIGN)
    return fail("a stride that is no multiple of the value accepted");
  if (moe_rms_norm(MOE_ACT_F32, 2, 64, at, 256, NULL, 0, at, 7, 1e-6f, NULL, 0, at, 256, NULL, NULL) != MOE_EDTYPE)
    return fail("a weight type accepted");
  if (moe_rms_norm(MOE_ACT_F32, 2, 64, at, 256, NULL, 0, at, MOE_ACT_F32, -1.f, NULL, 0, at, 256, NULL, NULL) != MOE_EINVAL)
    return fail("a negative eps accepted");
  {
    volatile float zero = 0.f;
    const float nan = zero / zero, inf = 1.f / zero;
    moe_router_rule bad = {MOE_SCORE_SOFTMAX, 1, 1, 2, 1, nan};
    if (moe_rms_norm(MOE_ACT_F32, 2, 64, at, 256, NULL, 0, at, MOE_ACT_F32, nan, NULL, 0, at, 256, NULL, NULL) != MOE_EINVAL ||
        moe_rms_norm(MOE_ACT_F32, 2, 64, at, 256, NULL, 0, at, MOE_ACT_F32, inf, NULL, 0, at, 256, NULL, NULL) != MOE_EINVAL)
      return fail("eps that is no number accepted");
    if (moe_select(&bad, 1, 8, 2, NULL, 8, NULL, NULL, NULL, NULL) != MOE_EINVAL) return fail("a NaN scale accepted");
  }
  if (moe_rms_norm_backward(MOE_ACT_F32, 0, 64, NULL, 0, NULL, 0, NULL, MOE_ACT_F32, 1e-6f, NULL, 0, NULL, 0, NULL, NULL, NULL) !=
      MOE_EINVAL)
    return fail("NULL dweight accepted");

  /* choice of experts */
  {
    const float* l = (const float*)at;
    int32_t* i = (int32_t*)at;
    float* w = (float*)at;
    moe_router_rule r = {MOE_SCORE_SIGMOID, 8, 4, 2, 1, 1.f};
    if (moe_select(NULL, 1, 8, 2, l, 8, NULL, i, w, NULL) != MOE_EINVAL) return fail("NULL rule accepted");
    if (moe_select(&r, 0, 384, 8, NULL, 0, NULL, NULL, NULL, NULL) != MOE_OK) return fail("no tokens");
    if (moe_select(&r, 1, 384, 8, l, 383, NULL, i, w, NULL) != MOE_EALIGN) return fail("a short logits stride accepted");
    if (moe_select(&r, 1, 384, 33, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("33 of 384 accepted");
    if (moe_select(&r, 1, 380, 8, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("groups of 47.5 experts accepted");
    if (moe_select(&r, 1, 8, 5, l, 8, NULL, i, w, NULL) != MOE_EINVAL) return fail("5 out of 4 experts accepted");
    if (moe_select(&r, 1, 384, 8, l, 384, (const float*)(at + 2), i, w, NULL) != MOE_EALIGN) return fail("unaligned balance");
    r.top_groups = 9;
    if (moe_select(&r, 1, 384, 8, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("9 of 8 groups accepted");
    r.top_groups = 4; r.group_best = 3;
    if (moe_select(&r, 1, 384, 8, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("group_best 3 accepted");
    r.group_best = 2; r.scale = 0.f;
    if (moe_select(&r, 1, 384, 8, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("scale 0 accepted");
    r.scale = 1.f; r.score = 2;
    if (moe_select(&r, 1, 384, 8, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("score 2 accepted");
    r.score = 0; r.renormalise = 2;
    if (moe_select(&r, 1, 384, 8, l, 384, NULL, i, w, NULL) != MOE_EINVAL) return fail("renormalise 2 accepted");
  }

  /* SwiGLU */
  if (moe_swiglu_checkpoint(MOE_ACT_BF16, 1, 2, 48, at, 192, NULL, at, 96, &ok, NULL) != MOE_EINVAL) return fail("hidden 48 accepted");
  if (moe_swiglu_checkpoint(MOE_ACT_BF16, 1, 2, 256, at, 1008, NULL, at, 512, &ok, NULL) != MOE_EALIGN) return fail("short gate_up rows");
  if (moe_swiglu_checkpoint(MOE_ACT_BF16, 1, 2, 256, at, 1024, NULL, at, 512, &tight, NULL) != MOE_EALIGN) return fail("short saved rows");
  if (moe_swiglu_backward(MOE_ACT_BF16, 1, 2, 256, at, 512, &ok, NULL, at, 1024, at + 8, 512, NULL) != MOE_EALIGN) return fail("unaligned h");
  if (moe_swiglu_backward(MOE_ACT_BF16, 0, 2, 256, NULL, 0, NULL, NULL, NULL, 0, NULL, 0, NULL) != MOE_OK) return fail("no groups");

  /* sizes, strides and rules at any value, pointers that are refused */
  for (int it = 0; it < 40000; ++it) {
    const int32_t type = (int32_t)(next_bits() % 4) - 1, groups = any32();
    const int64_t rows = any64(), cols = any64();
    const moe_mx_rows q = {it & 1 ? at : NULL, it & 2 ? at : NULL, any64(), any64()};
    int rc = moe_mxb_strides(cols, &c, &s);
    if (rc == MOE_OK ? c != cols || s < cols / 32 || s % 16 : rc != MOE_EINVAL) return fail("fuzz: moe_mxb_strides");
    rc = moe_mxb_quantize(type, rows, cols, NULL, any64(), &q, NULL);
    if (!refused(rc) && !(rc == MOE_OK && rows == 0)) return fail("fuzz: moe_mxb_quantize code");
    rc = moe_mxb_dequantize(type, rows, cols, &q, NULL, any64(), NULL);
    if (!refused(rc) && !(rc == MOE_OK && rows == 0)) return fail("fuzz: moe_mxb_dequantize code");
    rc = moe_mxb_gemm(type, groups, rows, any64(), cols, it & 4 ? &q : NULL, NULL, &q, NULL, any64(), NULL);
    if (!refused(rc) && !(rc == MOE_OK && (rows == 0 || groups == 0))) return fail("fuzz: moe_mxb_gemm code");
    rc = moe_rms_norm_workspace_size(rows, cols, &ws);
    if (rc == MOE_OK ? (rows > 0 && ws < (size_t)cols * 4) || ws > (size_t)4096 * MOE_NORM_COLS_MAX * 4 : !refused(rc))
      return fail("fuzz: moe_rms_norm_workspace_size");
    rc = moe_rms_norm(type, rows, cols, NULL, any64(), at, any64(), at, type, 1e-6f, at, any64(), at, any64(), it & 8 ? &q : NULL, NULL);
    if (!refused(rc) && !(rc == MOE_OK && rows == 0)) return fail("fuzz: moe_rms_norm code");
    rc = moe_rms_norm_backward(type, rows, cols, at, any64(), at, any64(), at, type, 1e-6f, at, any64(), at, any64(), NULL, at, NULL);
    if (!refused(rc)) return fail("fuzz: moe_rms_norm_backward code");
    const moe_router_rule r = {(int32_t)(next_bits() % 4) - 1, any32(), any32(), (int32_t)(next_bits() % 4), (int32_t)(next_bits() % 3),
                               1.f};
    rc = moe_select(&r, rows, any32(), any32(), NULL, any64(), (const float*)at, NULL, NULL, NULL);
    if (!refused(rc) && !(rc == MOE_OK && rows == 0)) return fail("fuzz: moe_select code");
    rc = moe_select_backward(&r, rows, any32(), any32(), NULL, NULL, NULL, NULL, any64(), NULL, any64(), NULL);
    if (!refused(rc) && !(rc == MOE_OK && rows == 0)) return fail("fuzz: moe_select_backward code");
    rc = moe_swiglu_checkpoint(type, groups, rows, cols, NULL, any64(), NULL, at, any64(), &q, NULL);
    if (!refused(rc) && !(rc == MOE_OK && (rows == 0 || groups == 0))) return fail("fuzz: moe_swiglu_checkpoint code");
    rc = moe_swiglu_backward(type, groups, rows, cols, NULL, any64(), &q, NULL, at, any64(), NULL, any64(), NULL);
    if (!refused(rc) && !(rc == MOE_OK && (rows == 0 || groups == 0))) return fail("fuzz: moe_swiglu_backward code");
  }
  printf("ok\n");
  return 0;
}
