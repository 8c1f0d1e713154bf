/* The MX-FP4 and few-token entry points from plain C: sizes on the host, and
 * refusals before any HIP call.  Every call that could launch gets a NULL
 * pointer or a size that is refused, so nothing here needs a GPU.  Prints "ok"
 * and exits 0 on success; the first failure is printed. */
#include <stdio.h>
#include <string.h>

#include <stdint.h>

#include "moe.h"

static int fail(const char* what) {
  printf("FAIL: %s (last error: %s)\n", what, moe_last_error());
  return 1;
}

static uint64_t lcg = 0x2545f4914f6cdd1dull;
static uint64_t next_bits(void) {
  lcg = lcg * 6364136223846793005ull + 1442695040888963407ull;
  return lcg >> 20;
}

/* extremes, sizes that fit and any other value */
static int64_t any64(void) {
  static const int64_t special[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 2, 16, 31, 32, 64, 1024, 4096, 1 << 24,
                                    (1 << 24) + 32, 1ll << 31, 1ll << 40, 1ll << 62, INT64_MAX - 1, INT64_MAX};
  const int n = (int)(sizeof(special) / sizeof(special[0]));
  const uint64_t r = next_bits();
  return r % 3 ? special[(r >> 8) % (uint64_t)n] : (int64_t)((r >> 8) % 100000) - 50;
}

static int refused(int rc) { return rc == MOE_EINVAL || rc == MOE_EALIGN || rc == MOE_EDTYPE; }

int main(void) {
  int64_t c = 0, s = 0;
  if (moe_mx_strides(2080, &c, &s) != MOE_OK || c != 1040 || s != 80) return fail("moe_mx_strides of 2080 values");
  if (moe_mx_strides(32, NULL, NULL) != MOE_OK) return fail("moe_mx_strides without outputs");
  if (moe_mx_strides(48, &c, &s) != MOE_EINVAL || strlen(moe_last_error()) == 0) return fail("a width of 48 accepted");

  /* one rank with all of 48 experts, 512 wide, latent 256, hidden 128 */
  moe_dims d = {7, 512, 256, 48, 4, 1, 1, 128, 2, 128, 0, MOE_ACT_BF16, 1, 1, 1, 1, 0, 0};
  size_t few = 0, few64 = 0, mx = 0;
  if (moe_few_workspace_size(&d, &few) != MOE_OK || few == 0) return fail("moe_few_workspace_size");
  d.tokens = 64;
  if (moe_few_workspace_size(&d, &few64) != MOE_OK || few64 < few) return fail("moe_few_workspace_size, 64 tokens");
  d.tokens = 65;
  if (moe_few_workspace_size(&d, &few) != MOE_EINVAL) return fail("65 tokens accepted");
  d.tokens = 0;
  if (moe_few_workspace_size(&d, &few) != MOE_OK || few != 0) return fail("moe_few_workspace_size, no tokens");
  if (moe_few_workspace_size(&d, NULL) != MOE_EINVAL || moe_few_workspace_size(NULL, &few) != MOE_EINVAL)
    return fail("NULL accepted");
  if (moe_few_tokens(&d, NULL, NULL, NULL, NULL, 0, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL,
                     NULL) != MOE_OK)
    return fail("moe_few_tokens without tokens");

  /* the 4K-context layer of one rank: 2 experts a wave, 12562 rows each, three live waves; codes and scales of the rows
     (3072 values: 1536 + 96 bytes) and of the hidden rows (1536 values: 768 + 48 bytes) */
  moe_dims big = {8192, 6144, 3072, 384, 8, 64, 3, 1536, 2, 1536, 0, MOE_ACT_BF16, 110, 100, 115, 100, 0, 0};
  if (moe_mx_workspace_size(&big, &mx) != MOE_OK) return fail("moe_mx_workspace_size");
  {
    const size_t rows = 2 * 12562, part[4] = {rows * 1536, rows * 96, rows * 768, rows * 48};
    size_t want = 0;
    for (int i = 0; i < 4; ++i) want += (part[i] + 255) / 256 * 256;
    if (mx != 3 * want) return fail("size of the MX-FP4 workspace");
  }

  /* fuzz: fields of both layers at any value; the answer is a documented code, and an accepted layer's workspace holds
     at least what it must (no size has wrapped) */
  {
    static const int32_t special[] = {INT32_MIN, -1, 0, 1, 2, 3, 7, 63, 64, 100, 1000, 4096, 65536,
                                      1 << 24, 1 << 30, INT32_MAX};
    const int nspecial = (int)(sizeof(special) / sizeof(special[0]));
    int accepted_few = 0, accepted_mx = 0;
    d.tokens = 64;
    for (int it = 0; it < 20000; ++it) {
      moe_dims f = it & 1 ? d : big;
      if (!(it & 1) && (it & 2)) f.tokens = 33;
      int32_t* fields = (int32_t*)&f;
      const int nfields = (int)(sizeof(moe_dims) / sizeof(int32_t));
      const int nedit = 1 + (int)(next_bits() % 3);
      for (int e = 0; e < nedit; ++e) {
        const uint64_t r = next_bits();
        fields[r % (uint64_t)nfields] =
            (r >> 8) % 3 ? special[(r >> 12) % (uint64_t)nspecial] : (int32_t)((r >> 12) % 70000) - 3;
      }
      size_t a = 0, b = 0;
      const int rc = moe_few_workspace_size(&f, &a), rc2 = moe_mx_workspace_size(&f, &b);
      if (rc != MOE_OK && !refused(rc)) return fail("fuzz: moe_few_workspace_size code");
      if (rc2 != MOE_OK && !refused(rc2)) return fail("fuzz: moe_mx_workspace_size code");
      if (rc == MOE_OK) {
        const size_t es = 4; /* two bf16 parts, or fp32 */
        const size_t least = (size_t)f.tokens * (4u * (size_t)f.n_experts + es * 2u * (size_t)f.latent +
                                                 es * (size_t)f.top_k * (size_t)f.expert_hidden +
                                                 es * (size_t)f.shared_experts * (size_t)f.shared_hidden);
        if (a < least) return fail("fuzz: few-token workspace wrapped");
        ++accepted_few;
      }
      if (rc2 == MOE_OK) {
        int64_t scap = 0, rcap = 0, prow = 0;
        if (moe_capacity(&f, &scap, &rcap, &prow) != MOE_OK) return fail("fuzz: moe_capacity of accepted dims");
        const size_t rows = f.wave_rows > 0 ? (size_t)f.wave_rows
                                            : (size_t)(f.n_experts / f.n_ranks / f.waves) * (size_t)rcap;
        if (b < rows * (size_t)(f.latent + f.expert_hidden) / 2u) return fail("fuzz: MX-FP4 workspace wrapped");
        ++accepted_mx;
      }
      /* the calls themselves: refused for a NULL pointer, or nothing to do */
      const int rc3 = moe_few_tokens(&f, NULL, NULL, NULL, NULL, (int32_t)any64(), NULL, NULL, NULL, NULL, NULL, NULL,
                                     NULL, NULL, NULL, NULL, NULL, NULL);
      if (!refused(rc3) && !(rc3 == MOE_OK && f.tokens == 0)) return fail("fuzz: moe_few_tokens code");
      const moe_mx_rows r13 = {NULL, NULL, any64(), any64()};
      if (!refused(moe_mx_expert_gemm(&f, (int32_t)any64(), NULL, NULL, any64(), NULL, NULL, &r13, &r13, NULL, any64(),
                                      NULL, NULL, NULL)))
        return fail("fuzz: moe_mx_expert_gemm code");
    }
    if (accepted_few == 0 || accepted_mx == 0) return fail("fuzz: nothing accepted");
  }

  /* fuzz: sizes and strides of the row operators at any value, pointers that are refused */
  {
    char at[64];
    for (int it = 0; it < 20000; ++it) {
      const int32_t type = (int32_t)(next_bits() % 4) - 1, groups = (int32_t)any64();
      const int64_t rows = any64(), cols = any64();
      const int rc = moe_mx_strides(cols, &c, &s);
      if (rc == MOE_OK ? c != cols / 2 || s < cols / 32 || s % 16 : rc != MOE_EINVAL) return fail("fuzz: moe_mx_strides");
      const int q = moe_mx_quantize(type, rows, cols, NULL, any64(), NULL, any64(), NULL, any64(), NULL);
      if (!refused(q) && !(q == MOE_OK && rows == 0)) return fail("fuzz: moe_mx_quantize code");
      const int b = moe_mx_dequantize(type, rows, cols, NULL, any64(), NULL, any64(), NULL, any64(), NULL);
      if (!refused(b) && !(b == MOE_OK && rows == 0)) return fail("fuzz: moe_mx_dequantize code");
      const moe_mx_rows a = {it & 1 ? at : NULL, it & 2 ? at : NULL, any64(), any64()};
      const int g = moe_mx_gemm(type, groups, rows, any64(), cols, it & 4 ? &a : NULL, NULL, &a, NULL, any64(), NULL);
      if (!refused(g) && !(g == MOE_OK && (rows == 0 || groups == 0))) return fail("fuzz: moe_mx_gemm code");
    }
  }
  printf("ok few=%zu mx=%zu\n", few64, mx);
  return 0;
}
