// MX-FP4 rows (include/moe.h): device helpers and the host launchers of
// ops/mx.hip.
#pragma once

#include "../gemm.h"
#include "../moe_common.h"
#include "../moe_internal.h"

namespace moe {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int MX_BLOCK = 32;  // values that share a scale: 16 bytes of codes

// Bytes of a row's scales as they are stored (rows of scales are read 16 bytes at a time).
__host__ __device__ __forceinline__ int64_t mx_scale_bytes(int64_t cols) { return (cols / MX_BLOCK + 15) / 16 * 16; }

// Exponent of a block's scale from the bits of its largest magnitude:
// floor(log2 m) - 2, at least -127 (a zero or subnormal m has exponent field
// 0 and lands below).  Field 255 (an infinity or a NaN) is the caller's case.
__device__ __forceinline__ int mx_exponent(uint32_t amax_bits) { return max((int)(amax_bits >> 23) - 129, -127); }

// 2^-e for e in [-127, 126]: exact, and so is every product with it that does
// not underflow below the grid's smallest border.
__device__ __forceinline__ float mx_inverse_scale(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// 2^(b - 127) for a scale byte; b = 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return __uint_as_float(b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23);
}

// Four values, already multiplied by 2^-e, to four codes (16 bits), the first
// in the low bits.  v_cvt_scalef32_pk_fp4_f32 rounds to nearest, ties to the
// even code, and saturates at 6; its own scale stays 1 (a subnormal or
// out-of-range scale would not survive it).
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, a, b, 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c, d, 1.0f, 1);
  return r & 0xffffu;
}

struct MxView {  // the rows of moe_mx_rows, for kernels
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ldc, lds;
};

hipError_t launch_mx_quantize(bool bf16, int64_t rows, int64_t cols, const void* x, int64_t ldx, uint8_t* codes,
                              int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t st);
hipError_t launch_mx_dequantize(bool bf16, int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc,
                                const uint8_t* scales, int64_t lds, void* out, int64_t ldo, hipStream_t st);

struct MxGemmArgs {
  MxView a, b;
  const int32_t* counts;  // rows per group, or NULL: max_rows
  int groups, max_rows, n, k;
  int64_t ldo;  // bytes
  void* out;
  bool bf16;
};
hipError_t launch_mx_gemm(const MxGemmArgs& g, int cus, hipStream_t st);

// Rows of one wave, gathered and quantised.  Row m of expert j goes to bank
// row j * rcap + m, or (ragged_rows > 0) right behind the rows of the experts
// before it, as far as the bank reaches.
struct MxGather {
  const char* wave_buf;  // [nj][rcap][L], or NULL: rows straight from the pools
  const char* pools;
  int64_t src_stride, row_stride;  // of the pools
  int cap;
  const int32_t* row_src;  // [nj][rcap]
  const int32_t* counts;   // [nj]
  int nj, rcap;
  int64_t ragged_rows;
};
hipError_t launch_mx_gather(bool bf16, const MxGather& g, int64_t cols, uint8_t* codes, uint8_t* scales,
                            hipStream_t st);

struct MxExpertArgs {
  MxView x, h;  // quantised rows of the wave and its hidden rows (banks of the layout above)
  MxView w13, w2;  // first row: the wave's first expert
  const int32_t* counts;
  int nj, rcap, L, H;
  int64_t ragged_rows;
  bool bf16;
  char* ret;
  int64_t ret_src_stride, row_bytes;
  int cap;
  const int32_t* row_src;
};
hipError_t launch_mx_gate_up(const MxExpertArgs& g, int cus, hipStream_t st);
hipError_t launch_mx_down(const MxExpertArgs& g, int cus, hipStream_t st);

}  // namespace moe
