// The operators around the experts' products (include/moe.h: MX-FP8 rows, norm,
// choice of experts, SwiGLU with an 8-bit checkpoint): device helpers and the
// host launchers of the kernels in this directory.
#pragma once

#include "../ops/mx.h"

namespace moe {

// ------------------------------------------------------------ MX-FP8 blocks

// Exponent of a block's scale from the bits of its largest magnitude m: the
// smallest e with m 2^-e <= 448, so one more than floor(log2 m) - 8 where the
// fraction of m is above 1.75.  Field 255 (an infinity or a NaN) is the caller's case.
__device__ __forceinline__ int mx8_exponent(uint32_t amax_bits) {
  return max((int)((amax_bits + 0x1fffffu) >> 23) - 135, -127);
}

// Four values, already multiplied by 2^-e (at most 448 in magnitude), to four
// E4M3 codes, the first in the low byte.  v_cvt_pk_fp8_f32 rounds to nearest,
// ties to the even code.
__device__ __forceinline__ uint32_t mx8_codes4(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

// Four E4M3 codes times the scale `unit`.
__device__ __forceinline__ void mx8_values4(uint32_t codes, float unit, float* v) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, true);
  v[0] = lo[0] * unit; v[1] = lo[1] * unit; v[2] = hi[0] * unit; v[3] = hi[1] * unit;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}

// Maximum over groups of G = 4 or 8 neighbouring lanes: quad permutations
// [1,0,3,2] and [2,3,0,1], then a mirror of 8 lanes, which swaps the two quads.
template <int G>
__device__ __forceinline__ uint32_t lane_group_max(uint32_t v) {
  v = max(v, dpp_move<0xB1>(v));
  v = max(v, dpp_move<0x4E>(v));
  if (G == 8) v = max(v, dpp_move<0x141>(v));
  return v;
}

// V values of a lane (a block is 32 / V neighbouring lanes, all active) to
// codes (V bytes, in c) and the block's scale byte, which is returned.
template <int V>
__device__ __forceinline__ int mx8_block(const float (&x)[V], uint32_t (&c)[V / 4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  m = lane_group_max<MX_BLOCK / V>(m);
  const bool nan = (m >> 23) == 255;
  const int e = nan ? 0 : mx8_exponent(m);
  const float inv = mx_inverse_scale(e);
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    c[i] = nan ? 0u : mx8_codes4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  return nan ? 255 : e + 127;
}

// The scale byte of block b of a row, by the block's first lane; the row's
// last block clears the padding up to a multiple of 16.
__device__ __forceinline__ void mx8_store_scale(uint8_t* row, int b, int blocks, int byte) {
  row[b] = (uint8_t)byte;
  if (b == blocks - 1)
    for (int p = blocks; p & 15; ++p) row[p] = 0;
}

// Values past the caches (STREAM): a call that touches more than the 256 MB
// Infinity Cache reads and writes them with nontemporal accesses, so that what
// it writes does not push out what it has yet to read.  Ordinary and nontemporal:
// norm of 8192 x 6144 with both outputs 85 and 75 us, backward of 65,536 x 6144 with
// a gradient beside the norm 632 and 590, SwiGLU step of two experts of 10,050 rows
// x 2048 135 and 119.  Smaller ones leave what they wrote to the next kernel: norm
// of 2048 x 6144 and the quantisation after it 26.1 and 28.7.
constexpr int64_t STREAM_BYTES = 1ll << 28;

template <bool STREAM, class V>
__device__ __forceinline__ V load_as(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load((const V*)p);
  else return *(const V*)p;
}
template <bool STREAM, class V>
__device__ __forceinline__ void store_as(void* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, (V*)p);
  else *(V*)p = v;
}

// 16 bytes at an address that is a multiple of 2.  The card moves them as one
// access all the same: a copy of 1 GB reads and writes 4.5 TB/s with either side
// 2 bytes off, as it does aligned, and 2.9 with 2 bytes a lane.
typedef int i32x1_any __attribute__((aligned(2)));
typedef int i32x2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// (Codes, 4 or 8 bytes a lane, are faster with ordinary accesses in any case.)
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&c)[N]) {
  if constexpr (N == 1) *(uint32_t*)p = c[0];
  else *(uint2*)p = make_uint2(c[0], c[1]);
}
template <int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&c)[N]) {
  if constexpr (N == 1) {
    c[0] = *(const uint32_t*)p;
  } else {
    const uint2 d = *(const uint2*)p;
    c[0] = d.x;
    c[1] = d.y;
  }
}

// ------------------------------------------------------------ values of a row
//
// V consecutive values: 16 bytes (8 bf16, 4 fp32), or one at a time.  IV: how
// the 16 bytes are aligned (i32x4, i32x4_any).

template <class T, int V>
struct Piece {
  uint32_t w[4];
};
template <class T>
struct Piece<T, 1> {
  T v;
};

template <class T, int V, bool STREAM, class IV = i32x4>
__device__ __forceinline__ Piece<T, V> piece_load(const void* p) {
  Piece<T, V> r;
  if constexpr (V == 1) {
    r.v = *(const T*)p;
  } else {
    const IV d = load_as<STREAM, IV>(p);
    r.w[0] = d[0]; r.w[1] = d[1]; r.w[2] = d[2]; r.w[3] = d[3];
  }
  return r;
}

template <class T, int V>
__device__ __forceinline__ Piece<T, V> piece_zero() {
  Piece<T, V> r;
  if constexpr (V == 1) r.v = (T)0;
  else
    for (int i = 0; i < 4; ++i) r.w[i] = 0;
  return r;
}

template <class T, int V>
__device__ __forceinline__ void piece_values(const Piece<T, V>& r, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = Act<T>::load(r.v);
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i]);
  }
}

// Without its first `n` values, zeros behind the others.
template <class T, int V>
__device__ __forceinline__ void piece_drop(Piece<T, V>& r, int n) {
  if constexpr (V > 1) {
    const int halves = n * (int)sizeof(T) / 2;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t stay = r.w[i], moved = (r.w[i] >> 16) | (i < 3 ? r.w[i + 1] << 16 : 0u);
        r.w[i] = halves & 1 ? moved : stay;
      }
    }
#pragma unroll
    for (int by = 1; by <= 2; ++by)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t stay = r.w[i], moved = i + by < 4 ? r.w[i + by] : 0u;
        r.w[i] = halves & (2 * by) ? moved : stay;
      }
  }
}

template <class T, int V, bool STREAM, class IV = i32x4>
__device__ __forceinline__ void piece_store(void* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *(T*)p = Act<T>::store(v[0]);
  } else if constexpr (sizeof(T) == 2) {
    store_as<STREAM>(p, IV{(int)f32x2_to_bf16x2(v[0], v[1]), (int)f32x2_to_bf16x2(v[2], v[3]),
                           (int)f32x2_to_bf16x2(v[4], v[5]), (int)f32x2_to_bf16x2(v[6], v[7])});
  } else {
    store_as<STREAM>(p, IV{__float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3])});
  }
}

// The first n values, n < V, to any aligned place of a value.
template <class T, int V>
__device__ __forceinline__ void piece_store_first(T* p, const float (&v)[V], int n) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_bf16x2(v[2 * i], v[2 * i + 1]);
    if (n & 4) {
      *(i32x2_any*)p = i32x2_any{(int)w[0], (int)w[1]};
      w[0] = w[2];
      w[1] = w[3];
      p += 4;
    }
    if (n & 2) {
      *(i32x1_any*)p = (int)w[0];
      w[0] = w[1];
      p += 2;
    }
    if (n & 1) *(uint16_t*)p = (uint16_t)w[0];
  } else {
#pragma unroll
    for (int i = 0; i < V - 1; ++i)
      if (i < n) p[i] = v[i];
  }
}

// V values of a vector that is fp32 or bf16 (a uniform choice).
template <int V>
__device__ __forceinline__ void weight_values(const void* w, bool f32, int64_t i, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = f32 ? ((const float*)w)[i] : bf16_to_f32(((const bf16_t*)w)[i]);
  } else if (f32) {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const i32x4_any d = *(const i32x4_any*)((const float*)w + i + q);
      v[q] = __int_as_float(d[0]); v[q + 1] = __int_as_float(d[1]); v[q + 2] = __int_as_float(d[2]); v[q + 3] = __int_as_float(d[3]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < V; q += 4) {
      const i32x2_any d = *(const i32x2_any*)((const bf16_t*)w + i + q);
      const uint32_t x = (uint32_t)d[0], y = (uint32_t)d[1];
      v[q] = __uint_as_float(x << 16); v[q + 1] = __uint_as_float(x & 0xffff0000u);
      v[q + 2] = __uint_as_float(y << 16); v[q + 3] = __uint_as_float(y & 0xffff0000u);
    }
  }
}

// ------------------------------------------------------------ launchers

struct Rows8 {  // MX-FP8 rows to write or read; codes NULL: none
  uint8_t* codes;
  uint8_t* scales;
  int64_t ldc, lds;
};

hipError_t launch_mx8_quantize(bool bf16, int64_t rows, int64_t cols, const void* x, int64_t ldx, const Rows8& q,
                               hipStream_t st);
hipError_t launch_mx8_dequantize(bool bf16, int64_t rows, int64_t cols, const Rows8& q, void* out, int64_t ldo,
                                 hipStream_t st);

struct NormArgs {
  int64_t rows, cols;
  const void *x, *residual, *weight;  // residual may be NULL
  int64_t ldx, ldr, lds, ldy;         // bytes
  void *stream, *y;                   // outputs, either may be NULL
  Rows8 q;
  float eps;
  bool bf16, weight_f32;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st);

struct NormBackArgs {
  int64_t rows, cols;
  const void *dy, *s, *dstream, *weight;  // dstream may be NULL
  int64_t lddy, lds, ldds, lddx;          // bytes
  void* dx;
  float* dweight;
  float* part;  // [parts][cols]
  int64_t parts;  // those written
  float eps;
  bool bf16, weight_f32;
};
// Rows of partial sums of the weight's gradient that a call keeps, at most.
int64_t norm_parts(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_backward(NormBackArgs& a, hipStream_t st);  // sets a.parts
hipError_t launch_norm_dweight(const NormBackArgs& a, hipStream_t st);

struct SelectRule {
  int score, groups, top_groups, group_best, renorm;
  float scale;
};
hipError_t launch_select_rule(const SelectRule& r, const float* logits, int64_t ld, const float* balance, int64_t T, int E,
                              int k, int32_t* idx, float* w, hipStream_t st);
hipError_t launch_select_backward(const SelectRule& r, const float* dw, const float* w, const int32_t* idx,
                                  const float* logits, int64_t ld, int64_t T, int E, int k, float* dlogits, int64_t ldd,
                                  hipStream_t st);

struct SwigluArgs {
  int groups;
  int64_t max_rows, hidden;
  const int32_t* counts;  // [groups], or NULL
  const void* gate_up;    // forward
  const void* dh;         // backward
  int64_t ldg, ldh, ldd;  // bytes: gate_up / dgate_up rows, h rows, dh rows
  void* h;                // forward: output; backward: output or NULL
  void* dgate_up;
  Rows8 q;
  bool bf16;
};
hipError_t launch_swiglu_checkpoint(const SwigluArgs& a, hipStream_t st);
hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t st);

hipError_t launch_mx8_gemm(const MxGemmArgs& g, int cus, hipStream_t st);

}  // namespace moe
