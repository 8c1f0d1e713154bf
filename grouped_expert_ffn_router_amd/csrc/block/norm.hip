// Root-mean-square norm of rows after the residual stream's addition, and its
// backward pass (gfx950).
//
//   s = x + residual,  r = (mean(s^2) + eps)^-1/2,  y = s r w
//   with n = s r, g = dy w:  dx = r (g - n mean(g n)) + dstream,  dw = sum over rows of dy n
//
// Bound by bytes: 8192 x 6144 bf16 with a residual, the sum, bf16 and 8-bit rows
// out, 72-76 us (6.0-6.3 TB/s); backward of 65,536 x 6144 with a gradient beside
// the norm 569-580 us (5.6-5.7 TB/s) and the sum of its 1024 partial rows 10; one
// row 3 us, a launch and a trip to memory.

#include "block.h"

#include <algorithm>

namespace moe {

namespace {

// A row is NC pieces of V values for each of TPR threads (piece tid + TPR i of
// thread tid), kept in registers between the row's sum and its use: every
// value is read once and written once.
template <int TPR_, int NC_>
struct RowCfg {
  static constexpr int TPR = TPR_, NC = NC_, NT = TPR > 256 ? TPR : 256, RPB = NT / TPR;
  static_assert((TPR == 16 || TPR % 64 == 0) && NT % TPR == 0, "16 lanes or whole waves to a row, whole rows to a workgroup");
};

// Sums over a wave's lanes, or each 16 of them, in all of them, in a fixed order:
// DPP steps inside the rows of 16 lanes, then the rows' sums as scalars.
template <bool WAVE>
__device__ __forceinline__ float wave_total(float v) {
  auto add = [&](uint32_t moved) { v += __uint_as_float(moved); };
  add(dpp_move<0xB1>(__float_as_uint(v)));
  add(dpp_move<0x4E>(__float_as_uint(v)));
  add(dpp_move<0x141>(__float_as_uint(v)));
  add(dpp_move<0x140>(__float_as_uint(v)));
  if (!WAVE) return v;
  auto row = [&](int lane) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Sums of K values over the TPR threads of a row, in all of them, with one
// barrier.  part: K x waves of LDS that the block's next sum must not use.
template <class C, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*part)[C::NT / 64]) {
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = wave_total<C::TPR >= 64>(v[i]);
  if constexpr (C::TPR > 64) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) part[i][threadIdx.x >> 6] = v[i];
    __syncthreads();
    const int first = threadIdx.x / C::TPR * (C::TPR / 64);
#pragma unroll
    for (int i = 0; i < K; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int j = 0; j < C::TPR / 64; ++j) v[i] += part[i][first + j];
    }
  }
}

// How a row is cut into pieces of V values.  EVEN: whole pieces, 16-byte aligned;
// else (rows of any alignment, V values at least) the last one may have fewer: it
// is loaded from V values before the row's end on, and those of the piece before
// it are dropped.  16,384 bf16 rows of 4099 values 111 us and backward 136 (of 4096
// values 90 and 107); one value at a time they took 339 and 277.  Unaligned fp32
// rows of 8193 values and more are furthest from aligned ones: the backward pass of
// their 16 columns a thread wants more than the 128 registers that 1024 threads
// leave, and 23 of them go to memory (4096 x 12,001 205 us, 12,000 155; 8201 154,
// 8200 114).
template <class T, int V, bool STREAM, bool EVEN>
struct Cut {
  using IV = std::conditional_t<EVEN, i32x4, i32x4_any>;
  int cols, pieces;
  __device__ explicit Cut(int64_t n) : cols((int)n), pieces(EVEN ? (int)n / V : ((int)n + V - 1) / V) {}
  // Values of piece c that the load has too many in front.
  __device__ int extra(int c) const { return EVEN ? 0 : max(0, c * V - (cols - V)); }
  __device__ Piece<T, V> load(const char* row, int c) const {
    return piece_load<T, V, STREAM, IV>(row + (int64_t)(c * V - extra(c)) * sizeof(T));
  }
  // Takes off what load() had too many.
  __device__ void trim(Piece<T, V>& p, int c) const {
    if constexpr (!EVEN)
      if (const int n = extra(c)) piece_drop<T, V>(p, n);
  }
  __device__ void store(char* row, int c, const float (&v)[V]) const {
    T* p = (T*)row + c * V;
    if (!EVEN && c * V + V > cols) {
      piece_store_first<T, V>(p, v, cols - c * V);
    } else {
      piece_store<T, V, STREAM, IV>(p, v);
    }
  }
  // Of the weight; zeros past the row.
  __device__ void weights(const void* w, bool f32, int c, float (&v)[V]) const {
    if (EVEN || c * V + V <= cols) {
      weight_values<V>(w, f32, (int64_t)c * V, v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float one[1] = {0.f};
        if (c * V + i < cols) weight_values<1>(w, f32, c * V + i, one);
        v[i] = one[0];
      }
    }
  }
};

template <class C, class T, int V, bool STREAM, bool EVEN>
__global__ void __launch_bounds__(C::NT)
rms_norm_kernel(NormArgs a) {
  __shared__ float part[1][C::NT / 64];
  const int tid = threadIdx.x % C::TPR;
  const int64_t row = (int64_t)blockIdx.x * C::RPB + threadIdx.x / C::TPR;
  const bool in = row < a.rows;
  const Cut<T, V, STREAM, EVEN> cut(a.cols);
  const int pieces = cut.pieces;
  const char* x = (const char*)a.x + row * a.ldx;
  const char* res = (const char*)a.residual + row * a.ldr;
  Piece<T, V> px[C::NC], pr[C::NC];
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    const int c = tid + C::TPR * i;
    const bool have = in && c < pieces;
    px[i] = have ? cut.load(x, c) : piece_zero<T, V>();
    pr[i] = have && a.residual ? cut.load(res, c) : piece_zero<T, V>();
  }
  float s[C::NC][V], sums[1] = {0.f};
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    float r[V];
    cut.trim(px[i], tid + C::TPR * i);
    cut.trim(pr[i], tid + C::TPR * i);
    piece_values<T, V>(px[i], s[i]);
    piece_values<T, V>(pr[i], r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[i][v] += r[v];
      sums[0] += s[i][v] * s[i][v];
    }
  }
  row_sums<C>(sums, part);
  const float scale = 1.0f / sqrtf(sums[0] / (float)a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    const int c = tid + C::TPR * i;
    const bool have = in && c < pieces;
    if (have && a.stream) cut.store((char*)a.stream + row * a.lds, c, s[i]);
    float w[V];
    if (have) {
      cut.weights(a.weight, a.weight_f32, c, w);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = s[i][v] * scale * w[v];
    if (have && a.y) cut.store((char*)a.y + row * a.ldy, c, w);
    if constexpr (EVEN && V > 1) {
      if (a.q.codes) {  // from the fp32 values: rounded once
        uint32_t codes[V / 4];
        const int byte = mx8_block<V>(w, codes);
        if (have) {
          constexpr int G = MX_BLOCK / V;
          store_codes(a.q.codes + row * a.q.ldc + (int64_t)c * V, codes);
          if (c % G == 0) mx8_store_scale(a.q.scales + row * a.q.lds, c / G, pieces / G, byte);
        }
      }
    }
  }
}

// Workgroup b takes rows b RPB .., (b + gridDim) RPB .., and keeps the weight and
// the weight's gradient of its threads' columns in registers; at the end it adds
// up those of its RPB rows at a time to one row of partial sums.  The next row's
// values are loaded before this row's sums are waited for (AHEAD; not where a
// thread has so many pieces that registers would run out).
template <class C, class T, int V, bool STREAM, bool EVEN>
__global__ void __launch_bounds__(C::NT)
rms_norm_backward_kernel(NormBackArgs a) {
  constexpr bool AHEAD = C::NC <= 3 && C::NT < 1024;
  __shared__ float part[4][C::NT / 64];
  const int tid = threadIdx.x % C::TPR, sub = threadIdx.x / C::TPR;
  const Cut<T, V, STREAM, EVEN> cut(a.cols);
  const int pieces = cut.pieces;
  const int64_t stride = (int64_t)gridDim.x * C::RPB;
  float dw[C::NC][V], w[C::NC][V];
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    const int c = tid + C::TPR * i;
#pragma unroll
    for (int v = 0; v < V; ++v) dw[i][v] = w[i][v] = 0.f;
    if (c < pieces) cut.weights(a.weight, a.weight_f32, c, w[i]);
  }
  struct Row {
    Piece<T, V> s[C::NC], d[C::NC], t[C::NC];
  };
  auto load = [&](Row& x, int64_t row) {
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      const bool have = row < a.rows && c < pieces;
      x.s[i] = have ? cut.load((const char*)a.s + row * a.lds, c) : piece_zero<T, V>();
      x.d[i] = have ? cut.load((const char*)a.dy + row * a.lddy, c) : piece_zero<T, V>();
      x.t[i] = have && a.dstream ? cut.load((const char*)a.dstream + row * a.ldds, c) : piece_zero<T, V>();
    }
  };
  Row x;
  if (AHEAD) load(x, (int64_t)blockIdx.x * C::RPB + sub);
  int slot = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * C::RPB; row0 < a.rows; row0 += stride, slot ^= 2) {
    const int64_t row = row0 + sub;
    if (!AHEAD) load(x, row);
    float sums[2] = {0.f, 0.f};  // of s^2 and of g s
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      float s[V], d[V];
      cut.trim(x.s[i], c);
      cut.trim(x.d[i], c);
      cut.trim(x.t[i], c);
      piece_values<T, V>(x.s[i], s);
      piece_values<T, V>(x.d[i], d);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sums[0] += s[v] * s[v];
        sums[1] += d[v] * w[i][v] * s[v];
      }
    }
    Row next;
    if (AHEAD) load(next, row + stride);
    row_sums<C>(sums, part + slot);
    // (0 past the last row, where eps 0 would make it infinite)
    const float r = row < a.rows ? 1.0f / sqrtf(sums[0] / (float)a.cols + a.eps) : 0.0f;
    const float mean = sums[1] * r / (float)a.cols;  // of g n
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      float s[V], d[V], t[V];
      piece_values<T, V>(x.s[i], s);
      piece_values<T, V>(x.d[i], d);
      piece_values<T, V>(x.t[i], t);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float n = s[v] * r;
        dw[i][v] += d[v] * n;
        t[v] += r * (d[v] * w[i][v] - n * mean);
      }
      if (row < a.rows && c < pieces) cut.store((char*)a.dx + row * a.lddx, c, t);
    }
    if (AHEAD) x = next;
  }
  float* out = a.part + (int64_t)blockIdx.x * a.cols;
  if constexpr (C::RPB > 1) {
    __shared__ float sums[C::NT * V];  // [sub][tid][V]
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) sums[threadIdx.x * V + v] = dw[i][v];
      __syncthreads();
      for (int j = threadIdx.x; j < C::TPR * V; j += C::NT) {
        float all = 0.f;
#pragma unroll
        for (int q = 0; q < C::RPB; ++q) all += sums[q * C::TPR * V + j];
        const int col = C::TPR * i * V + j;
        if (col < cut.cols) out[col] = all;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      if (c >= pieces) continue;
      if (EVEN || c * V + V <= cut.cols) {
#pragma unroll
        for (int v = 0; v < V; ++v) out[c * V + v] = dw[i][v];
      } else {
#pragma unroll
        for (int v = 0; v < V - 1; ++v)
          if (c * V + v < cut.cols) out[c * V + v] = dw[i][v];
      }
    }
  }
}

// Column sums of the partial rows, in a fixed order: 16 columns by 64 threads each.
__global__ void __launch_bounds__(1024)
norm_dweight_kernel(const float* __restrict__ part, int64_t parts, int64_t cols, float* __restrict__ dweight) {
  __shared__ float sums[64][17];
  const int cx = threadIdx.x & 15, py = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + cx;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int64_t p = py; p < parts; p += 64) s += part[p * cols + col];
  }
  sums[py][cx] = s;
  __syncthreads();
  if (threadIdx.x < 16 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += sums[i][cx];
    dweight[col] = s;
  }
}

// Threads to a row by its pieces (V = 1: rows of fewer values than 16 bytes
// hold).  Rows of 6144 bf16 values, 256 threads of 3 pieces, 384 of 2 and 768 of 1:
// backward of 65,536 rows 448, 490 and 510 us, with a gradient beside the norm 590,
// 613 and 590, of 8192 rows with one 88, 99 and 95 (all with the sum of the partial
// rows).  Forward with 256 and with 384 threads: 8192 rows with both outputs 78 and
// 75 us, without the 8-bit ones 68 and 65 (2048 rows and the quantisation after it
// 24 and 26: the larger calls decide).  65,536 rows of 100 bf16 values with 16
// lanes to a row 9 us, 12 with a residual, and backward 15.6; with a wave to a row
// 28 with a residual and backward 44.
template <int V, bool BACKWARD, class F>
void with_row(int64_t pieces, F f) {
  if constexpr (V == 1) {
    f(RowCfg<16, 1>());
  } else {
    if (pieces <= 16) f(RowCfg<16, 1>());
    else if (pieces <= 32) f(RowCfg<16, 2>());
    else if (pieces <= 64) f(RowCfg<64, 1>());
    else if (pieces <= 128) f(RowCfg<64, 2>());
    else if (pieces <= 256) f(RowCfg<128, 2>());
    else if (pieces <= 512) f(RowCfg<256, 2>());
    else if (pieces <= 768) f(RowCfg<BACKWARD ? 256 : 384, BACKWARD ? 3 : 2>());
    else if (pieces <= 1024) f(RowCfg<512, 2>());
    else if (V == 8 || pieces <= 2048) f(RowCfg<1024, 2>());  // 16,384 values at most
    else f(RowCfg<1024, V == 8 ? 2 : 4>());
  }
}

template <class T, int V, bool STREAM, bool EVEN>
hipError_t run_norm(const NormArgs& a, hipStream_t st) {
  with_row<V, false>((a.cols + V - 1) / V, [&](auto cfg) {
    using C = decltype(cfg);
    constexpr int64_t most = (int64_t)C::RPB << 21;  // rows of a launch, which has fewer than 2^32 threads
    for (int64_t r = 0; r < a.rows; r += most) {
      NormArgs b = a;
      b.rows = a.rows - r < most ? a.rows - r : most;
      b.x = (const char*)a.x + r * a.ldx;
      if (a.residual) b.residual = (const char*)a.residual + r * a.ldr;
      if (a.stream) b.stream = (char*)a.stream + r * a.lds;
      if (a.y) b.y = (char*)a.y + r * a.ldy;
      if (a.q.codes) {
        b.q.codes += r * a.q.ldc;
        b.q.scales += r * a.q.lds;
      }
      launch((rms_norm_kernel<C, T, V, STREAM, EVEN>), dim3((unsigned)((b.rows + C::RPB - 1) / C::RPB)), dim3(C::NT), 0, st, b);
    }
  });
  return hipGetLastError();
}

// Workgroups of the backward pass, which has `rpb` rows in each at a time.
int64_t norm_groups(int64_t rows, int64_t cols, int rpb) {
  const int64_t most = norm_parts(rows, cols), fill = most < 1024 ? most : 1024, rounds = (rows + rpb - 1) / rpb;
  return std::min(rounds, std::max(most / rpb, fill));
}

template <class T, int V, bool STREAM, bool EVEN>
hipError_t run_norm_backward(NormBackArgs& a, hipStream_t st) {
  with_row<V, true>((a.cols + V - 1) / V, [&](auto cfg) {
    using C = decltype(cfg);
    a.parts = norm_groups(a.rows, a.cols, C::RPB);
    launch((rms_norm_backward_kernel<C, T, V, STREAM, EVEN>), dim3((unsigned)a.parts), dim3(C::NT), 0, st, a);
  });
  return hipGetLastError();
}

// f(type, V, STREAM, EVEN) by the type, the width, the bytes touched and the alignment of every row that is touched.
template <class F>
hipError_t by_rows(bool bf16, int64_t cols, int64_t bytes, uintptr_t bits, F f) {
  const auto at = [&](auto t) {
    using T = decltype(t);
    constexpr int V = 16 / sizeof(T);
    const auto cut = [&](auto even) {
      return bytes > STREAM_BYTES ? f(t, std::integral_constant<int, V>(), std::true_type(), even)
                                  : f(t, std::integral_constant<int, V>(), std::false_type(), even);
    };
    if (cols < V) return f(t, std::integral_constant<int, 1>(), std::false_type(), std::true_type());
    return cols % V == 0 && bits % 16 == 0 ? cut(std::true_type()) : cut(std::false_type());
  };
  return bf16 ? at(bf16_t{}) : at(float{});
}

}  // namespace

// One for each row up to 1024, which fill the card, then one for 16 rows or
// more, and no more than 1024 workgroups need.
int64_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t most = cols <= 2048 ? 4096 : 1024;
  return std::min(most, std::max(std::min<int64_t>(rows, 1024), (rows + 15) / 16));
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st) {
  uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.ldx | (uintptr_t)a.weight;
  if (a.residual) bits |= (uintptr_t)a.residual | (uintptr_t)a.ldr;
  if (a.stream) bits |= (uintptr_t)a.stream | (uintptr_t)a.lds;
  if (a.y) bits |= (uintptr_t)a.y | (uintptr_t)a.ldy;
  const int64_t rows = 1 + (a.residual != nullptr) + (a.stream != nullptr) + (a.y != nullptr);
  return by_rows(a.bf16, a.cols, rows * a.rows * a.cols * (a.bf16 ? 2 : 4), bits, [&](auto t, auto v, auto stream, auto even) {
    return run_norm<decltype(t), decltype(v)::value, decltype(stream)::value, decltype(even)::value>(a, st);
  });
}

hipError_t launch_rms_norm_backward(NormBackArgs& a, hipStream_t st) {
  uintptr_t bits = (uintptr_t)a.dy | (uintptr_t)a.lddy | (uintptr_t)a.s | (uintptr_t)a.lds | (uintptr_t)a.dx |
                   (uintptr_t)a.lddx | (uintptr_t)a.weight;
  if (a.dstream) bits |= (uintptr_t)a.dstream | (uintptr_t)a.ldds;
  const int64_t bytes = (a.dstream ? 4 : 3) * a.rows * a.cols * (a.bf16 ? 2 : 4);
  return by_rows(a.bf16, a.cols, bytes, bits, [&](auto t, auto v, auto stream, auto even) {
    return run_norm_backward<decltype(t), decltype(v)::value, decltype(stream)::value, decltype(even)::value>(a, st);
  });
}

hipError_t launch_norm_dweight(const NormBackArgs& a, hipStream_t st) {
  launch(norm_dweight_kernel, dim3((unsigned)((a.cols + 15) / 16)), dim3(1024), 0, st, a.part, a.parts, a.cols, a.dweight);
  return hipGetLastError();
}

}  // namespace moe
