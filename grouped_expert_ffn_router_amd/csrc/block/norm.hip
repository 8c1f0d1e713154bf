// Root-mean-square norm of rows after the residual stream's addition, and its
// backward pass (gfx950).
//
//   s = x + residual,  r = (mean(s^2) + eps)^-1/2,  y = s r w
//   with n = s r, g = dy w:  dx = r (g - n mean(g n)) + dstream,  dw = sum over rows of dy n

#include "block.h"

namespace moe {

namespace {

// A row is NC pieces of V values for each of TPR threads (piece tid + TPR i of
// thread tid), kept in registers between the row's sum and its use: every
// value is read once and written once.
template <int TPR_, int NC_>
struct RowCfg {
  static constexpr int TPR = TPR_, NC = NC_, NT = TPR > 256 ? TPR : 256, RPB = NT / TPR;
};

// Sum over the TPR threads of a row, in all of them, in a fixed order.
// part: NT / 64 values of LDS, used alternately (slot) by the block's rows.
template <class C>
__device__ __forceinline__ float row_sum(float v, float (*part)[C::NT / 64], int slot) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if constexpr (C::TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < C::TPR / 64; ++i) v += part[slot][i];
  }
  return v;
}

template <class C, class T, int V>
__global__ void __launch_bounds__(C::NT)
rms_norm_kernel(NormArgs a) {
  __shared__ float part[1][C::NT / 64];
  const int tid = threadIdx.x % C::TPR;
  const int64_t row = (int64_t)blockIdx.x * C::RPB + threadIdx.x / C::TPR;
  const bool in = row < a.rows;
  const int pieces = (int)(a.cols / V);
  const char* x = (const char*)a.x + row * a.ldx;
  const char* res = (const char*)a.residual + row * a.ldr;
  Piece<T, V> px[C::NC], pr[C::NC];
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    const int c = tid + C::TPR * i;
    const bool have = in && c < pieces;
    px[i] = have ? piece_load<T, V>(x + (int64_t)c * (V * sizeof(T))) : piece_zero<T, V>();
    pr[i] = have && a.residual ? piece_load<T, V>(res + (int64_t)c * (V * sizeof(T))) : piece_zero<T, V>();
  }
  float s[C::NC][V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    float r[V];
    piece_values<T, V>(px[i], s[i]);
    piece_values<T, V>(pr[i], r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[i][v] += r[v];
      sum += s[i][v] * s[i][v];
    }
  }
  sum = row_sum<C>(sum, part, 0);
  const float scale = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    const int c = tid + C::TPR * i;
    const bool have = in && c < pieces;
    if (have && a.stream) piece_store<T, V>((char*)a.stream + row * a.lds + (int64_t)c * (V * sizeof(T)), s[i]);
    float w[V];
    if (have) {
      weight_values<V>(a.weight, a.weight_f32, (int64_t)c * V, w);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = s[i][v] * scale * w[v];
    if (have && a.y) piece_store<T, V>((char*)a.y + row * a.ldy + (int64_t)c * (V * sizeof(T)), w);
    if constexpr (V > 1) {
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

// Workgroup b takes rows b RPB .., b RPB + gridDim RPB .., and keeps the weight's
// gradient of its threads' columns in registers; one row of partial sums for
// each RPB-th of a workgroup.
template <class C, class T, int V>
__global__ void __launch_bounds__(C::NT)
rms_norm_backward_kernel(NormBackArgs a) {
  __shared__ float part[4][C::NT / 64];
  const int tid = threadIdx.x % C::TPR, sub = threadIdx.x / C::TPR;
  const int pieces = (int)(a.cols / V);
  float dw[C::NC][V];
#pragma unroll
  for (int i = 0; i < C::NC; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[i][v] = 0.f;
  int slot = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * C::RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * C::RPB, slot ^= 2) {
    const int64_t row = row0 + sub;
    const bool in = row < a.rows;
    Piece<T, V> pd[C::NC], ps[C::NC], pt[C::NC];
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      const bool have = in && c < pieces;
      const int64_t at = (int64_t)c * (V * sizeof(T));
      ps[i] = have ? piece_load<T, V>((const char*)a.s + row * a.lds + at) : piece_zero<T, V>();
      pd[i] = have ? piece_load<T, V>((const char*)a.dy + row * a.lddy + at) : piece_zero<T, V>();
      pt[i] = have && a.dstream ? piece_load<T, V>((const char*)a.dstream + row * a.ldds + at) : piece_zero<T, V>();
    }
    float square = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      float s[V], d[V], w[V];
      piece_values<T, V>(ps[i], s);
      piece_values<T, V>(pd[i], d);
      if (c < pieces) {
        weight_values<V>(a.weight, a.weight_f32, (int64_t)c * V, w);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        square += s[v] * s[v];
        dot += d[v] * w[v] * s[v];
      }
    }
    square = row_sum<C>(square, part, slot);
    dot = row_sum<C>(dot, part, slot + 1);
    const float r = 1.0f / sqrtf(square / (float)a.cols + a.eps);
    const float mean = dot * r / (float)a.cols;  // of g n
#pragma unroll
    for (int i = 0; i < C::NC; ++i) {
      const int c = tid + C::TPR * i;
      if (!in || c >= pieces) continue;
      float s[V], d[V], w[V], t[V];
      piece_values<T, V>(ps[i], s);
      piece_values<T, V>(pd[i], d);
      piece_values<T, V>(pt[i], t);
      weight_values<V>(a.weight, a.weight_f32, (int64_t)c * V, w);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float n = s[v] * r;
        dw[i][v] += d[v] * n;
        t[v] += r * (d[v] * w[v] - n * mean);
      }
      piece_store<T, V>((char*)a.dx + row * a.lddx + (int64_t)c * (V * sizeof(T)), t);
    }
  }
  float* out = a.part + ((int64_t)blockIdx.x * C::RPB + sub) * a.cols;
#pragma unroll
  for (int i = 0; i < C::NC; ++i) {
    const int c = tid + C::TPR * i;
    if (c >= pieces) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) out[(int64_t)c * V + v] = dw[i][v];
  }
}

// Column sums of the partial rows, in a fixed order: 32 columns by 32 threads each.
__global__ void __launch_bounds__(1024)
norm_dweight_kernel(const float* __restrict__ part, int64_t parts, int64_t cols, float* __restrict__ dweight) {
  __shared__ float sums[32][33];
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + cx;
  float s = 0.f;
  if (col < cols)
    for (int64_t p = py; p < parts; p += 32) s += part[p * cols + col];
  sums[py][cx] = s;
  __syncthreads();
  if (py == 0 && col < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sums[i][cx];
    dweight[col] = s;
  }
}

// Threads to a row by its pieces.  V = 1 (rows that are not 16-byte aligned) has the fewest forms.
template <int V, class F>
void with_row(int64_t pieces, F f) {
  if constexpr (V == 1) {
    if (pieces <= 256) f(RowCfg<64, 4>());
    else if (pieces <= 2048) f(RowCfg<256, 8>());
    else f(RowCfg<1024, 16>());
  } else {
    if (pieces <= 64) f(RowCfg<64, 1>());
    else if (pieces <= 256) f(RowCfg<64, 4>());
    else if (pieces <= 768) f(RowCfg<256, 3>());
    else if (pieces <= 2048) f(RowCfg<256, 8>());
    else f(RowCfg<1024, 4>());
  }
}

template <class T, int V>
hipError_t run_norm(const NormArgs& a, hipStream_t st) {
  with_row<V>(a.cols / V, [&](auto cfg) {
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
      launch((rms_norm_kernel<C, T, V>), dim3((unsigned)((b.rows + C::RPB - 1) / C::RPB)), dim3(C::NT), 0, st, b);
    }
  });
  return hipGetLastError();
}

template <class T, int V>
hipError_t run_norm_backward(const NormBackArgs& a, hipStream_t st) {
  with_row<V>(a.cols / V, [&](auto cfg) {
    using C = decltype(cfg);
    launch((rms_norm_backward_kernel<C, T, V>), dim3((unsigned)(a.parts / C::RPB)), dim3(C::NT), 0, st, a);
  });
  return hipGetLastError();
}

// 16 bytes at a time where every row that is touched allows it.
bool wide(bool bf16, int64_t cols, uintptr_t bits) { return cols % (bf16 ? 8 : 4) == 0 && bits % 16 == 0; }

}  // namespace

// A multiple of 4, the most rows that a workgroup has at once.  1024 workgroups
// fill the card four times over; 16 rows or more of each keep the partial sums'
// bytes below an eighth of the rows'.
int64_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t p = (rows + 15) / 16, most = cols <= 2048 ? 4096 : 1024;
  return p >= most ? most : (p + 3) / 4 * 4;
}

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t st) {
  uintptr_t bits = (uintptr_t)a.x | (uintptr_t)a.ldx | (uintptr_t)a.weight;
  if (a.residual) bits |= (uintptr_t)a.residual | (uintptr_t)a.ldr;
  if (a.stream) bits |= (uintptr_t)a.stream | (uintptr_t)a.lds;
  if (a.y) bits |= (uintptr_t)a.y | (uintptr_t)a.ldy;
  if (wide(a.bf16, a.cols, bits)) return a.bf16 ? run_norm<bf16_t, 8>(a, st) : run_norm<float, 4>(a, st);
  return a.bf16 ? run_norm<bf16_t, 1>(a, st) : run_norm<float, 1>(a, st);
}

hipError_t launch_rms_norm_backward(const NormBackArgs& a, hipStream_t st) {
  uintptr_t bits = (uintptr_t)a.dy | (uintptr_t)a.lddy | (uintptr_t)a.s | (uintptr_t)a.lds | (uintptr_t)a.dx |
                   (uintptr_t)a.lddx | (uintptr_t)a.weight;
  if (a.dstream) bits |= (uintptr_t)a.dstream | (uintptr_t)a.ldds;
  if (wide(a.bf16, a.cols, bits)) return a.bf16 ? run_norm_backward<bf16_t, 8>(a, st) : run_norm_backward<float, 4>(a, st);
  return a.bf16 ? run_norm_backward<bf16_t, 1>(a, st) : run_norm_backward<float, 1>(a, st);
}

hipError_t launch_norm_dweight(const NormBackArgs& a, hipStream_t st) {
  launch(norm_dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, st, a.part, a.parts, a.cols, a.dweight);
  return hipGetLastError();
}

}  // namespace moe
