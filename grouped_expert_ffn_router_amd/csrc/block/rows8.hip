// MX-FP8 rows: quantisation and its inverse, SwiGLU with its checkpoint in
// that form, and the backward pass that reads the checkpoint (gfx950).

#include "block.h"

namespace moe {

namespace {

// Launches f(first block, blocks) over `blocks` blocks of 256 threads, 2^23 at
// a time (a launch has fewer than 2^32 threads).
template <class F>
hipError_t in_launches(int64_t blocks, F f) {
  for (int64_t b = 0; b < blocks; b += 1 << 23) f(b, dim3((unsigned)(blocks - b < 1 << 23 ? blocks - b : 1 << 23)));
  return hipGetLastError();
}

// The rows and pieces of `per` to a row that thread threadIdx.x of a block has:
// pieces (block * U + u) * 256 + threadIdx.x, row after row.
struct Place {
  int64_t row;
  int piece;
};
template <int U>
__device__ __forceinline__ void places(int64_t block, int per, Place (&p)[U]) {
  const int64_t first = block * (256 * U);
  const int64_t row0 = first / per;
  const uint32_t off0 = (uint32_t)(first - row0 * per);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t loc = off0 + threadIdx.x + 256 * u, r = loc / (uint32_t)per;
    p[u].row = row0 + r;
    p[u].piece = (int)(loc - r * (uint32_t)per);
  }
}

// ------------------------------------------------------------ rows <-> MX-FP8
//
// One lane takes 16 bytes of activations (8 bf16 or 4 fp32 values), so a block
// of 32 is a group of 4 or 8 neighbouring lanes, whose largest magnitude is a
// maximum over bit patterns taken with DPP moves.  Bound by bytes: 8192 x 6144
// from bf16 and back to it 24 us each (6.4 TB/s; a copy of 4 GB reaches 4.8 on
// this card, a kernel that mostly reads 6.8, and here part of the operands are in
// the caches).

constexpr int UNROLL = 2;  // pieces a lane

template <class T, bool STREAM>
__global__ void __launch_bounds__(256)
mx8_quantize_kernel(const char* __restrict__ x, int64_t ldx, int64_t rows, int64_t block0, int per, Rows8 q) {
  constexpr int V = 16 / sizeof(T), G = MX_BLOCK / V;
  Place p[UNROLL];
  places(block0 + blockIdx.x, per, p);
  Piece<T, V> d[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u)
    d[u] = p[u].row < rows ? piece_load<T, V, STREAM>(x + p[u].row * ldx + (int64_t)p[u].piece * 16) : piece_zero<T, V>();
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    float v[V];
    uint32_t c[V / 4];
    piece_values<T, V>(d[u], v);
    const int byte = mx8_block<V>(v, c);  // rows start at a group boundary, so a group is one block
    if (p[u].row >= rows) continue;
    store_codes(q.codes + p[u].row * q.ldc + (int64_t)p[u].piece * V, c);
    if (p[u].piece % G == 0) mx8_store_scale(q.scales + p[u].row * q.lds, p[u].piece / G, per / G, byte);
  }
}

template <class T, bool STREAM>
__global__ void __launch_bounds__(256)
mx8_dequantize_kernel(Rows8 q, int64_t rows, int64_t block0, int per, char* __restrict__ out, int64_t ldo) {
  constexpr int V = 16 / sizeof(T), G = MX_BLOCK / V;
  Place p[UNROLL];
  places(block0 + blockIdx.x, per, p);
  uint32_t c[UNROLL][V / 4], s[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const bool in = p[u].row < rows;
    const uint8_t* row = q.codes + p[u].row * q.ldc + (int64_t)p[u].piece * V;
    s[u] = in ? q.scales[p[u].row * q.lds + p[u].piece / G] : 0;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) c[u][i] = 0;
    if (in) load_codes(row, c[u]);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    if (p[u].row >= rows) continue;
    float v[V];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) mx8_values4(c[u][i], mx_scale(s[u]), v + 4 * i);
    piece_store<T, V, STREAM>(out + p[u].row * ldo + (int64_t)p[u].piece * 16, v);
  }
}

// ------------------------------------------------------------ SwiGLU
//
// h = a sigmoid(a) b of a gate value a and an up value b; with sg = sigmoid(a),
//   da = dh b sg (1 + a (1 - sg)),  db = dh a sg.
// Everything between the loads and the stores is fp32 (exp and reciprocal are
// the hardware's: (2 + 1.5 |a|) 2^-24 off).  A lane has 16 bytes of gate values and
// the up values that belong to them.  Bound by bytes: two experts of 12,562
// places, 80 % of them taken, x 2048 hidden units in bf16, forward 56 us (5.9
// TB/s), backward with h again 65 us (6.4 TB/s); with two pieces a lane 3 and 4 %
// more, with four 10 and 14.

template <class T, bool STREAM>
__global__ void __launch_bounds__(256)
swiglu_checkpoint_kernel(SwigluArgs a, int64_t block0, int per) {
  constexpr int V = 16 / sizeof(T), G = MX_BLOCK / V;
  Place p[1];
  places(block0 + blockIdx.x, per, p);
  const int64_t rows = a.groups * a.max_rows, row = p[0].row;
  bool in = row < rows;
  if (in && a.counts) {
    const int64_t g = row / a.max_rows;
    in = row - g * a.max_rows < a.counts[g];
  }
  const char* src = (const char*)a.gate_up + row * a.ldg + (int64_t)p[0].piece * 16;
  const int64_t half = a.hidden * sizeof(T);
  const Piece<T, V> pg = in ? piece_load<T, V, STREAM>(src) : piece_zero<T, V>();
  const Piece<T, V> pu = in ? piece_load<T, V, STREAM>(src + half) : piece_zero<T, V>();
  float g[V], u[V], h[V];
  uint32_t cg[V / 4], cu[V / 4];
  piece_values<T, V>(pg, g);
  piece_values<T, V>(pu, u);
  const int sg = mx8_block<V>(g, cg), su = mx8_block<V>(u, cu);
  if (!in) return;
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = silu(g[i]) * u[i];
  piece_store<T, V, STREAM>((char*)a.h + row * a.ldh + (int64_t)p[0].piece * 16, h);
  uint8_t* codes = a.q.codes + row * a.q.ldc + (int64_t)p[0].piece * V;
  store_codes(codes, cg);
  store_codes(codes + a.hidden, cu);
  if (p[0].piece % G == 0) {
    const int b = p[0].piece / G, nb = per / G;
    uint8_t* srow = a.q.scales + row * a.q.lds;
    srow[b] = (uint8_t)sg;
    mx8_store_scale(srow, nb + b, 2 * nb, su);
  }
}

template <class T, bool STREAM>
__global__ void __launch_bounds__(256)
swiglu_backward_kernel(SwigluArgs a, int64_t block0, int per) {
  constexpr int V = 16 / sizeof(T), G = MX_BLOCK / V;
  Place p[1];
  places(block0 + blockIdx.x, per, p);
  const int64_t row = p[0].row;
  if (row >= a.groups * a.max_rows) return;
  if (a.counts) {
    const int64_t g = row / a.max_rows;
    if (row - g * a.max_rows >= a.counts[g]) return;
  }
  const uint8_t* codes = a.q.codes + row * a.q.ldc + (int64_t)p[0].piece * V;
  const uint8_t* srow = a.q.scales + row * a.q.lds + p[0].piece / G;
  const Piece<T, V> pd = piece_load<T, V, STREAM>((const char*)a.dh + row * a.ldd + (int64_t)p[0].piece * 16);
  const float ug = mx_scale(srow[0]), uu = mx_scale(srow[per / G]);
  float g[V], u[V], d[V], h[V];
  uint32_t cg[V / 4], cu[V / 4];
  load_codes(codes, cg);
  load_codes(codes + a.hidden, cu);
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    mx8_values4(cg[i], ug, g + 4 * i);
    mx8_values4(cu[i], uu, u + 4 * i);
  }
  piece_values<T, V>(pd, d);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float sg = __builtin_amdgcn_rcpf(1.0f + __expf(-g[i])), act = g[i] * sg, dd = d[i];
    h[i] = act * u[i];
    d[i] = dd * u[i] * sg * (1.0f + g[i] * (1.0f - sg));
    u[i] = dd * act;
  }
  char* out = (char*)a.dgate_up + row * a.ldg + (int64_t)p[0].piece * 16;
  piece_store<T, V, STREAM>(out, d);
  piece_store<T, V, STREAM>(out + a.hidden * sizeof(T), u);
  if (a.h) piece_store<T, V, STREAM>((char*)a.h + row * a.ldh + (int64_t)p[0].piece * 16, h);
}

int64_t blocks_of(int64_t pieces, int unroll) { return (pieces + 256 * unroll - 1) / (256 * unroll); }

// f<T, STREAM>() by type and by whether the bytes touched go past the caches.
template <class F>
void by_form(bool bf16, int64_t bytes, F f) {
  if (bytes > STREAM_BYTES) {
    if (bf16) f(bf16_t{}, std::true_type());
    else f(float{}, std::true_type());
  } else {
    if (bf16) f(bf16_t{}, std::false_type());
    else f(float{}, std::false_type());
  }
}

}  // namespace

hipError_t launch_mx8_quantize(bool bf16, int64_t rows, int64_t cols, const void* x, int64_t ldx, const Rows8& q,
                               hipStream_t st) {
  const int size = bf16 ? 2 : 4, per = (int)(cols * size / 16);
  return in_launches(blocks_of(rows * per, UNROLL), [&](int64_t b, dim3 grid) {
    by_form(bf16, rows * cols * (size + 1), [&](auto t, auto stream) {
      launch((mx8_quantize_kernel<decltype(t), decltype(stream)::value>), grid, dim3(256), 0, st, (const char*)x, ldx, rows, b,
             per, q);
    });
  });
}

hipError_t launch_mx8_dequantize(bool bf16, int64_t rows, int64_t cols, const Rows8& q, void* out, int64_t ldo,
                                 hipStream_t st) {
  const int size = bf16 ? 2 : 4, per = (int)(cols * size / 16);
  return in_launches(blocks_of(rows * per, UNROLL), [&](int64_t b, dim3 grid) {
    by_form(bf16, rows * cols * (size + 1), [&](auto t, auto stream) {
      launch((mx8_dequantize_kernel<decltype(t), decltype(stream)::value>), grid, dim3(256), 0, st, q, rows, b, per, (char*)out,
             ldo);
    });
  });
}

hipError_t launch_swiglu_checkpoint(const SwigluArgs& a, hipStream_t st) {
  const int size = a.bf16 ? 2 : 4, per = (int)(a.hidden * size / 16);
  const int64_t rows = a.groups * a.max_rows;
  return in_launches(blocks_of(rows * per, 1), [&](int64_t b, dim3 grid) {
    by_form(a.bf16, rows * a.hidden * (3 * size + 2), [&](auto t, auto stream) {
      launch((swiglu_checkpoint_kernel<decltype(t), decltype(stream)::value>), grid, dim3(256), 0, st, a, b, per);
    });
  });
}

hipError_t launch_swiglu_backward(const SwigluArgs& a, hipStream_t st) {
  const int size = a.bf16 ? 2 : 4, per = (int)(a.hidden * size / 16);
  const int64_t rows = a.groups * a.max_rows;
  return in_launches(blocks_of(rows * per, 1), [&](int64_t b, dim3 grid) {
    by_form(a.bf16, rows * a.hidden * ((a.h ? 4 : 3) * size + 2), [&](auto t, auto stream) {
      launch((swiglu_backward_kernel<decltype(t), decltype(stream)::value>), grid, dim3(256), 0, st, a, b, per);
    });
  });
}

}  // namespace moe
