// MX-FP4 rows: quantisation, its inverse, and the grouped product (gfx950).

#include "mx.h"

namespace moe {

// ------------------------------------------------------------ rows <-> MX-FP4
//
// One lane takes 16 bytes of activations (8 bf16 or 4 fp32 values), so a block
// of 32 is a group of 4 or 8 neighbouring lanes: the block's largest magnitude
// is a maximum over the bit patterns (sign dropped; infinities and NaN come out
// on top) taken with DPP moves inside the group.  Bytes bound both ways: a value
// is read or written once as an activation and once as 17/32 of a byte.
// MI355X, 131,072 x 2048 bf16: 142 us to MX-FP4 (4.8 TB/s, the rate of a large
// copy) and 101 us back (6.7 TB/s).

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}

// Maximum over groups of G = 4 or 8 lanes: quad permutations [1,0,3,2] and
// [2,3,0,1], then a mirror of 8 lanes, which swaps the two quads.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, dpp_u32<0xB1>(v));
  v = max(v, dpp_u32<0x4E>(v));
  if (G == 8) v = max(v, dpp_u32<0x141>(v));
  return v;
}

struct QStrided {  // row r of a plain buffer
  const char* base;
  int64_t ld;
  int64_t rows;
  // in: input row, out: output row index; false: no such row
  __device__ bool at(int64_t r, const char*& in, int64_t& out) const {
    in = base + r * ld;
    out = r;
    return r < rows;
  }
};

struct QGather {  // row r = j * rcap + m of a wave
  MxGather g;
  int64_t row_bytes;
  __device__ bool at(int64_t r, const char*& in, int64_t& out) const {
    if (r >= (int64_t)g.nj * g.rcap) return false;
    const int j = (int)(r / g.rcap), m = (int)(r - (int64_t)j * g.rcap);
    if (m >= g.counts[j]) return false;
    out = r;
    if (g.ragged_rows > 0) {
      out = ragged_row0(g.counts, j) + m;
      if (out >= g.ragged_rows) return false;
    }
    if (g.wave_buf) {
      in = g.wave_buf + r * row_bytes;
    } else {
      const int rs = g.row_src[r];
      const int s = rs / g.cap;
      in = g.pools + s * g.src_stride + (int64_t)(rs - s * g.cap) * g.row_stride;
    }
    return true;
  }
};

constexpr int Q_UNROLL = 2;

// Launches f(first block, blocks) over `blocks` blocks of 256 threads, 2^23 at
// a time (a launch has fewer than 2^32 threads).
template <class F>
hipError_t in_launches(int64_t blocks, F f) {
  for (int64_t b = 0; b < blocks; b += 1 << 23) f(b, dim3((unsigned)(blocks - b < 1 << 23 ? blocks - b : 1 << 23)));
  return hipGetLastError();
}

// cpr: 16-byte pieces of an input row.  Block b (counted from block0) covers
// pieces b * 512 .., row after row.
template <class T, class Src>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(Src src, int64_t block0, int cpr, uint8_t* __restrict__ codes, int64_t ldc,
                   uint8_t* __restrict__ scales, int64_t lds) {
  constexpr int V = 16 / sizeof(T), G = MX_BLOCK / V;
  const int64_t first = (block0 + blockIdx.x) * (256 * Q_UNROLL);
  const int64_t row0 = first / cpr;
  const uint32_t off0 = (uint32_t)(first - row0 * cpr);
  uint4 d[Q_UNROLL];
  int64_t out[Q_UNROLL];
  uint32_t piece[Q_UNROLL];
  bool ok[Q_UNROLL];
#pragma unroll
  for (int u = 0; u < Q_UNROLL; ++u) {
    const uint32_t loc = off0 + threadIdx.x + 256 * u;
    const uint32_t r = loc / (uint32_t)cpr;
    piece[u] = loc - r * (uint32_t)cpr;
    const char* in = nullptr;
    ok[u] = src.at(row0 + r, in, out[u]);
    d[u] = make_uint4(0, 0, 0, 0);
    if (ok[u]) d[u] = *(const uint4*)(in + (int64_t)piece[u] * 16);
  }
#pragma unroll
  for (int u = 0; u < Q_UNROLL; ++u) {
    float v[V];
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      v[0] = __uint_as_float(d[u].x); v[1] = __uint_as_float(d[u].y);
      v[2] = __uint_as_float(d[u].z); v[3] = __uint_as_float(d[u].w);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = group_max<G>(m);  // rows start at a group boundary, so a group is one block
    const bool nan = (m >> 23) == 255;
    const int e = mx_exponent(m);
    const float inv = nan ? 0.f : mx_inverse_scale(e);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = nan ? 0.f : v[i] * inv;
    if (!ok[u]) continue;
    uint8_t* crow = codes + out[u] * ldc;
    if constexpr (sizeof(T) == 2)
      *(uint32_t*)(crow + (int64_t)piece[u] * 4) =
          mx_codes4(v[0], v[1], v[2], v[3]) | (mx_codes4(v[4], v[5], v[6], v[7]) << 16);
    else
      *(uint16_t*)(crow + (int64_t)piece[u] * 2) = (uint16_t)mx_codes4(v[0], v[1], v[2], v[3]);
    if (piece[u] % G == 0) {
      uint8_t* srow = scales + out[u] * lds;
      const int nb = cpr / G, b = (int)piece[u] / G;
      srow[b] = nan ? 255 : (uint8_t)(e + 127);
      if (b == nb - 1)
        for (int p = nb; p & 15; ++p) srow[p] = 0;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ldc, const uint8_t* __restrict__ scales, int64_t lds,
                     int64_t rows, int64_t block0, int cpr, char* __restrict__ outp, int64_t ldo) {
  constexpr int V = 16 / sizeof(T), G = MX_BLOCK / V;
  const int64_t first = (block0 + blockIdx.x) * (256 * Q_UNROLL);
  const int64_t row0 = first / cpr;
  const uint32_t off0 = (uint32_t)(first - row0 * cpr);
  uint32_t c[Q_UNROLL], s[Q_UNROLL], piece[Q_UNROLL];
  int64_t row[Q_UNROLL];
#pragma unroll
  for (int u = 0; u < Q_UNROLL; ++u) {
    const uint32_t loc = off0 + threadIdx.x + 256 * u;
    const uint32_t r = loc / (uint32_t)cpr;
    piece[u] = loc - r * (uint32_t)cpr;
    row[u] = row0 + r;
    c[u] = s[u] = 0;
    if (row[u] < rows) {
      const uint8_t* crow = codes + row[u] * ldc;
      c[u] = sizeof(T) == 2 ? *(const uint32_t*)(crow + (int64_t)piece[u] * 4)
                            : *(const uint16_t*)(crow + (int64_t)piece[u] * 2);
      s[u] = scales[row[u] * lds + piece[u] / G];
    }
  }
#pragma unroll
  for (int u = 0; u < Q_UNROLL; ++u) {
    if (row[u] >= rows) continue;
    const float sc = mx_scale(s[u]);
    float v[8];
    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 0);
    const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 1);
    const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 2);
    const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], 1.0f, 3);
    v[0] = p0[0] * sc; v[1] = p0[1] * sc; v[2] = p1[0] * sc; v[3] = p1[1] * sc;
    v[4] = p2[0] * sc; v[5] = p2[1] * sc; v[6] = p3[0] * sc; v[7] = p3[1] * sc;
    char* o = outp + row[u] * ldo + (int64_t)piece[u] * 16;
    if constexpr (sizeof(T) == 2)
      *(uint4*)o = make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                              f32x2_to_bf16x2(v[6], v[7]));
    else
      *(float4*)o = make_float4(v[0], v[1], v[2], v[3]);
  }
}

template <class T, class Src>
hipError_t run_quantize(const Src& src, int64_t rows, int64_t cols, uint8_t* codes, int64_t ldc, uint8_t* scales,
                        int64_t lds, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  const int64_t cpr = cols * sizeof(T) / 16, blocks = (rows * cpr + 256 * Q_UNROLL - 1) / (256 * Q_UNROLL);
  return in_launches(blocks, [&](int64_t b, dim3 grid) {
    launch((mx_quantize_kernel<T, Src>), grid, dim3(256), 0, st, src, b, (int)cpr, codes, ldc, scales, lds);
  });
}

hipError_t launch_mx_quantize(bool bf16, int64_t rows, int64_t cols, const void* x, int64_t ldx, uint8_t* codes,
                              int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t st) {
  const QStrided src{(const char*)x, ldx, rows};
  return bf16 ? run_quantize<bf16_t>(src, rows, cols, codes, ldc, scales, lds, st)
              : run_quantize<float>(src, rows, cols, codes, ldc, scales, lds, st);
}

hipError_t launch_mx_gather(bool bf16, const MxGather& g, int64_t cols, uint8_t* codes, uint8_t* scales,
                            hipStream_t st) {
  const int64_t rows = (int64_t)g.nj * g.rcap, ldc = cols / 2, lds = mx_scale_bytes(cols);
  const QGather src{g, cols * (bf16 ? 2 : 4)};
  return bf16 ? run_quantize<bf16_t>(src, rows, cols, codes, ldc, scales, lds, st)
              : run_quantize<float>(src, rows, cols, codes, ldc, scales, lds, st);
}

hipError_t launch_mx_dequantize(bool bf16, int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc,
                                const uint8_t* scales, int64_t lds, void* out, int64_t ldo, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  const int64_t cpr = cols * (bf16 ? 2 : 4) / 16, blocks = (rows * cpr + 256 * Q_UNROLL - 1) / (256 * Q_UNROLL);
  return in_launches(blocks, [&](int64_t b, dim3 grid) {
    if (bf16)
      launch(mx_dequantize_kernel<bf16_t>, grid, dim3(256), 0, st, codes, ldc, scales, lds, rows, b, (int)cpr, (char*)out, ldo);
    else
      launch(mx_dequantize_kernel<float>, grid, dim3(256), 0, st, codes, ldc, scales, lds, rows, b, (int)cpr, (char*)out, ldo);
  });
}

// ------------------------------------------------------------ product, rows by operand

struct MxARows {  // rows of group g: bank rows g * group_rows .., or end to end (ragged_rows > 0)
  MxView v;
  int64_t group_rows;
  const int32_t* counts;
  int max_rows;
  int64_t ragged_rows;
  __device__ int rows(int g) const { return counts ? min(max(counts[g], 0), max_rows) : max_rows; }
  __device__ int64_t index(int g, int m) const {
    if (ragged_rows > 0) {
      const int64_t r = ragged_row0(counts, g) + m;
      return r < ragged_rows ? r : ragged_rows - 1;
    }
    return g * group_rows + m;
  }
};

// Tile of workgroup `bid`: the tiles of the rows that exist, group by group and
// 4 tile rows at a time inside a group, in 8 contiguous ranges, one for each
// XCD (workgroups go round-robin to the XCDs), so that an XCD's L2 sees
// neighbouring tiles.  False: none is left.  Every workgroup goes through the
// groups' rows twice, one after the other: groups of 128 rows x 128 x 512 take
// 5.8 us for 8 of them and 14 for 64, but 74 for 384 and 5.3 ms for 4096.
template <int BM>
__device__ __forceinline__ bool mx_tile_of(const MxARows& a, int groups, int tiles_n, int bid, int& g, int& tm, int& tn) {
  int total = 0;
  for (int i = 0; i < groups; ++i) total += (a.rows(i) + BM - 1) / BM * tiles_n;
  const int xcd = bid & 7, idx = bid >> 3, per = total >> 3, rem = total & 7;
  if (idx >= per + (xcd < rem ? 1 : 0)) return false;
  int t = xcd * per + min(xcd, rem) + idx, mt = 0;
  for (g = 0; g < groups; ++g) {
    mt = (a.rows(g) + BM - 1) / BM;
    if (t < mt * tiles_n) break;
    t -= mt * tiles_n;
  }
  constexpr int GROUP_M = 4;
  const int gid = t / (GROUP_M * tiles_n), first = gid * GROUP_M, size = min(mt - first, GROUP_M);
  const int rest = t - gid * GROUP_M * tiles_n;
  tm = first + rest % size;
  tn = rest / size;
  return true;
}

struct MxBRows {
  MxView v;
  int n;
  __device__ int64_t index(int g, int i) const { return (int64_t)g * n + i; }
};

// Gate and up rows interleaved in blocks of 32 as in BGateUp: columns 64 b ..
// 64 b + 31 are the gate rows of hidden units 32 b .., the next 32 their up rows.
struct MxBGateUp {
  MxView v;
  int hidden;
  __device__ int64_t index(int g, int i) const {
    const int w = i & 63;
    return (int64_t)g * 2 * hidden + (int64_t)(w >> 5) * hidden + (i >> 6) * 32 + (w & 31);
  }
};

// Output rows of any alignment: 4 columns at a time where `vec` says that
// rows and columns stay aligned to 4 values, else one by one.
template <class T>
struct EMxOut {
  static constexpr bool STAGED = sizeof(T) == 2;
  char* out;
  int64_t ldo;  // bytes
  int64_t group_rows;
  bool vec, wide;  // rows aligned to 4 values; to 16 bytes with n a multiple of 8
  struct Row { T* p; };
  __device__ Row row(int g, int m) const { return {(T*)(out + (g * group_rows + m) * ldo)}; }
  __device__ int64_t row_key(int g, int m) const { return g * group_rows + m; }
  __device__ T* key_dst(int64_t key) const { return (T*)(out + key * ldo); }
  __device__ void store4(const Row& r, int n, int N, const float* v) const {
    if (vec && n + 4 <= N) {
      if constexpr (sizeof(T) == 2) *(uint2*)(r.p + n) = pack_bf16x4(v);
      else *(float4*)(r.p + n) = make_float4(v[0], v[1], v[2], v[3]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) r.p[n + i] = Act<T>::store(v[i]);
  }
};

__device__ __forceinline__ i32x8 mx_operand(i32x4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// ------------------------------------------------------------ product, few rows
//
// A workgroup of NW waves computes 16 columns (rows of B) for up to 16 * MT
// rows of A, straight from memory: the waves take K in pieces of 512 in turn
// and their sums meet in LDS.  v_mfma_scale_f32_16x16x128: a lane holds one
// block of one row (16 bytes of codes) and its scale byte.  The 16 scales of
// a 512-piece are one 16-byte load, whose dword j holds the scales of MFMA j.
// The last piece may end early: codes past the row are read from its last
// block, and their scales are 0 on both sides (2^-254: nothing in fp32).
// One row x 6144 x 2048 takes 4.4 us, one row x 4096 x 6144 4.8: the bytes are
// 1.4 and 2.8 us, the rest is one launch and one trip to memory and back.  More
// rows: 16 x 4096 x 6144 5.9 us, 32 7.6, 48 9.6, 64 10.8 (the bytes 2.9 us).
// Each workgroup reads all rows of A for its 16 columns, 1.6 us for each 16 rows
// of A (64 rows: 209 KB a workgroup, 53 MB in all out of the L2s).
template <int MT, int NW, class T>
__global__ void __launch_bounds__(NW * 64)
mx_gemm_rows(MxARows a, MxBRows b, EMxOut<T> e, int N, int K) {
  const int g = blockIdx.y, M = a.rows(g), n0 = blockIdx.x * 16;
  if (M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r16 = lane & 15, grp = lane >> 4;
  const int nb = K / MX_BLOCK, pieces = (nb + 15) / 16;
  const int64_t br = b.index(g, min(n0 + r16, N - 1));
  const uint8_t* bc = b.v.codes + br * b.v.ldc;
  const uint8_t* bs = b.v.scales + br * b.v.lds;
  const uint8_t *ac[MT], *as[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t ar = a.index(g, min(t * 16 + r16, M - 1));
    ac[t] = a.v.codes + ar * a.v.ldc;
    as[t] = a.v.scales + ar * a.v.lds;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p = wave; p < pieces; p += NW) {
    int64_t off[4];
    uint32_t keep[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int blk = p * 16 + j * 4 + grp;
      off[j] = (int64_t)min(blk, nb - 1) * 16;
      keep[j] = blk < nb ? 0xffu : 0u;
    }
    i32x4 bv[4], av[MT][4];
    const i32x4 bsc = *(const i32x4*)(bs + p * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) bv[j] = *(const i32x4*)(bc + off[j]);
    i32x4 asc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      asc[t] = *(const i32x4*)(as[t] + p * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) av[t][j] = *(const i32x4*)(ac[t] + off[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int sb = (int)(((uint32_t)bsc[j] >> (8 * grp)) & keep[j]);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int sa = (int)(((uint32_t)asc[t][j] >> (8 * grp)) & keep[j]);
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(bv[j]), mx_operand(av[t][j]), acc[t], 4, 4,
                                                                   0, sb, 0, sa);
      }
    }
  }
  // lane: row 16 t + lane % 16, columns n0 + 4 (lane / 16) ..
  __shared__ f32x4 part[NW][MT][64];
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  if (wave < MT) {
    const int t = wave;
    f32x4 s = part[0][t][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += part[w][t][lane];
    const int m = t * 16 + r16, n = n0 + grp * 4;
    if (m < M && n < N) {
      const float v[4] = {s[0], s[1], s[2], s[3]};
      e.store4(e.row(g, m), n, N, v);
    }
  }
}

// ------------------------------------------------------------ product, many rows
//
// The layout of the bf16 core (gemm.h) carries over byte for byte: a
// workgroup of 8 waves (2 x 4) per 256 x 256 tile, two LDS buffers of 128-byte
// row pieces (256 values here) with the same chunk swizzle, one 16-byte chunk
// a lane and fragment: v_mfma_scale_f32_32x32x64_f8f6f4 takes a block of 32
// values of one row from each lane, four times the bf16 instruction's work for
// the same LDS bytes and the same 32 cycles.  Lane (row, half) of fragment step
// ks holds block 2 ks + half of the step's eight.
//
// Scales: a row's 16 scale bytes of two K steps are one 16-byte piece, so one
// more global->LDS load a thread every second step brings in those of all
// rows (two buffers).  A lane reads the 4 bytes of a row and half a step,
// shifts its half's bytes down once, and the MFMA picks byte 0 or 2.
//
// A last step that reaches past K reads the row's last block again in the
// place of what is missing, and clears the scales of those blocks on both
// sides: 2^-254 times at most 36 adds nothing to an fp32 sum.
//
// A tile of 128 x 128 by 4 waves (2 x 2, 64 x 64 each) has the same layout;
// two such workgroups share a CU.
//
// MI355X: 8192 x 6144 x 6144 in 160 us, 3.86 PFLOP/s (2.8 times the rate of a
// large bf16 library product on the card), the matrix units busy half of the
// cycles.  The same MFMAs with nothing else in the loop take 0.72 of the time, at
// a clock the power limit sets; half of the other 0.28 is the loads, half the LDS
// reads.  Slower here: 4 waves of 128 x 128 (two thirds of the LDS reads,
// but one wave a SIMD has nothing to hide its address arithmetic behind), and a
// ring of four 64-byte-deep buffers with counted waits (187 us against 166).
template <int B_>
struct MxTile {
  static_assert(B_ == 256 || B_ == 128, "a wave loads 32 rows of each operand");
  static constexpr int BM = B_, BN = B_, NW = B_ / 32, NT = NW * 64;
  static constexpr int WN = NW / 2, WTM = BM / 2, WTN = 64;  // waves along n; a wave's part of the tile
  static constexpr int FM = WTM / 32, FN = 2, NF = FM + FN;
  static constexpr int ROW = 128, STAGE = (BM + BN) * ROW;  // bytes of an LDS row and of one buffer
  static constexpr int RPW = 32, WBYTES = RPW * ROW;        // rows of each operand that one wave loads
  static constexpr int SCALES = (BM + BN) * 16;             // bytes of one scale buffer
  static constexpr int STEP = 8;                            // 32-value blocks of one K step
};

template <int FM>
struct MxFrags {
  i32x4 a[FM], b[2];
};

__device__ __forceinline__ void mx_read16(i32x4& v, uint32_t addr) {
  asm volatile("ds_read_b128 %0, %1" : "=v"(v) : "v"(addr) : "memory");
}
__device__ __forceinline__ void mx_read4(int& v, uint32_t addr) {
  asm volatile("ds_read_b32 %0, %1" : "=v"(v) : "v"(addr) : "memory");
}
// Every LDS read so far has landed; the registers pass through, so that their
// consumers stay behind it.
__device__ __forceinline__ void mx_wait(MxFrags<4>& f) {
  asm volatile("s_waitcnt lgkmcnt(0)"
               : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.b[0]), "+v"(f.b[1])::"memory");
}
__device__ __forceinline__ void mx_wait(MxFrags<4>& f, int (&s)[6]) {
  asm volatile("s_waitcnt lgkmcnt(0)"
               : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.b[0]), "+v"(f.b[1]), "+v"(s[0]),
                 "+v"(s[1]), "+v"(s[2]), "+v"(s[3]), "+v"(s[4]), "+v"(s[5])::"memory");
}
__device__ __forceinline__ void mx_wait(MxFrags<2>& f) {
  asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.b[0]), "+v"(f.b[1])::"memory");
}
__device__ __forceinline__ void mx_wait(MxFrags<2>& f, int (&s)[4]) {
  asm volatile("s_waitcnt lgkmcnt(0)"
               : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.b[0]), "+v"(f.b[1]), "+v"(s[0]), "+v"(s[1]), "+v"(s[2]), "+v"(s[3])
               ::"memory");
}

// A bf16 tile by way of LDS (free of operands by now), whole row pieces at a
// time: the accumulators' own stores would write 8 bytes (2 where a row is not
// aligned) of 32 different rows each.  16-byte chunks are swizzled by row.
template <class C, class E>
__device__ __forceinline__ void mx_staged(const E& e, int m0, int n0, int M, int N, char* smem, const int64_t* keys,
                                          const f32x16 (&acc)[C::FM][C::FN]) {
  constexpr int RB = C::BN * 2, CH = RB / 16;
  static_assert(C::BM * RB <= 2 * C::STAGE, "the staged tile fits the operand buffers");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WN, wn = wave % C::WN, frow = lane & 31, half = lane >> 5;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row = wm * C::WTM + i * 32 + frow;
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int byte = (wn * C::WTN + j * 32 + q * 8 + half * 4) * 2;
        const float v[4] = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
        *(uint2*)(smem + row * RB + (((byte >> 4) ^ (row & (CH - 1))) << 4) + (byte & 15)) = pack_bf16x4(v);
      }
  }
  __syncthreads();
  if (e.wide) {
    constexpr int RPI = 64 / CH;  // rows a store instruction covers
    const int c = lane % CH;
#pragma unroll 4
    for (int it = 0; it < C::RPW / RPI; ++it) {
      const int row = wave * C::RPW + it * RPI + lane / CH;
      if (m0 + row < M && n0 + c * 8 < N)
        *(uint4*)(e.key_dst(keys[row]) + n0 + c * 8) = *(const uint4*)(smem + row * RB + ((c ^ (row & (CH - 1))) << 4));
    }
  } else {
    // 4-byte stores from a row's first 4-byte boundary on were slower (6 x 942 x
    // 2815 x 2080: 52 us, 49 here): partial cache lines cost this, not the stores
    constexpr int R = 8, X = C::BN / 64;  // rows in flight, 64-column pieces of a row
    for (int r0 = 0; r0 < C::RPW; r0 += R) {
      bf16_t v[R][X];
      int64_t key[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = wave * C::RPW + r0 + r;
        key[r] = keys[row];
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const int col = x * 64 + lane;
          v[r][x] = *(const bf16_t*)(smem + row * RB + (((col >> 3) ^ (row & (CH - 1))) << 4) + (col & 7) * 2);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (m0 + wave * C::RPW + r0 + r >= M) return;
        bf16_t* dst = e.key_dst(key[r]) + n0;
#pragma unroll
        for (int x = 0; x < X; ++x)
          if (n0 + x * 64 + lane < N) dst[x * 64 + lane] = v[r][x];
      }
    }
  }
}

// Hidden rows out of a gate / up tile: 64 columns of a wave are the 32 gate and
// the 32 up columns of one block of hidden units, 16 of them in this lane and
// 16 in lane ^ 32, so silu(gate) * up is quantised where it is: one exchange
// for the block's maximum and one that pairs the halves' codes.
struct EMxHidden {
  static constexpr bool STAGED = false;
  MxView h;
  int64_t group_rows;
  const int32_t* counts;
  int64_t ragged_rows;  // as MxARows; a row past the bank is not stored
  __device__ void store(int g, int m, int M, int block, bool in, int half, const f32x16& gate, const f32x16& up) const {
    float v[16];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = silu(gate[i]) * up[i];
      top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    const bool nan = (top >> 23) == 255;
    const int ex = mx_exponent(top);
    const float inv = mx_inverse_scale(nan ? 0 : ex);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = nan ? 0.f : v[i] * inv;
    // units 8 q + 4 half + 0..3 are 16 bits of dword q of the block's codes
    const uint32_t lo = mx_codes4(v[0], v[1], v[2], v[3]) | (mx_codes4(v[4], v[5], v[6], v[7]) << 16);
    const uint32_t hi = mx_codes4(v[8], v[9], v[10], v[11]) | (mx_codes4(v[12], v[13], v[14], v[15]) << 16);
    const uint32_t olo = (uint32_t)__shfl_xor((int)lo, 32), ohi = (uint32_t)__shfl_xor((int)hi, 32);
    const uint2 d = half ? make_uint2((ohi & 0xffffu) | (hi << 16), (ohi >> 16) | (hi & 0xffff0000u))
                         : make_uint2((lo & 0xffffu) | (olo << 16), (lo >> 16) | (olo & 0xffff0000u));
    if (m >= M || !in) return;
    const int64_t r = ragged_rows > 0 ? ragged_row0(counts, g) + m : g * group_rows + m;
    if (ragged_rows > 0 && r >= ragged_rows) return;
    *(uint2*)(const_cast<uint8_t*>(h.codes) + r * h.ldc + block * 16 + half * 8) = d;
    if (!half) const_cast<uint8_t*>(h.scales)[r * h.lds + block] = nan ? 255 : (uint8_t)(ex + 127);
  }
};

// grid: gemm_grid of the tiles; block: C::NT.
template <class C, bool GATEUP, class B, class E>
__global__ void __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2, 2)))
mx_gemm_tile(MxARows a, B b, E e, int N, int K, int groups, int tiles_n) {
  constexpr int FM = C::FM, FN = C::FN, NF = C::NF, NMMA = FM * FN;
  __shared__ __attribute__((aligned(1024))) char smem[2 * C::STAGE + 2 * C::SCALES];
  const int nch = K / MX_BLOCK, nk = (nch + C::STEP - 1) / C::STEP;
  int g, tm, tn;
  if (!mx_tile_of<C::BM>(a, groups, tiles_n, blockIdx.x, g, tm, tn)) return;
  const int M = a.rows(g);
  const int m0 = tm * C::BM, n0 = tn * C::BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WN, wn = wave % C::WN;
  __shared__ int64_t keys[E::STAGED ? C::BM : 1];
  if constexpr (E::STAGED)  // where the tile's rows go, looked up while the first loads are under way
    if (tid < C::BM && m0 + tid < M) keys[tid] = e.row_key(g, m0 + tid);

  // codes: load d of a wave brings in rows 32 wave + 8 d + lane / 8; its
  // immediate offset moves both addresses by 1024 d, taken off the row pointer
  const int lrow = lane >> 3, lcol = lane & 7;
  const int gcol = lcol ^ swz(wave * C::RPW + lrow);  // rows 8 further: ^ 4
  const uint8_t *pa[4], *pb[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int row = wave * C::RPW + d * 8 + lrow;
    pa[d] = a.v.codes + a.index(g, min(m0 + row, M - 1)) * a.v.ldc - 1024 * d;
    pb[d] = b.v.codes + b.index(g, min(n0 + row, N - 1)) * b.v.ldc - 1024 * d;
  }
  // scales: thread tid brings in row tid of A (below BM) or of B
  const uint8_t* ps = tid < C::BM ? a.v.scales + a.index(g, min(m0 + tid, M - 1)) * a.v.lds
                                  : b.v.scales + b.index(g, min(n0 + tid - C::BM, N - 1)) * b.v.lds;

  const int frow = lane & 31, half = lane >> 5, fswz = swz(frow);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  const uint32_t fa_base = lds0 + (wm * C::WTM + frow) * C::ROW, fb_base = lds0 + (C::BM + wn * C::WTN + frow) * C::ROW;
  const uint32_t sa_base = lds0 + 2 * C::STAGE + (wm * C::WTM + frow) * 16;
  const uint32_t sb_base = lds0 + 2 * C::STAGE + (C::BM + wn * C::WTN + frow) * 16;

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  MxFrags<FM> F[2];
  int sc[2][NF];  // the scale bytes of substeps 2 w and 2 w + 1 (bytes 0 and 2)
  auto read_codes = [&](MxFrags<FM>& f, int kt, int ks, int q) {
    const uint32_t st = (uint32_t)((kt & 1) * C::STAGE) + (uint32_t)(((ks * 2 + half) ^ fswz) << 4);
    if (q < FM) mx_read16(f.a[q], fa_base + st + q * 32 * C::ROW);
    else mx_read16(f.b[q - FM], fb_base + st + (q - FM) * 32 * C::ROW);
  };
  auto read_scales = [&](int kt, int w, int q) {  // blocks 4 w .. 4 w + 3 of step kt
    const uint32_t st = (uint32_t)(((kt >> 1) & 1) * C::SCALES + (kt & 1) * 8 + w * 4);
    if (q < FM) mx_read4(sc[w][q], sa_base + st + q * 32 * 16);
    else mx_read4(sc[w][q], sb_base + st + (q - FM) * 32 * 16);
  };
  auto load_codes = [&](int kt, int d) {  // d in [0, 8)
    const int dd = d & 3;
    const void* gp = (const void*)((d < 4 ? pa[dd] : pb[dd]) + min(kt * C::STEP + (gcol ^ (dd & 1) * 4), nch - 1) * 16);
    auto lp = (__attribute__((address_space(3))) void*)(smem + (kt & 1) * C::STAGE + (d < 4 ? 0 : C::BM * C::ROW) +
                                                         wave * C::WBYTES);
    switch (dd) {
      case 0: __builtin_amdgcn_global_load_lds(gp, lp, 16, 0, 0); break;
      case 1: __builtin_amdgcn_global_load_lds(gp, lp, 16, 1024, 0); break;
      case 2: __builtin_amdgcn_global_load_lds(gp, lp, 16, 2048, 0); break;
      default: __builtin_amdgcn_global_load_lds(gp, lp, 16, 3 * 1024, 0); break;
    }
  };
  auto load_scales = [&](int pair) {  // steps 2 pair and 2 pair + 1
    auto lp = (__attribute__((address_space(3))) void*)(smem + 2 * C::STAGE + (pair & 1) * C::SCALES + wave * 1024);
    __builtin_amdgcn_global_load_lds((const void*)(ps + (int64_t)pair * 16), lp, 16, 0, 0);
  };
  // Scale dwords are read one half step ahead, where their registers are
  // free: those of substeps 0 and 1 in the last substep of the step before,
  // those of 2 and 3 in the first of their own.
  auto shift_scales = [&](int w, uint32_t keep) {
#pragma unroll
    for (int q = 0; q < NF; ++q) sc[w][q] = (int)(((uint32_t)sc[w][q] >> (8 * half)) & keep);
  };
  // MODE 0: issues the loads of step kt + 2; 1: no new loads; 2: the last
  // step.  HALF: loads 4..7 of step kt + 1 were left to this step's start.
  auto substep = [&](int kt, auto ks_tag, auto mode_tag, auto half_tag) {
    constexpr int ks = decltype(ks_tag)::value, MODE = decltype(mode_tag)::value;
    constexpr bool HALF = decltype(half_tag)::value;
    constexpr int SEL = (ks & 1) * 2;
    MxFrags<FM>& cur = F[ks & 1];
    MxFrags<FM>& nxt = F[(ks + 1) & 1];
    if constexpr (ks == 3 && MODE != 2) {
      vm_wait<0>();   // step kt + 1's codes and scales (this lane's part)
      lds_barrier();  // ... every lane's; every wave is done with step kt's buffers
    }
#pragma unroll
    for (int q = 0; q < NMMA; ++q) {
      const int j = q / FM, i = q % FM;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(cur.b[j]), mx_operand(cur.a[i]), acc[i][j],
                                                                  4, 4, SEL, sc[ks >> 1][FM + j], SEL, sc[ks >> 1][i]);
      if constexpr (ks < 3) {
        if (q < NF) read_codes(nxt, kt, ks + 1, q);
        if (ks == 0) {
          if (q < NF) read_scales(kt, 1, q);
          if (HALF && q < 4) load_codes(kt + 1, 4 + q);
          // the scales of the next pair of steps, into the buffer that step kt - 1 was the last to use
          if (q == NMMA - 1 && MODE == 0 && !(kt & 1)) load_scales(kt / 2 + 1);
        }
      } else if constexpr (MODE != 2) {
        if (q < NF) {
          read_codes(nxt, kt + 1, 0, q);
          read_scales(kt + 1, 0, q);
        }
        if (MODE == 0 && q < 4) load_codes(kt + 2, q);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (ks == 0) mx_wait(nxt, sc[1]);
    else if constexpr (ks < 3) mx_wait(nxt);
    else if constexpr (MODE != 2) mx_wait(nxt, sc[0]);
  };
  auto step = [&](int kt, auto mode_tag, auto half_tag) {
    uint32_t keep[2] = {~0u, ~0u};
    if constexpr (decltype(mode_tag)::value == 2) {  // blocks of this step that K still has
      const int have = nch - kt * C::STEP - half;
      keep[0] = (have > 0 ? 0xffu : 0u) | (have > 2 ? 0xff0000u : 0u);
      keep[1] = (have > 4 ? 0xffu : 0u) | (have > 6 ? 0xff0000u : 0u);
    }
    shift_scales(0, keep[0]);
    substep(kt, std::integral_constant<int, 0>(), mode_tag, half_tag);
    shift_scales(1, keep[1]);
    substep(kt, std::integral_constant<int, 1>(), mode_tag, half_tag);
    substep(kt, std::integral_constant<int, 2>(), mode_tag, half_tag);
    substep(kt, std::integral_constant<int, 3>(), mode_tag, half_tag);
  };
  using Loads = std::integral_constant<int, 0>;
  using NoLoads = std::integral_constant<int, 1>;
  using Last = std::integral_constant<int, 2>;
  load_scales(0);
#pragma unroll
  for (int d = 0; d < 8; ++d) load_codes(0, d);
  vm_wait<0>();
  lds_barrier();
  if (nk > 1) {
#pragma unroll
    for (int d = 0; d < 8; ++d) load_codes(1, d);
  }
#pragma unroll
  for (int q = 0; q < NF; ++q) {
    read_codes(F[0], 0, 0, q);
    read_scales(0, 0, q);
  }
  mx_wait(F[0], sc[0]);
  if (nk >= 3) {
    step(0, Loads(), std::false_type());
    for (int kt = 1; kt + 2 < nk; ++kt) step(kt, Loads(), std::true_type());
    step(nk - 2, NoLoads(), std::true_type());
    step(nk - 1, Last(), std::false_type());
  } else if (nk == 2) {
    step(0, NoLoads(), std::false_type());
    step(1, Last(), std::false_type());
  } else {
    step(0, Last(), std::false_type());
  }

  if constexpr (GATEUP) {
#pragma unroll
    for (int j = 0; j < FN; j += 2) {
      const int n = n0 + wn * C::WTN + j * 32;
#pragma unroll
      for (int i = 0; i < FM; ++i)
        e.store(g, m0 + wm * C::WTM + i * 32 + frow, M, n >> 6, n < N, half, acc[i][j], acc[i][j + 1]);
    }
  } else {
    if constexpr (E::STAGED) {
      mx_staged<C>(e, m0, n0, M, N, smem, keys, acc);
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i)
        epilogue_row<false, FN>(e, g, m0 + wm * C::WTM + i * 32 + frow, M, n0 + wn * C::WTN, N, half, acc[i]);
    }
  }
}

template <class C, bool GATEUP, class B, class E>
hipError_t run_mx_tiles(const MxARows& a, const B& b, const E& e, int N, int K, int groups, hipStream_t st) {
  const int64_t tiles_n = (N + C::BN - 1) / C::BN, tiles = groups * (((int64_t)a.max_rows + C::BM - 1) / C::BM) * tiles_n;
  if (tiles <= 0) return hipSuccess;
  launch((mx_gemm_tile<C, GATEUP, B, E>), dim3((unsigned)(8 * ((tiles + 7) / 8))), dim3(C::NT), 0, st, a, b, e, N, K,
         groups, (int)tiles_n);
  return hipGetLastError();
}

// Rounds of the card's CUs that the tiles take: one workgroup of 256 x 256 a
// CU, or two of 128 x 128, which together take MX_SMALL_ROUND of a large
// tile's time for half of its work.  Measured, large and small tiles:
// 1024 x 4096 x 4096 26 and 17 us, 2048 x 4096 x 4096 29 and 24,
// 4096 x 4096 x 4096 40 and 47, 8192 x 6144 x 6144 167 and 210; with rows of 512
// values 10.0 and 7.5, 11.7 and 10.5, 14.5 and 15.2 us (8192 x 6144: 34 and 36).
// 3000 x 3100 x 512, 2048 and 6144: 15.6 and 17.3, 23.9 and 27.1, 45 and 57.
// The rows are max_rows, as the launch does not know the counts.
constexpr double MX_SMALL_ROUND = 0.65;

template <bool GATEUP, class B, class E>
hipError_t run_mx_tile(const MxARows& a, const B& b, const E& e, int N, int K, int groups, int cus, hipStream_t st) {
  auto rounds = [&](int64_t tile, int64_t at_once) {
    const int64_t tiles = groups * ((a.max_rows + tile - 1) / tile) * ((N + tile - 1) / tile);
    return (double)((tiles + at_once - 1) / at_once);
  };
  if (rounds(128, 2 * cus) * MX_SMALL_ROUND < rounds(256, cus))
    return run_mx_tiles<MxTile<128>, GATEUP>(a, b, e, N, K, groups, st);
  return run_mx_tiles<MxTile<256>, GATEUP>(a, b, e, N, K, groups, st);
}

template <class T>
hipError_t run_mx_gemm(const MxGemmArgs& q, int cus, hipStream_t st) {
  const MxARows a{q.a, q.max_rows, q.counts, q.max_rows, 0};
  const MxBRows b{q.b, q.n};
  const uintptr_t at = (uintptr_t)q.out | (uintptr_t)q.ldo;
  const EMxOut<T> e{(char*)q.out, q.ldo, q.max_rows, at % (4 * sizeof(T)) == 0, at % 16 == 0 && q.n % 8 == 0};
  // up to 64 rows: 11 us for 64 x 4096 x 6144, where one row of 128-tiles takes 18
  if (q.max_rows > 64) return run_mx_tile<false>(a, b, e, q.n, q.k, q.groups, cus, st);
  // one wave for each 512-piece of K, as far as a workgroup goes
  const dim3 grid((unsigned)((q.n + 15) / 16), (unsigned)q.groups);
  const int pieces = (q.k + 511) / 512;
  auto rows = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    if (pieces <= 4) launch((mx_gemm_rows<MT, 4, T>), grid, dim3(256), 0, st, a, b, e, q.n, q.k);
    else if (pieces <= 8) launch((mx_gemm_rows<MT, 8, T>), grid, dim3(512), 0, st, a, b, e, q.n, q.k);
    else launch((mx_gemm_rows<MT, 16, T>), grid, dim3(1024), 0, st, a, b, e, q.n, q.k);
  };
  if (q.max_rows <= 16) rows(std::integral_constant<int, 1>());
  else if (q.max_rows <= 32) rows(std::integral_constant<int, 2>());
  else rows(std::integral_constant<int, 4>());
  return hipGetLastError();
}

hipError_t launch_mx_gemm(const MxGemmArgs& g, int cus, hipStream_t st) {
  return g.bf16 ? run_mx_gemm<bf16_t>(g, cus, st) : run_mx_gemm<float>(g, cus, st);
}

hipError_t launch_mx_gate_up(const MxExpertArgs& g, int cus, hipStream_t st) {
  const MxARows a{g.x, g.rcap, g.counts, g.rcap, g.ragged_rows};
  const MxBGateUp b{g.w13, g.H};
  const EMxHidden e{g.h, g.rcap, g.counts, g.ragged_rows};
  return run_mx_tile<true>(a, b, e, 2 * g.H, g.L, g.nj, cus, st);
}

template <class T>
struct EMxReturn : EScatter<T> {
  static constexpr bool STAGED = sizeof(T) == 2;  // the staged copy of a tile is bf16
  static constexpr bool wide = true;              // latent is a multiple of 64 in bf16 layers
};

template <class T>
hipError_t run_mx_down(const MxExpertArgs& g, int cus, hipStream_t st) {
  const MxARows a{g.h, g.rcap, g.counts, g.rcap, g.ragged_rows};
  const MxBRows b{g.w2, g.L};
  const EMxReturn<T> e{{g.ret, g.ret_src_stride, g.row_bytes, g.cap, g.row_src, g.rcap}};
  return run_mx_tile<false>(a, b, e, g.L, g.H, g.nj, cus, st);
}

hipError_t launch_mx_down(const MxExpertArgs& g, int cus, hipStream_t st) {
  return g.bf16 ? run_mx_down<bf16_t>(g, cus, st) : run_mx_down<float>(g, cus, st);
}

}  // namespace moe
