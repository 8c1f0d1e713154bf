// Grouped product of MX-FP8 rows with MX-FP4 rows (gfx950): out[g] = A[g] . B[g]^T.
//
// The products run on v_mfma_scale_f32_{32x32x64,16x16x128}_f8f6f4 with an FP4
// and an FP8 operand.  Layout of an FP8 operand of 64 (128) values a row: the
// lane of half h (quarter q) holds values 16 h .. and 32 + 16 h .. (16 q .. and
// 64 + 16 q ..), its FP4 counterpart the block 32 h .. (32 q ..), and both the
// scale of block h (q).
//
// What the instruction keeps: it adds eight products at a time, each cut off
// 13 bits below the largest of the eight (found with single products of known
// size; FP4 by FP4 never gets there).  That is 1e-4 of a bf16 output's RMS, a
// twentieth of its rounding, and is taken there.  An fp32 output takes A in two
// parts that add up to it, the codes of 8 and more (of at most 448) and the
// rest, each with a product of its own: the first part's products, multiples
// of 1/2 up to 2688, fit 13 bits, so that nothing of them is cut off, and what
// is cut off of the others is below 2^-13 of 6 * 7.5, 2^-19 of a block's
// largest product.

#include "block.h"

#include <algorithm>
#include <cmath>

namespace moe {

namespace {

struct Operand {  // rows of all groups, group by group
  MxView v;
  int64_t per_group;
};

__device__ __forceinline__ int group_rows(const int32_t* counts, int g, int max_rows) {
  return counts ? min(max(counts[g], 0), max_rows) : max_rows;
}

// Output rows of any alignment, 4 columns at a time.
template <class T>
struct Out {
  char* p;
  int64_t ld;  // bytes
  __device__ T* row(int64_t r) const { return (T*)(p + r * ld); }
  __device__ void store4(T* r, int n, int N, const float (&v)[4]) const {
    if (n + 4 <= N) {
      if constexpr (sizeof(T) == 2)
        *(i32x2_any*)(r + n) = i32x2_any{(int)f32x2_to_bf16x2(v[0], v[1]), (int)f32x2_to_bf16x2(v[2], v[3])};
      else
        *(i32x4_any*)(r + n) = i32x4_any{__float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3])};
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) r[n + i] = Act<T>::store(v[i]);
  }
};

__device__ __forceinline__ i32x8 fp4_operand(i32x4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }
__device__ __forceinline__ i32x8 fp8_operand(i32x4 lo, i32x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The codes of 8 and more in magnitude (exponent field 10 and up), the others 0.
__device__ __forceinline__ int fp8_large(int c) {
  const uint32_t x = (uint32_t)c;
  const uint32_t m = (x & ((x << 1) | (x << 2))) & 0x40404040u;  // field >= 10: its top bit and one of the next two
  return (int)(x & ((m << 2) - (m >> 6)));                       // a byte 0xff where m has 0x40
}
__device__ __forceinline__ i32x8 fp8_large(i32x8 v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fp8_large(v[i]);
  return v;
}

// ------------------------------------------------------------ few rows
//
// A workgroup of NW waves computes 16 columns (rows of B) for up to 16 MT rows
// of A straight from memory: the waves take K in pieces of 512 in turn and
// their sums meet in LDS.  The 16 scales of a piece are one 16-byte load, whose
// dword j holds those of MFMA j.  The last piece may end early: codes past the
// row are read from its last chunk, and their scales are 0 on both sides
// (2^-254: nothing in fp32).  1, 16, 32 and 64 rows x 4096 x 6144 5.2, 7.3, 10.2 and
// 16 us (the bytes 2.8 to 3).  The compiler moves a piece's loads down between its
// matrix instructions, which makes about three trips to memory of it with 16 rows,
// eight with 32 and more with 64; and every workgroup reads all rows of A for its
// 16 columns.
template <int MT, int NW, class T>
__global__ void __launch_bounds__(NW * 64)
mx8_gemm_rows(Operand a, Operand b, Out<T> out, const int32_t* counts, int max_rows, int N, int K) {
  constexpr bool SPLIT = sizeof(T) == 4;
  const int g = blockIdx.y, M = group_rows(counts, g, max_rows), n0 = blockIdx.x * 16;
  if (M <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r16 = lane & 15, grp = lane >> 4;
  const int nb = K / MX_BLOCK, nc = K / 16, pieces = (nb + 15) / 16;
  const int64_t br = g * b.per_group + min(n0 + r16, N - 1);
  const uint8_t* bc = b.v.codes + br * b.v.ldc;
  const uint8_t* bs = b.v.scales + br * b.v.lds;
  const uint8_t *ac[MT], *as[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t ar = g * a.per_group + min(t * 16 + r16, M - 1);
    ac[t] = a.v.codes + ar * a.v.ldc;
    as[t] = a.v.scales + ar * a.v.lds;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p = wave; p < pieces; p += NW) {
    i32x4 bv[4], av[MT][4][2], asc[MT];
    const i32x4 bsc = *(const i32x4*)(bs + p * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) bv[j] = *(const i32x4*)(bc + (int64_t)min(p * 16 + j * 4 + grp, nb - 1) * 16);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      asc[t] = *(const i32x4*)(as[t] + p * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          av[t][j][i] = *(const i32x4*)(ac[t] + (int64_t)min(p * 32 + j * 8 + i * 4 + grp, nc - 1) * 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t keep = p * 16 + j * 4 + grp < nb ? 0xffu : 0u;
      const int sb = (int)(((uint32_t)bsc[j] >> (8 * grp)) & keep);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int sa = (int)(((uint32_t)asc[t][j] >> (8 * grp)) & keep);
        i32x8 v = fp8_operand(av[t][j][0], av[t][j][1]);
        if constexpr (SPLIT) {
          const i32x8 large = fp8_large(v);
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(bv[j]), large, acc[t], 4, 0, 0, sb, 0, sa);
          v ^= large;
        }
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(bv[j]), v, acc[t], 4, 0, 0, sb, 0, sa);
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
      out.store4(out.row(g * a.per_group + m), n, N, v);
    }
  }
}

// ------------------------------------------------------------ many rows
//
// A workgroup of 8 waves (2 x 4) per 256 x 256 tile, or of 4 (2 x 2) per 128 x
// 128, and steps of 128 values along K: 128-byte row pieces of A, and of B
// 64-byte ones, two rows to a 128-byte line, both in 16-byte chunks swizzled by
// line so that LDS reads have no bank conflicts.  Three buffers.  A step is two
// substeps of 64 values; each reads the fragments of the next from LDS between
// its matrix instructions.  The second waits for the loads of the next step
// (those of the one after stay under way), passes the barrier (after which
// every wave is done with the step's buffer), and issues those of the step
// three further into that buffer.
//
// Scales: a row's 16 scale bytes of four steps are one 16-byte piece, so one
// more global->LDS load a thread every fourth step brings in those of all rows
// (two buffers).  A lane reads the 4 bytes of a row and step, shifts its half's
// byte down, and the MFMA of substep s picks byte 2 s.
//
// A last step that reaches past K reads the row's last chunk again in the
// place of what is missing, and clears the scales of those blocks on both
// sides: 2^-254 adds nothing to an fp32 sum, and a NaN there is a NaN of the row.
//
// MI355X: 8192 x 6144 x 6144 to bf16 219-233 us, 2.7-2.8 PFLOP/s (2.1 times the
// rate of a large bf16 library product on the card), the matrix units busy 72 %
// of the cycles at the 1.9 GHz that the power limit leaves (tens of calls without a
// pause bring the clock further down: up to 290 us); to fp32, with twice the matrix
// instructions and tiles of 128 x 128 (the parts of A take registers), 505-534.
// Slower here, beside 219: two buffers instead of three with addresses worked out anew at
// each read (236), 4 scale bytes a row loaded with every step, which leaves no
// bank conflicts but has 64 lanes read 64 lines (250).
template <int B_>
struct Tile {
  static_assert(B_ == 256 || B_ == 128, "a wave loads 32 rows of each operand");
  static constexpr int BM = B_, BN = B_, NW = B_ / 32, NT = NW * 64;
  static constexpr int WN = NW / 2, WTM = BM / 2, WTN = 64;
  static constexpr int FM = WTM / 32, FN = 2, NF = FM + FN;
  static constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + BN * 64;
  static constexpr int SCALES = (BM + BN) * 16;
  static constexpr int STAGES = 3, OPERANDS = STAGES * STAGE + 2 * SCALES, STAGED = BM * BN * 2;
};

template <int FM>
struct Frags {
  i32x8 a[FM];
  i32x4 b[2];
};

template <int OFFSET>
__device__ __forceinline__ void read16(i32x4& v, uint32_t addr) {
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFFSET) : "memory");
}
template <int OFFSET>
__device__ __forceinline__ void read4(int& v, uint32_t addr) {
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFFSET) : "memory");
}
// f(0), f(1) .. f(N - 1) with each index a constant.
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>());
  }
}
// Every LDS read so far has landed; the registers pass through, so that their
// consumers stay behind it.
__device__ __forceinline__ void wait_reads(Frags<4>& f) {
  asm volatile("s_waitcnt lgkmcnt(0)"
               : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.b[0]), "+v"(f.b[1])::"memory");
}
__device__ __forceinline__ void wait_reads(Frags<2>& f) {
  asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.b[0]), "+v"(f.b[1])::"memory");
}
__device__ __forceinline__ void wait_reads(Frags<4>& f, int (&s)[6]) {
  asm volatile("s_waitcnt lgkmcnt(0)"
               : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.a[2]), "+v"(f.a[3]), "+v"(f.b[0]), "+v"(f.b[1]), "+v"(s[0]), "+v"(s[1]),
                 "+v"(s[2]), "+v"(s[3]), "+v"(s[4]), "+v"(s[5])::"memory");
}
__device__ __forceinline__ void wait_reads(Frags<2>& f, int (&s)[4]) {
  asm volatile("s_waitcnt lgkmcnt(0)"
               : "+v"(f.a[0]), "+v"(f.a[1]), "+v"(f.b[0]), "+v"(f.b[1]), "+v"(s[0]), "+v"(s[1]), "+v"(s[2]), "+v"(s[3])
               ::"memory");
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_prefix(int v) {
  const int lane = lane_id();
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const int x = __shfl_up(v, off);
    v += lane >= off ? x : 0;
  }
  return v;
}

// Tile of workgroup `bid`: the tiles of the rows that exist, group by group and
// 4 tile rows at a time inside a group, in 8 contiguous ranges, one for each
// XCD (workgroups go round-robin to the XCDs), so that an XCD's L2 sees
// neighbouring tiles.  The groups' tiles are added up by a wave, 64 groups at a
// time: groups of 128 rows x 128 x 512 take 6.5 us for 64 of them, 16 for 384,
// 490 for 4096 (counts looked at one after the other, as in ops/mx.hip: 14, 74, 5300).
// False: none is left.
template <int BM>
__device__ __forceinline__ bool tile_of(const int32_t* counts, int max_rows, int groups, int tiles_n, int bid, int& g, int& tm,
                                        int& tn) {
  const int lane = lane_id();
  auto tile_rows = [&](int i) { return i < groups ? (group_rows(counts, i, max_rows) + BM - 1) / BM : 0; };
  int total = 0, upto = 0;  // upto: of the first 64 groups, a lane's and those before it
  for (int first = 0; first < groups; first += 64) {
    const int p = wave_prefix(tile_rows(first + lane));
    if (first == 0) upto = p;
    total += __builtin_amdgcn_readlane(p, 63);
  }
  total *= tiles_n;
  const int xcd = bid & 7, at = bid >> 3, per = total >> 3, rem = total & 7;
  if (at >= per + (xcd < rem ? 1 : 0)) return false;
  int t = xcd * per + min(xcd, rem) + at, first = 0;
  for (;;) {  // to the 64 groups that have it
    const int all = __builtin_amdgcn_readlane(upto, 63) * tiles_n;
    if (t < all) break;
    t -= all;
    first += 64;
    if (first >= groups) return false;
    upto = wave_prefix(tile_rows(first + lane));
  }
  const int in = __ffsll((unsigned long long)__ballot(t < upto * tiles_n)) - 1;
  const int before = in > 0 ? __builtin_amdgcn_readlane(upto, max(in - 1, 0)) : 0;
  const int mt = __builtin_amdgcn_readlane(upto, in) - before;
  g = first + in;
  t -= before * tiles_n;
  const int band = t / (4 * tiles_n), row = band * 4, size = min(mt - row, 4), rest = t - band * 4 * tiles_n;
  tm = row + rest % size;
  tn = rest / size;
  return true;
}

// A bf16 tile by way of LDS (free of operands by now), whole row pieces at a
// time, 16-byte chunks swizzled by row; the lanes' own stores would write 8
// bytes of 32 different rows each.
template <class C, class T>
__device__ __forceinline__ void store_staged(const Out<T>& out, int64_t row0, int m0, int n0, int M, int N, char* smem,
                                             const f32x16 (&acc)[C::FM][C::FN]) {
  constexpr int RB = C::BN * 2, CH = RB / 16, RPW = C::BM / C::NW;
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
        *(uint2*)(smem + row * RB + (((byte >> 4) ^ (row & (CH - 1))) << 4) + (byte & 15)) =
            make_uint2(f32x2_to_bf16x2(acc[i][j][q * 4], acc[i][j][q * 4 + 1]),
                       f32x2_to_bf16x2(acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]));
      }
  }
  __syncthreads();
  constexpr int RPI = 64 / CH;  // rows a store instruction covers
  const int c = lane % CH, n = n0 + c * 8;
#pragma unroll 4
  for (int it = 0; it < RPW / RPI; ++it) {
    const int row = wave * RPW + it * RPI + lane / CH;
    if (m0 + row >= M || n >= N) continue;
    const char* src = smem + row * RB + ((c ^ (row & (CH - 1))) << 4);
    T* dst = out.row(row0 + row) + n;
    if (n + 8 <= N) {
      *(i32x4_any*)dst = *(const i32x4*)src;
    } else {
      for (int i = 0; i < N - n; ++i) dst[i] = ((const bf16_t*)src)[i];
    }
  }
}

template <class C, class T>
__global__ void __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(2, 2)))
mx8_gemm_tile(Operand a, Operand b, Out<T> out, const int32_t* counts, int max_rows, int N, int K, int groups, int tiles_n) {
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int FM = C::FM, FN = C::FN, NF = C::NF, NMMA = FM * FN;
  constexpr int LDS = SPLIT || C::OPERANDS > C::STAGED ? C::OPERANDS : C::STAGED;
  __shared__ __attribute__((aligned(1024))) char smem[LDS];
  int g, tm, tn;
  if (!tile_of<C::BM>(counts, max_rows, groups, tiles_n, blockIdx.x, g, tm, tn)) return;
  const int M = group_rows(counts, g, max_rows), m0 = tm * C::BM, n0 = tn * C::BN;
  const int nb = K / MX_BLOCK, nc = K / 16, nk = (nb + 3) / 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int64_t arow = g * a.per_group, brow = g * b.per_group;

  // A: load d of a wave brings in rows 32 wave + 8 d + lane / 8; B: load d the
  // lines 16 wave + 8 d + lane / 8 of two rows.  An immediate offset moves both
  // addresses of a load by 1024 d, which is taken off the row's pointer.
  const int lrow = lane >> 3, lcol = lane & 7;
  const int acol = lcol ^ swz(wave * 32 + lrow);  // rows 8 further: ^ 4
  const int bcol = lcol ^ swz(wave * 16 + lrow);  // lines 8 further: ^ 4, the line's other row
  const uint8_t *pa[4], *pb[2];                   // where the next step to load has them
#pragma unroll
  for (int d = 0; d < 4; ++d)
    pa[d] = a.v.codes + (arow + min(m0 + wave * 32 + d * 8 + lrow, M - 1)) * a.v.ldc + (acol ^ (d & 1) * 4) * 16 - 1024 * d;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const int row = 2 * (wave * 16 + d * 8 + lrow) + ((bcol >> 2) ^ d);
    pb[d] = b.v.codes + (brow + min(n0 + row, N - 1)) * b.v.ldc + (bcol & 3) * 16 - 1024 * d;
  }
  // scales: thread tid brings in row tid of A (below BM) or of B
  const uint8_t* ps = tid < C::BM ? a.v.scales + (arow + min(m0 + tid, M - 1)) * a.v.lds
                                  : b.v.scales + (brow + min(n0 + tid - C::BM, N - 1)) * b.v.lds;

  const int frow = lane & 31, half = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  // Where a lane's fragments are in buffer 0: of A by substep and half of the
  // operand, of B by substep (32 rows further: 32 lines of A, 16 of B).
  const int fa_swz = swz(frow), fb_swz = swz(frow >> 1) ^ ((frow & 1) << 2);
  uint32_t fa[2][2], fb[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      fa[ks][p] = lds0 + (wm * C::WTM + frow) * 128 + (uint32_t)(((ks * 4 + p * 2 + half) ^ fa_swz) << 4);
    fb[ks] = lds0 + C::A_BYTES + (wn * C::WTN + frow) / 2 * 128 + (uint32_t)(((ks * 2 + half) ^ fb_swz) << 4);
  }
  const uint32_t sa = lds0 + C::STAGES * C::STAGE + (wm * C::WTM + frow) * 16;
  const uint32_t sb = lds0 + C::STAGES * C::STAGE + (C::BM + wn * C::WTN + frow) * 16;

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  Frags<FM> F[2];
  int raw[NF], sc[NF];  // a step's scale bytes as read, and those of its substeps as bytes 0 and 2
  // Fragment q in [0, NF) of a substep; at: its buffer's place.
  auto read_codes = [&](Frags<FM>& f, uint32_t at, auto ks_tag, auto q_tag) {
    constexpr int ks = decltype(ks_tag)::value, q = decltype(q_tag)::value;
    if constexpr (q < FM) {  // the two halves of a register tuple
      i32x4 lo, hi;
      read16<q * 32 * 128>(lo, fa[ks][0] + at);
      read16<q * 32 * 128>(hi, fa[ks][1] + at);
      f.a[q] = fp8_operand(lo, hi);
    } else {
      read16<(q - FM) * 16 * 128>(f.b[q - FM], fb[ks] + at);
    }
  };
  auto read_scales = [&](uint32_t at, auto q_tag) {  // q in [0, NF)
    constexpr int q = decltype(q_tag)::value;
    if constexpr (q < FM) read4<q * 32 * 16>(raw[q], sa + at);
    else read4<(q - FM) * 32 * 16>(raw[q], sb + at);
  };
  auto scales_at = [&](int kt) { return (uint32_t)(((kt >> 2) & 1) * C::SCALES + (kt & 3) * 4); };
  // Load d in [0, 6) of step kt, the next one in order.  LAST: it may be the
  // last step, whose chunks past K are the row's last one in their place.
  auto load_codes = [&](int kt, int buf, int d, auto last_tag) {
    const int dd = d < 4 ? d : d - 4;
    const uint8_t*& p = d < 4 ? pa[dd] : pb[dd];
    int64_t back = 0;
    if constexpr (decltype(last_tag)::value)
      back = 16 * (int64_t)(d < 4 ? min(0, nc - 1 - (kt * 8 + (acol ^ (dd & 1) * 4))) : min(0, nb - 1 - (kt * 4 + (bcol & 3))));
    const void* gp = p + back;
    auto lp = (__attribute__((address_space(3))) void*)(smem + buf * C::STAGE +
                                                         (d < 4 ? wave * 32 * 128 : C::A_BYTES + wave * 16 * 128));
    switch (dd) {
      case 0: __builtin_amdgcn_global_load_lds(gp, lp, 16, 0, 0); break;
      case 1: __builtin_amdgcn_global_load_lds(gp, lp, 16, 1024, 0); break;
      case 2: __builtin_amdgcn_global_load_lds(gp, lp, 16, 2048, 0); break;
      default: __builtin_amdgcn_global_load_lds(gp, lp, 16, 3 * 1024, 0); break;
    }
    p += d < 4 ? 128 : 64;
  };
  auto load_scales = [&](int four) {  // steps 4 four .. 4 four + 3
    auto lp = (__attribute__((address_space(3))) void*)(smem + C::STAGES * C::STAGE + (four & 1) * C::SCALES + wave * 1024);
    __builtin_amdgcn_global_load_lds((const void*)(ps + (int64_t)four * 16), lp, 16, 0, 0);
  };
  i32x8 large, small;  // SPLIT: the two parts of the fragment of A in use
  auto mma = [&](Frags<FM>& f, int i, int j, auto sel_tag) {
    constexpr int SEL = decltype(sel_tag)::value;
    if constexpr (SPLIT) {
      if (j == 0) {
        large = fp8_large(f.a[i]);
        small = f.a[i] ^ large;
      }
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(f.b[j]), large, acc[i][j], 4, 0, SEL, sc[FM + j],
                                                                  SEL, sc[i]);
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(f.b[j]), small, acc[i][j], 4, 0, SEL, sc[FM + j],
                                                                  SEL, sc[i]);
    } else {
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(f.b[j]), f.a[i], acc[i][j], 4, 0, SEL, sc[FM + j],
                                                                  SEL, sc[i]);
    }
  };
  // Step kt out of buffer buf, the next one out of nbuf.  LEFT: steps that follow
  // it, 4 for four and more: with three and more the loads of step kt + 3 are issued.
  auto step = [&](int kt, int buf, int nbuf, auto left_tag) {
    constexpr int LEFT = decltype(left_tag)::value;
    // The scales of the four steps from kt + 3 on, into the buffer whose last
    // step was kt - 2.  (A branch further down would let the compiler move the
    // matrix instructions past it, away from the reads they hide.)
    if constexpr (LEFT >= 3)
      if (((kt + 3) & 3) == 0) load_scales((kt + 3) >> 2);
    // A lane's bytes of the step's scales come down to bytes 0 and 2; those of
    // blocks that K does not have are cleared.
    uint32_t keep = 0xff00ffu;
    if constexpr (LEFT == 0) {
      const int have = nb - kt * 4 - half;  // blocks from this lane's first one on
      keep = (have > 0 ? 0xffu : 0u) | (have > 2 ? 0xff0000u : 0u);
    }
#pragma unroll
    for (int q = 0; q < NF; ++q) sc[q] = (int)(((uint32_t)raw[q] >> (8 * half)) & keep);
    const uint32_t at = (uint32_t)(buf * C::STAGE), nat = (uint32_t)(nbuf * C::STAGE), sat = scales_at(kt + 1);
    each<NMMA>([&](auto q) {
      mma(F[0], q / FN, q % FN, std::integral_constant<int, 0>());
      if constexpr (q < NF) read_codes(F[1], at, std::integral_constant<int, 1>(), q);
      __builtin_amdgcn_sched_barrier(0);
    });
    wait_reads(F[1]);
    if constexpr (LEFT > 0) {
      // step kt + 1's codes and scales (this lane's part); step kt + 2's 6 loads may be under way
      vm_wait<(LEFT > 1 ? 6 : 0)>();
      lds_barrier();  // ... every lane's; every wave is done with step kt's buffer
    }
    each<NMMA>([&](auto q) {
      mma(F[1], q / FN, q % FN, std::integral_constant<int, 2>());
      if constexpr (LEFT > 0 && q < NF) {
        read_codes(F[0], nat, std::integral_constant<int, 0>(), q);
        read_scales(sat, q);
      }
      if constexpr (LEFT >= 3) {
        using Last = std::integral_constant<bool, LEFT == 3>;
        if (q < 6) load_codes(kt + 3, buf, q, Last());
        if (q + NMMA < 6) load_codes(kt + 3, buf, q + NMMA, Last());
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (LEFT > 0) wait_reads(F[0], raw);
  };
  load_scales(0);
  for (int t = 0; t < 3; ++t)
    if (t < nk) {
#pragma unroll
      for (int d = 0; d < 6; ++d) load_codes(t, t, d, std::true_type());
    }
  if (nk > 2) vm_wait<12>();
  else if (nk > 1) vm_wait<6>();
  else vm_wait<0>();
  lds_barrier();
  each<NF>([&](auto q) {
    read_codes(F[0], 0, std::integral_constant<int, 0>(), q);
    read_scales(0, q);
  });
  wait_reads(F[0], raw);
  int kt = 0, buf = 0;
  auto go = [&](auto left_tag) {
    const int next = buf == 2 ? 0 : buf + 1;
    step(kt, buf, next, left_tag);
    buf = next;
    ++kt;
  };
  while (kt + 4 < nk) go(std::integral_constant<int, 4>());
  if (nk > 3) go(std::integral_constant<int, 3>());
  if (nk > 2) go(std::integral_constant<int, 2>());
  if (nk > 1) go(std::integral_constant<int, 1>());
  go(std::integral_constant<int, 0>());

  if constexpr (!SPLIT) {
    store_staged<C>(out, arow + m0, m0, n0, M, N, smem, acc);
  } else {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = m0 + wm * C::WTM + i * 32 + frow;
      if (m >= M) continue;
      T* row = out.row(arow + m);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn * C::WTN + j * 32 + q * 8 + half * 4;
          const float v[4] = {acc[i][j][q * 4], acc[i][j][q * 4 + 1], acc[i][j][q * 4 + 2], acc[i][j][q * 4 + 3]};
          if (n < N) out.store4(row, n, N, v);
        }
    }
  }
}

template <class C, class T>
void run_tiles(const MxGemmArgs& q, const Operand& a, const Operand& b, const Out<T>& out, hipStream_t st) {
  const int64_t tiles_n = (q.n + C::BN - 1) / C::BN, tiles = q.groups * (((int64_t)q.max_rows + C::BM - 1) / C::BM) * tiles_n;
  launch((mx8_gemm_tile<C, T>), dim3((unsigned)(8 * ((tiles + 7) / 8))), dim3(C::NT), 0, st, a, b, out, q.counts, q.max_rows, q.n,
         q.k, q.groups, (int)tiles_n);
}

// Up to 64 rows: whether tiles of 128 x 128 are faster.  Times beside the launch
// in units of K / 10 ns.  Without tiles: a CU's share of the workgroups, which
// read each row's lines by themselves (two workgroups at a time where there are
// more than CUs).  By tiles: the steps' latency, until a CU has more than one;
// twice the matrix instructions with an fp32 output; a start and an end of 1.3
// us.  The rows are max_rows, as the launch does not know the counts.  8 groups of
// 64 rows x 4096 x 6144 to bf16 26 us by tiles and 109 without, of 8 rows 24 and
// 34; 64 x 4096 x 6144 20 and 15; 48 groups of one row x 2048 x 2048 22 and 20.
bool few_by_tiles(const MxGemmArgs& q, int cus) {
  const double groups = q.groups, k = q.k;
  const double workgroups = groups * ((q.n + 15) / 16) / cus, share = workgroups <= 1 ? 1 : std::max(2.0, workgroups);
  const double tiles = groups * ((q.n + 127) / 128) / cus, step = q.bf16 ? 27 : 57;
  return share * (3 + 4.5 * q.max_rows / 16) > step * std::max(1.0, 1.1 * tiles) + 13000 / k;
}

template <class T>
hipError_t run_mx8_gemm(const MxGemmArgs& q, int cus, hipStream_t st) {
  const Operand a{q.a, q.max_rows}, b{q.b, q.n};
  const Out<T> out{(char*)q.out, q.ldo};
  if (q.max_rows > 64 || few_by_tiles(q, cus)) {
    if constexpr (sizeof(T) == 4) {
      run_tiles<Tile<128>>(q, a, b, out, st);
    } else {
      // Rounds of the card's CUs that the tiles take: one workgroup of 256 x 256 a
      // CU, or two of 128 x 128, which together take 0.65 of a large tile's time
      // (at 4096 values a row 33 and 50 us) for half of its work.  The rows are
      // max_rows, as the launch does not know the counts.
      auto rounds = [&](int64_t tile, int64_t at_once) {
        const int64_t tiles = q.groups * ((q.max_rows + tile - 1) / tile) * ((q.n + tile - 1) / tile);
        return (double)((tiles + at_once - 1) / at_once);
      };
      if (q.max_rows <= 64 || rounds(128, 2 * cus) * 0.65 < rounds(256, cus)) run_tiles<Tile<128>>(q, a, b, out, st);
      else run_tiles<Tile<256>>(q, a, b, out, st);
    }
    return hipGetLastError();
  }
  // one wave for each 512-piece of K, as far as a workgroup goes
  const dim3 grid((unsigned)((q.n + 15) / 16), (unsigned)q.groups);
  const int pieces = (q.k + 511) / 512;
  auto rows = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    if (pieces <= 4) launch((mx8_gemm_rows<MT, 4, T>), grid, dim3(256), 0, st, a, b, out, q.counts, q.max_rows, q.n, q.k);
    else if (pieces <= 8) launch((mx8_gemm_rows<MT, 8, T>), grid, dim3(512), 0, st, a, b, out, q.counts, q.max_rows, q.n, q.k);
    else launch((mx8_gemm_rows<MT, 16, T>), grid, dim3(1024), 0, st, a, b, out, q.counts, q.max_rows, q.n, q.k);
  };
  if (q.max_rows <= 16) rows(std::integral_constant<int, 1>());
  else if (q.max_rows <= 32) rows(std::integral_constant<int, 2>());
  else rows(std::integral_constant<int, 4>());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx8_gemm(const MxGemmArgs& g, int cus, hipStream_t st) {
  return g.bf16 ? run_mx8_gemm<bf16_t>(g, cus, st) : run_mx8_gemm<float>(g, cus, st);
}

}  // namespace moe
