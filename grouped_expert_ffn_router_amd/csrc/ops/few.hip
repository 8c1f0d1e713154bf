// The few-token layer (gfx950): one whole mixture-of-experts layer for up to
// 64 tokens.
//
// Every product is [a few tokens] x [rows of weights], so the weights' bytes
// bound it: each is read once, 16 bytes a lane straight from memory into the
// A operand of a 16 x 16 matrix instruction (16 weight rows; the tokens are
// the B operand, 16 at a time), and the tokens' rows come from the caches.
// The layer is a chain of all-to-all dependencies, a launch for each:
//   project  logits = x W_r^T, z = x W_d^T
//   select   top-k of each token, the chosen experts and their tokens (one
//            workgroup); beside it hs = silu(x Wg^T) (x Wu^T) of the shared experts
//   gate_up  h = silu(z Wg^T) (z Wu^T) of each chosen expert
//   down     c = sum over the chosen experts of w (h W2^T)
//   up       out = c U^T + sum hs W2s^T
// MI355X, model width 6144, latent 2048, 8 of 384 experts of 1536 and two
// shared ones: one token 95 us (319 MB: 3.4 TB/s), 64 tokens 0.91 - 0.94 ms (5.5
// GB: 5.9 TB/s), 16 tokens with MX-FP4 experts 214 us (0.72 GB: 3.4 TB/s); a small
// layer (512 wide, one token) 23 us.  What bounds the small ones is the five
// round trips to memory, 2 us and more each with cold caches, and launching.
// One launch for all after the projections (a queue of items in order of
// dependency, device-scope counters and waits between them) was built and
// took 58 us for the small layer and 216 us for one token: a wait across the
// eight XCDs costs more than the end of a launch.  Also slower or level: bf16
// tokens' rows staged in LDS with the weights one group ahead (108 us for one
// token; the registers halve the waves in flight), 16 waves a workgroup in the
// products with all tokens, one read of the tokens' rows for several row tiles
// in the experts' gate and up products, and in the MX-FP4 experts' down product
// (58 us) the tokens' rows staged in LDS by each wave (77 us) or the next piece's
// weights loaded ahead (70 us: 147 registers, a quarter of the waves less).

#include "few.h"

namespace moe {

namespace {

constexpr int FEW_CUS = 256;  // what the products' splits are sized for (the workspace's size depends on it)
constexpr int NW = 8;       // waves of a workgroup
constexpr int NTHREADS = NW * 64;

// ------------------------------------------------------------ operands

__device__ __forceinline__ float silu_exact(float a) { return a / (1.0f + expf(-a)); }

// 16 rows of weights by 16-byte pieces.  Lane (r, g) = (lane % 16, lane / 16)
// holds row r and the g-th piece of a step of KSTEP values.
struct WBf16 {
  static constexpr int KSTEP = 32;
  const bf16_t* p;  // this lane's row
  struct Piece { i32x4 w; };
  __device__ Piece load(int k, int g) const { return {__builtin_nontemporal_load((const i32x4*)(p + k + g * 8))}; }
};

struct WMx {
  static constexpr int KSTEP = 128;
  const uint8_t* p;
  const uint8_t* s;
  struct Piece { i32x4 w; uint32_t scale; };
  __device__ Piece load(int k, int g) const {
    return {__builtin_nontemporal_load((const i32x4*)(p + (k >> 1) + g * 16)), s[(k >> 5) + g]};
  }
};

struct WF32 {
  static constexpr int KSTEP = 16;
  const float* p;
  struct Piece { float w[4]; };
};

// acc[t] += 16 weight rows x tokens 16 t .. over one step, tokens' rows at hi[t] / lo[t].
template <bool LO, int NT>
__device__ __forceinline__ void mma(f32x4 (&acc)[NT], const WBf16::Piece& w, const bf16_t* const (&hi)[NT], int64_t lo, int k,
                                    int g) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const bf16_t* a = hi[t] + k + g * 8;
    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.w), *(const bf16x8*)a, acc[t], 0, 0, 0);
    if (LO)
      acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.w), *(const bf16x8*)(a + lo), acc[t],
                                                       0, 0, 0);
  }
}

// Eight codes (one dword) with their block's scale as bf16 values: exact (a
// code has two significant bits) up to bf16's range, which only scale bytes 253
// and 254 pass.  The conversion takes the scale's exponent field as the scale
// byte itself: 0 stands for 2^-127 and 255 for NaN.
__device__ __forceinline__ bf16x8 mx_to_bf16(uint32_t codes, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// `in`: false in lanes whose block is past the rows' end; they read nothing and
// multiply zeros (a token's value there instead would be 0 * inf = NaN).
template <bool LO, int NT>
__device__ __forceinline__ void mma(f32x4 (&acc)[NT], const WMx::Piece& w, const bf16_t* const (&hi)[NT], int64_t lo, int k,
                                    int g, bool in = true) {
  auto load = [&](const bf16_t* a) { return in ? *(const bf16x8*)a : bf16x8{}; };
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bf16x8 wv = mx_to_bf16((uint32_t)w.w[q], w.scale);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const bf16_t* a = hi[t] + k + g * 32 + q * 8;
      acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, load(a), acc[t], 0, 0, 0);
      if (LO) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, load(a + lo), acc[t], 0, 0, 0);
    }
  }
}

// Products of RT x 16 weight rows with the tokens over the steps [s0, s1) that
// fall to wave `part` of `parts`, in groups of U steps.  LO: the tokens' rows
// have a second part, `lo` elements behind the first.  FORM: ROUND, each
// workgroup begins at another group, so that workgroups that run together do not
// read the same columns of rows a power of two apart, which lie in the same
// channels of memory; AHEAD, the tokens' values of a group are loaded before its
// first product (bf16 rows).
enum DotForm { PLAIN, ROUND, AHEAD };
template <class W, bool LO, int RT, int NT, int U = (sizeof(typename W::Piece) == 16 ? 4 : 2), DotForm FORM = PLAIN>
__device__ __forceinline__ void dot(f32x4 (&acc)[RT][NT], const W (&w)[RT], const bf16_t* const (&hi)[NT], int64_t lo,
                                    int K, int part, int parts) {
  const int g = lane_id() >> 4;
  const int full = K / W::KSTEP, groups = (full + U - 1) / U;
  const int mine = part < groups ? (groups - part + parts - 1) / parts : 0;
  const int begin = FORM == ROUND && mine > 0 ? (int)(blockIdx.x % (unsigned)mine) * parts : 0;
  for (int j = part; j < groups; j += parts) {
    int i = j;
    if (FORM == ROUND && (i += begin) >= part + mine * parts) i -= mine * parts;
    const int s0 = i * U;
    if (s0 + U <= full) {
      typename W::Piece p[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < RT; ++r) p[u][r] = w[r].load((s0 + u) * W::KSTEP, g);
      if constexpr (FORM == AHEAD) {
        bf16x8 x[U][NT][1 + LO];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const bf16_t* a = hi[t] + (s0 + u) * W::KSTEP + g * 8;
            x[u][t][0] = *(const bf16x8*)a;
            if constexpr (LO) x[u][t][1] = *(const bf16x8*)(a + lo);
          }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int l = 0; l < 1 + LO; ++l)
                acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p[u][r].w), x[u][t][l],
                                                                    acc[r][t], 0, 0, 0);
        continue;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < RT; ++r) mma<LO, NT>(acc[r], p[u][r], hi, lo, (s0 + u) * W::KSTEP, g);
    } else {
      for (int s = s0; s < full; ++s)
#pragma unroll
        for (int r = 0; r < RT; ++r) mma<LO, NT>(acc[r], w[r].load(s * W::KSTEP, g), hi, lo, s * W::KSTEP, g);
    }
  }
  if constexpr (W::KSTEP == 128) {
    // the last blocks of 32 that do not fill a step: lanes past them have nothing
    const int k = full * W::KSTEP;
    if (k < K && part == groups % parts) {
      const bool in = k + g * 32 < K;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        typename W::Piece p = {i32x4{0, 0, 0, 0}, 0};
        if (in) p = w[r].load(k, g);
        mma<LO, NT>(acc[r], p, hi, lo, k, g, in);
      }
    }
  }
}

// fp32: any K and any alignment, 4 values a lane and step, U steps at a time.
template <class W, bool LO, int RT, int NT, int = 0, DotForm = PLAIN>
__device__ __forceinline__ void dot(f32x4 (&acc)[RT][NT], const W (&w)[RT], const float* const (&hi)[NT], int64_t, int K,
                                    int part, int parts) {
  constexpr int U = 4;
  const int g = lane_id() >> 4;
  const int steps = (K + 15) / 16, full = K / 16;
  uintptr_t at = 0;
#pragma unroll
  for (int r = 0; r < RT; ++r) at |= (uintptr_t)w[r].p;
#pragma unroll
  for (int t = 0; t < NT; ++t) at |= (uintptr_t)hi[t];
  const bool vec = __all((at & 15) == 0);
  auto mma = [&](const float (&b)[RT][4], const float (&x)[NT][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[r][i], x[t][i], acc[r][t], 0, 0, 0);
  };
  int s = part;
  if (vec)
    for (; s + (U - 1) * parts < full; s += U * parts) {
      float b[U][RT][4], x[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + u * parts) * 16 + g * 4;
#pragma unroll
        for (int r = 0; r < RT; ++r) *(float4*)b[u][r] = *(const float4*)(w[r].p + k);
#pragma unroll
        for (int t = 0; t < NT; ++t) *(float4*)x[u][t] = *(const float4*)(hi[t] + k);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) mma(b[u], x[u]);
    }
  for (; s < steps; s += parts) {
    const int k = s * 16 + g * 4;
    float b[RT][4], x[NT][4];
    if (vec && s < full) {
#pragma unroll
      for (int r = 0; r < RT; ++r) *(float4*)b[r] = *(const float4*)(w[r].p + k);
#pragma unroll
      for (int t = 0; t < NT; ++t) *(float4*)x[t] = *(const float4*)(hi[t] + k);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int r = 0; r < RT; ++r) b[r][i] = k + i < K ? w[r].p[k + i] : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t][i] = k + i < K ? hi[t][k + i] : 0.f;
      }
    }
    mma(b, x);
  }
}

// ------------------------------------------------------------ activations

__device__ __forceinline__ void put_act(const FewAct& a, bf16_t*, int64_t i, float v) {
  bf16_t hi = f32_to_bf16(v);
  if ((hi & 0x7fff) == 0x7f80 && __builtin_isfinite(v)) --hi;  // rounded past bf16's largest: that, and the rest below
  const float rest = v - bf16_to_f32(hi);
  ((bf16_t*)a.hi)[i] = hi;
  ((bf16_t*)a.lo)[i] = __builtin_isfinite(rest) ? f32_to_bf16(rest) : (bf16_t)0;
}
__device__ __forceinline__ void put_act(const FewAct& a, float*, int64_t i, float v) { ((float*)a.hi)[i] = v; }

// Elements from a value's first part to its second.
template <class T>
__device__ __forceinline__ int64_t lo_offset(const FewAct& a) { return (const T*)a.lo - (const T*)a.hi; }

// ------------------------------------------------------------ phases

// Sums of the accumulators of the KS waves (all of a workgroup, or 1) that
// share rows, in wave order, G row tiles at a time (a gate tile and its up tile
// together): f(group, t, sums) gets those of token tile t, each 4 weight rows
// 4 g .. of token r16.
template <int G, int KS, int RT, int NT, class F>
__device__ __forceinline__ void reduce(f32x4 (&acc)[RT][NT], f32x4* lds, F f) {
  static_assert(RT % G == 0 && (KS == 1 || KS == NW), "whole groups");
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if constexpr (KS == 1) {
#pragma unroll
    for (int grp = 0; grp < RT / G; ++grp)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 s[G];
#pragma unroll
        for (int i = 0; i < G; ++i) s[i] = acc[grp * G + i][t];
        f(grp, t, s);
      }
    return;
  }
#pragma unroll
  for (int grp = 0; grp < RT / G; ++grp) {  // a group at a time: NW * G * NT KB of LDS
    __syncthreads();
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) lds[((wave * G + i) * NT + t) * 64 + lane] = acc[grp * G + i][t];
    __syncthreads();
    if (wave < NT) {
      f32x4 s[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        s[i] = lds[(i * NT + wave) * 64 + lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s[i] += lds[((w * G + i) * NT + wave) * 64 + lane];
      }
      f(grp, wave, s);
    }
  }
}

template <class T> struct Weights { using type = WBf16; };
template <> struct Weights<float> { using type = WF32; };

template <int RT, int NT>
__device__ __forceinline__ void zero(f32x4 (&acc)[RT][NT]) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
}

__host__ __device__ __forceinline__ int tiles_of(int n, int rows) { return (n + rows - 1) / rows; }

// Products over K shared by the waves of a workgroup.  bf16 rows with one token
// tile: eight steps in flight as long as every wave has them, then four (one
// token, 6144 wide: 13, 22 and 19 us for the three phases with all tokens; 14, 24
// and 20 with four; fp32: level).  More token tiles: their values loaded ahead
// (64 tokens: 34, 43 and 52 us, 38, 44 and 61 without).  Groups of steps go
// round the waves: `turn` is the wave that takes the first, the next product's
// turn comes back.
template <class W, bool LO, int RT, int NT, class T>
__device__ __forceinline__ int dot_waves(f32x4 (&acc)[RT][NT], const W (&w)[RT], const T* const (&hi)[NT], int64_t lo, int K,
                                         int turn = 0) {
  const int part = ((threadIdx.x >> 6) + NW - turn) % NW;
  if constexpr (W::KSTEP == 32 && NT == 1) {
    const int deep = K - K % (8 * W::KSTEP * NW);
    if (deep) {
      dot<W, LO, RT, NT, 8>(acc, w, hi, lo, deep, part, NW);
      W w2[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) w2[r] = W{w[r].p + deep};
      const T* const hi2[NT] = {hi[0] + deep};
      dot<W, LO, RT, NT>(acc, w2, hi2, lo, K - deep, part, NW);
    } else {
      dot<W, LO, RT, NT>(acc, w, hi, lo, K, part, NW);
    }
    return (turn + tiles_of(K - deep, 4 * W::KSTEP)) % NW;
  } else {
    dot<W, LO, RT, NT, 4, AHEAD>(acc, w, hi, lo, K, part, NW);
    return (turn + tiles_of(K, (W::KSTEP == 32 ? 4 : 1) * W::KSTEP)) % NW;
  }
}

// Items: 16 router rows, then 16 rows of W_down.
template <class T, int NT>
__device__ __forceinline__ void project(const FewArgs& a, int item, f32x4* lds) {
  const FewDims& d = a.d;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  using W = typename Weights<T>::type;
  const T* hi[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) hi[t] = (const T*)a.x + (int64_t)min(t * 16 + r16, d.T - 1) * d.D;
  const int nr = tiles_of(d.E, 16);
  const bool router = item < nr;
  const int n0 = (router ? item : item - nr) * 16, N = router ? d.E : d.L;
  const W w[1] = {{(const T*)(router ? a.w_router : a.w_down) + (int64_t)min(n0 + r16, N - 1) * d.D}};
  f32x4 acc[1][NT];
  zero(acc);
  dot_waves<W, false, 1, NT>(acc, w, hi, 0, d.D);
  reduce<1, NW, 1, NT>(acc, lds, [&](int, int t, const f32x4 (&s)[1]) {
    const int m = t * 16 + r16;
    if (m >= d.T) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int n = n0 + g * 4 + v;
      if (n >= N) break;
      if (router) {
        float b = 0.f;
        if (a.bias) b = a.bias[(int64_t)(a.bias_row_tokens ? m / a.bias_row_tokens : 0) * d.E + n];
        a.logits[(int64_t)m * d.E + n] = s[0][v] + b;
      } else {
        put_act(a.z, (T*)nullptr, (int64_t)m * d.L + n, s[0][v]);
      }
    }
  });
}

// Item: 16 hidden units of a shared expert.
template <class T, int NT>
__device__ __forceinline__ void shared_expert(const FewArgs& a, int item, f32x4* lds) {
  const FewDims& d = a.d;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  using W = typename Weights<T>::type;
  const T* hi[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) hi[t] = (const T*)a.x + (int64_t)min(t * 16 + r16, d.T - 1) * d.D;
  const int ns = tiles_of(d.HS, 16), j = item / ns, u0 = (item - j * ns) * 16;
  const T* base = (const T*)a.ws13 + ((int64_t)j * 2 * d.HS + min(u0 + r16, d.HS - 1)) * d.D;
  const W w[2] = {{base}, {base + (int64_t)d.HS * d.D}};
  f32x4 acc[2][NT];
  zero(acc);
  dot_waves<W, false, 2, NT>(acc, w, hi, 0, d.D);
  reduce<2, NW, 2, NT>(acc, lds, [&](int, int t, const f32x4 (&s)[2]) {
    const int m = t * 16 + r16;
    if (m >= d.T) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int u = u0 + g * 4 + v;
      if (u < d.HS) put_act(a.hs, (T*)nullptr, ((int64_t)m * d.S + j) * d.HS + u, silu_exact(s[0][v]) * s[1][v]);
    }
  });
}

// The tokens of chosen expert i, by rank.  One token id per thread below 64.
__device__ __forceinline__ int token_list(uint64_t mask, int* list) {
  const int t = threadIdx.x;
  __syncthreads();
  if (t < 64 && ((mask >> t) & 1)) list[__popcll(mask & ((1ull << t) - 1))] = t;
  __syncthreads();
  return __popcll(mask);
}

template <class W> struct Bank {  // a routed expert's weight rows
  const void* codes;
  const uint8_t* scales;
  __device__ W row(int64_t r, int K) const;
};
template <> __device__ __forceinline__ WBf16 Bank<WBf16>::row(int64_t r, int K) const { return {(const bf16_t*)codes + r * K}; }
template <> __device__ __forceinline__ WF32 Bank<WF32>::row(int64_t r, int K) const { return {(const float*)codes + r * K}; }
template <> __device__ __forceinline__ WMx Bank<WMx>::row(int64_t r, int K) const {
  return {(const uint8_t*)codes + r * (K / 2), scales + r * mx_scale_bytes(K)};
}

constexpr int STAGE_BYTES = 32 * 1024;  // LDS that a workgroup may fill with tokens' rows
__host__ __device__ __forceinline__ int staged_row(int L) { return 2 * L + 8; }  // elements of a row in LDS

// 16 hidden units of a chosen expert for its tokens m0 .. m0 + 16 NT - 1, by
// one wave (KS = 1) or with K shared by the waves of a workgroup (KS = NW).
// STAGED: the tokens' rows are in LDS (staged), first part, second part and
// padding to a row.
template <class T, class W, int KS, int NT, bool STAGED = false>
__device__ __forceinline__ void gate_up(const FewArgs& a, int i, int u0, const int* list, int m0, int n, f32x4* lds,
                                        const T* staged = nullptr) {
  const FewDims& d = a.d;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, g = lane >> 4;
  const T* hi[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    hi[t] = STAGED ? staged + min(r16, n - 1) * staged_row(d.L)
                   : (const T*)a.z.hi + (int64_t)list[min(m0 + t * 16 + r16, n - 1)] * d.L;
  const Bank<W> bank{a.w13, a.w13_scales};
  const int64_t row = (int64_t)a.active[i] * 2 * d.H + min(u0 + r16, d.H - 1);
  const W w[2] = {bank.row(row, d.L), bank.row(row + d.H, d.L)};
  f32x4 acc[2][NT];
  zero(acc);
  // 284 bf16 experts of 1536 x 2048: 516 us, all from the first group on 553
  dot<W, sizeof(T) == 2, 2, NT, W::KSTEP == 128 ? 2 : 4, W::KSTEP == 32 ? ROUND : PLAIN>(
      acc, w, hi, STAGED ? d.L : lo_offset<T>(a.z), d.L, KS == 1 ? 0 : wave, KS);
  const int64_t first = a.first[i];
  reduce<2, KS, 2, NT>(acc, lds, [&](int, int t, const f32x4 (&s)[2]) {
    const int m = m0 + t * 16 + r16;
    if (m >= n) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int u = u0 + g * 4 + v;
      if (u < d.H) put_act(a.h, (T*)nullptr, (first + m) * d.H + u, silu_exact(s[0][v]) * s[1][v]);
    }
  });
}

// Item: 16 RT rows of the latent width and one of `parts` shares of the chosen
// experts' hidden units.  A wave takes pieces (expert, DOWN_K hidden units) in
// turn, weighs each piece's sums with the tokens' routing weights and adds
// them to its own rows in LDS; the waves' rows are added in wave order, and
// the last of a tile's shares to finish adds the shares in their order.
// Hidden units of a piece, measured: bf16, one token, 16.0 us with 256 and 18.7 with 512; MX-FP4, 16 tokens, 57.5 us
// with 256, 59.9 with 512 and 64.8 with 1024; fp32, 7 tokens, 8.7 us with 128, 10.0 with 64 and 11 with 256.
constexpr int DOWN_K_ACT = 256, DOWN_K_MX = 256, DOWN_K_F32 = 128;
template <class W>
constexpr int DOWN_K = W::KSTEP == 128 ? DOWN_K_MX : W::KSTEP == 16 ? DOWN_K_F32 : DOWN_K_ACT;

template <class T, class W, int RT, int NT>
__device__ __forceinline__ void down_piece(const FewArgs& a, int i, int k0, int l0, uint64_t mask, int m0, float* rows) {
  const FewDims& d = a.d;  // the expert's tokens m0 .. m0 + 16 NT - 1
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4, n = __popcll(mask);
  const int K = min(DOWN_K<W>, d.H - k0);
  const int64_t first = a.first[i], e = a.active[i];
  const T* hi[NT];
  int tok[NT];
  float gate[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = min(m0 + t * 16 + r16, n - 1);
    hi[t] = (const T*)a.h.hi + (first + m) * d.H + k0;
    uint64_t rest = mask;  // the m-th set bit
    for (int s = 0; s < m; ++s) rest &= rest - 1;
    tok[t] = __ffsll((unsigned long long)rest) - 1;
    gate[t] = a.gate[(int64_t)tok[t] * d.X + e];
  }
  const Bank<W> bank{a.w2, a.w2_scales};
  W w[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    w[r] = bank.row(e * d.L + min(l0 + r * 16 + r16, d.L - 1), d.H);
    if constexpr (W::KSTEP == 128) {
      w[r].p += k0 / 2;
      w[r].s += k0 / 32;
    } else {
      w[r].p += k0;
    }
  }
  f32x4 acc[RT][NT];
  zero(acc);
  dot<W, sizeof(T) == 2, RT, NT>(acc, w, hi, lo_offset<T>(a.h), K, 0, 1);
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (m0 + t * 16 + r16 < n) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        f32x4* p = (f32x4*)(rows + (tok[t] * RT + r) * 16 + g * 4);
        f32x4 v = *p;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = fmaf(gate[t], acc[r][t][q], v[q]);
        *p = v;
      }
    }
}

template <class T, class W, int RT, int NTMAX>
__device__ __forceinline__ void down(const FewArgs& a, int part, int tile, float* lds) {  // lds: [NW][T][16 RT]
  const FewDims& d = a.d;
  constexpr int R = 16 * RT;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l0 = tile * R;
  float* rows = lds + wave * d.T * R;
  for (int i = lane; i < d.T * R; i += 64) rows[i] = 0.f;
  const int active = a.count[0], chunks = tiles_of(d.H, DOWN_K<W>), pieces = active * chunks;
  for (int p = part * NW + wave; p < pieces; p += a.parts * NW) {
    const int i = p / chunks, k0 = (p - i * chunks) * DOWN_K<W>;
    const uint64_t mask = a.mask[i];
    const int n = __popcll(mask);
    if (NTMAX == 1 || n <= 16) down_piece<T, W, RT, 1>(a, i, k0, l0, mask, 0, rows);
    else  // more than 32 tokens read the expert's piece twice
      for (int m0 = 0; m0 < n; m0 += 32) down_piece<T, W, RT, NTMAX>(a, i, k0, l0, mask, m0, rows);
  }
  __syncthreads();
  const int64_t n = (int64_t)d.T * d.L;
  for (int i = threadIdx.x; i < d.T * R; i += NTHREADS) {
    float s = lds[i];
    for (int w = 1; w < NW; ++w) s += lds[w * d.T * R + i];
    const int t = i / R, l = l0 + i % R;
    if (l >= d.L) continue;
    if (a.parts == 1) put_act(a.c, (T*)nullptr, (int64_t)t * d.L + l, s);
    else __hip_atomic_store(&a.part[part * n + (int64_t)t * d.L + l], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.parts == 1) return;
  // The shares of a tile meet: the last workgroup to arrive adds them.  The
  // shares were stored, and are read, with device scope (through the L2 of the
  // XCD, which others do not see), so waiting for the stores is all the
  // release that is needed; a device-wide fence writes back the whole L2,
  // which took 100 us here.
  __shared__ int last;
  vm_wait<0>();
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(&a.arrived[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.parts - 1;
  __syncthreads();
  if (!last) return;
  for (int i = threadIdx.x; i < d.T * R; i += NTHREADS) {
    const int t = i / R, l = l0 + i % R;
    if (l >= d.L) continue;
    const float* p = a.part + (int64_t)t * d.L + l;
    float s = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int q = 1; q < a.parts; ++q) s += __hip_atomic_load(p + q * n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    put_act(a.c, (T*)nullptr, (int64_t)t * d.L + l, s);
  }
}

// Item: 16 RT output columns.
template <class T, int RT, int NT>
__device__ __forceinline__ void up(const FewArgs& a, int n0, f32x4* lds) {
  const FewDims& d = a.d;
  const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
  using W = typename Weights<T>::type;
  int64_t row[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) row[r] = min(n0 + r * 16 + r16, d.D - 1);
  f32x4 acc[RT][NT];
  zero(acc);
  const T* hi[NT];
  W w[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) w[r] = W{(const T*)a.w_up + row[r] * d.L};
#pragma unroll
  for (int t = 0; t < NT; ++t) hi[t] = (const T*)a.c.hi + (int64_t)min(t * 16 + r16, d.T - 1) * d.L;
  int turn = dot_waves<W, sizeof(T) == 2, RT, NT>(acc, w, hi, lo_offset<T>(a.c), d.L);
  for (int j = 0; j < d.S; ++j) {
#pragma unroll
    for (int r = 0; r < RT; ++r) w[r] = W{(const T*)a.ws2 + ((int64_t)j * d.D + row[r]) * d.HS};
#pragma unroll
    for (int t = 0; t < NT; ++t)
      hi[t] = (const T*)a.hs.hi + ((int64_t)min(t * 16 + r16, d.T - 1) * d.S + j) * d.HS;
    turn = dot_waves<W, sizeof(T) == 2, RT, NT>(acc, w, hi, lo_offset<T>(a.hs), d.HS, turn);
  }
  reduce<1, NW, RT, NT>(acc, lds, [&](int r, int t, const f32x4 (&s)[1]) {
    const int m = t * 16 + r16;
    if (m >= d.T) return;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int n = n0 + r * 16 + g * 4 + v;
      if (n < d.D) ((T*)a.out)[(int64_t)m * d.D + n] = Act<T>::store(s[0][v]);
    }
  });
}

}  // namespace

// ------------------------------------------------------------ kernels

// The products with all tokens have a workgroup a CU or fewer at the widths above
// (152 to 192): with several token tiles their two waves a SIMD may have all
// registers (64 tokens: the last of them 53 us, 61 with fewer).
#define DENSE_WAVES __attribute__((amdgpu_waves_per_eu(2, NT > 1 ? 2 : 8)))

template <class T, int NT>
__global__ void __launch_bounds__(NTHREADS) DENSE_WAVES few_project(FewArgs a) {
  __shared__ f32x4 lds[NW * NT * 64];
  project<T, NT>(a, blockIdx.x, lds);
}

// Largest key of the wave, in every lane: rotations inside each row of 16
// lanes (DPP row_ror by 8, 4, 2, 1), then the four rows' maxima.
template <int CTRL>
__device__ __forceinline__ uint64_t ror_max(uint64_t k) {
  const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_update_dpp(0, (int)(k >> 32), CTRL, 0xf, 0xf, false) << 32) |
                     (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)k, CTRL, 0xf, 0xf, false);
  return o > k ? o : k;
}
__device__ __forceinline__ uint64_t key_at(uint64_t k, int lane) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32) |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, lane);
}
__device__ __forceinline__ uint64_t max_key(uint64_t k) {
  k = ror_max<0x121>(ror_max<0x122>(ror_max<0x124>(ror_max<0x128>(k))));
  const uint64_t a = key_at(k, 0), b = key_at(k, 16), c = key_at(k, 32), d = key_at(k, 48);
  const uint64_t ab = a > b ? a : b, cd = c > d ? c : d;
  return ab > cd ? ab : cd;
}

// One workgroup: every wave takes tokens in turn, k rounds of a maximum over
// (logit, lower expert first) keys, EPL of them a lane (-0 counts as 0, and a
// NaN by its bits, so that a token always gets k experts); then the chosen
// experts in ascending order with their tokens (a bit each: an expert is
// chosen once a token).  It also clears the counters of the down product.
struct SelectLds {
  unsigned long long mask[2048];
  int wave_n[NW], wave_p[NW];
};

template <int EPL>
__device__ __forceinline__ void select(const FewArgs& a, SelectLds& lds) {
  auto& mask = lds.mask;
  const FewDims& d = a.d;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int e = tid; e < d.X; e += NTHREADS) mask[e] = 0;
  for (int i = tid; i < a.tiles; i += NTHREADS) a.arrived[i] = 0;
  __syncthreads();
  for (int t = wave; t < d.T; t += NW) {
    uint64_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 64 * j;
      key[j] = 0;
      if (e < d.E) {
        uint32_t u = __float_as_uint(a.logits[(int64_t)t * d.E + e]);
        if (u == 0x80000000u) u = 0;
        key[j] = ((uint64_t)((u & 0x80000000u) ? ~u : (u | 0x80000000u)) << 32) | (uint32_t)~(uint32_t)e;
      }
    }
    float my_v = 0.f, v0 = 0.f;
    int my_e = 0;
    for (int r = 0; r < d.k; ++r) {
      uint64_t best = key[0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) best = key[j] > best ? key[j] : best;
      best = max_key(best);
      const int e = (int)~(uint32_t)best;
      const uint32_t o = (uint32_t)(best >> 32);
      const float v = __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
      if (r == 0) v0 = v;
      if (lane == r) {
        my_v = v;
        my_e = e;
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (lane + 64 * j == e) key[j] = 0;
    }
    const float ex = lane < d.k ? expf(my_v - v0) : 0.f;
    float sum = ex;
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane < d.k) {
      a.topk_idx[(int64_t)t * d.k + lane] = my_e;
      a.topk_w[(int64_t)t * d.k + lane] = ex / sum;
      const int le = my_e - d.x0;
      if (le >= 0 && le < d.X) {
        atomicOr(&mask[le], 1ull << t);  // in LDS; the order does not matter
        a.gate[(int64_t)t * d.X + le] = ex / sum;
      }
    }
  }
  __syncthreads();
  // chosen experts and their pair rows: four experts a thread, scans inside the waves and over them
  constexpr int PER = 2048 / NTHREADS;
  int n = 0, p = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    const uint64_t m = e < d.X ? mask[e] : 0;
    n += m != 0;
    p += __popcll(m);
  }
  int sn = n, sp = p;
  for (int o = 1; o < 64; o <<= 1) {
    const int an = __shfl_up(sn, o), ap = __shfl_up(sp, o);
    if (lane >= o) {
      sn += an;
      sp += ap;
    }
  }
  if (lane == 63) {
    lds.wave_n[wave] = sn;
    lds.wave_p[wave] = sp;
  }
  __syncthreads();
  int at = sn - n, row = sp - p;
  for (int w = 0; w < wave; ++w) {
    at += lds.wave_n[w];
    row += lds.wave_p[w];
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = tid * PER + j;
    const uint64_t m = e < d.X ? mask[e] : 0;
    if (!m) continue;
    a.active[at] = e;
    a.mask[at] = m;
    a.first[at] = row;
    ++at;
    row += __popcll(m);
  }
  if (tid == NTHREADS - 1) a.count[0] = at;
}

// The choice needs one workgroup and the shared experts do not wait for it:
// workgroup 0 chooses while the others stream the shared experts' weights.
template <class T, int EPL, int NT>
__global__ void __launch_bounds__(NTHREADS) DENSE_WAVES few_select_shared(FewArgs a) {
  constexpr int SUMS = NW * 2 * NT * 64 * (int)sizeof(f32x4), SELECT = (int)sizeof(SelectLds);
  __shared__ __attribute__((aligned(16))) char lds[SUMS > SELECT ? SUMS : SELECT];
  if (blockIdx.x) {
    shared_expert<T, NT>(a, blockIdx.x - 1, (f32x4*)lds);
    return;
  }
  select<EPL>(a, *(SelectLds*)lds);
}

// Workgroups of 4 waves that work apart (KS = 1), or of NW that share K.
constexpr int GU_WAVES = 4;

template <class T, class W, int KS, int NTMAX>
__global__ void __launch_bounds__(KS == 1 ? GU_WAVES * 64 : NTHREADS) few_gate_up(FewArgs a) {
  __shared__ f32x4 lds[KS == 1 ? 1 : NW * 2 * NTMAX * 64];
  __shared__ f32x4 rows[KS == 1 && W::KSTEP == 128 ? STAGE_BYTES / 16 : 1];
  __shared__ int list[64];
  constexpr int BLOCK = KS == 1 ? GU_WAVES * 16 : 16;
  const int tiles = tiles_of(a.d.H, BLOCK);
  const int i = blockIdx.x / tiles, u0 = (blockIdx.x - i * tiles) * BLOCK + (KS == 1 ? (threadIdx.x >> 6) * 16 : 0);
  if (i >= a.count[0]) return;
  const int n = token_list(a.mask[i], list);
  if constexpr (KS == 1 && W::KSTEP == 128) {
    // MX-FP4: the tokens' rows are eight times the weights' bytes in the L1
    // (two parts of 16 bits a value, read by every wave); from LDS they leave
    // the weights' loads alone (110 experts of 1536 x 2048: 90 us, without 116)
    if (n <= 16 && n * staged_row(a.d.L) * 2 <= STAGE_BYTES) {
      const int per = a.d.L / 8;
      for (int x = threadIdx.x; x < n * 2 * per; x += GU_WAVES * 64) {
        const int r = x / per, c = x - r * per;
        *(uint4*)((bf16_t*)rows + (r >> 1) * staged_row(a.d.L) + (r & 1) * a.d.L + c * 8) =
            *(const uint4*)((const bf16_t*)(r & 1 ? a.z.lo : a.z.hi) + (int64_t)list[r >> 1] * a.d.L + c * 8);
      }
      __syncthreads();
      if (u0 < a.d.H) gate_up<T, W, KS, 1, true>(a, i, u0, list, 0, n, lds, (const T*)rows);
      return;
    }
  }
  if (KS == 1 && u0 >= a.d.H) return;
  if (NTMAX == 1 || n <= 16) gate_up<T, W, KS, 1>(a, i, u0, list, 0, n, lds);
  else  // more than 32 tokens read the expert's rows twice
    for (int m0 = 0; m0 < n; m0 += 32) gate_up<T, W, KS, NTMAX>(a, i, u0, list, m0, n, lds);
}

template <class T, class W, int RT, int NTMAX>
__global__ void __launch_bounds__(NTHREADS) few_down(FewArgs a) {
  extern __shared__ float rows[];
  const int part = blockIdx.x / a.tiles;
  down<T, W, RT, NTMAX>(a, part, blockIdx.x - part * a.tiles, rows);
}

template <class T, int RT, int NT>
__global__ void __launch_bounds__(NTHREADS) DENSE_WAVES few_up(FewArgs a) {
  __shared__ f32x4 lds[NW * NT * 64];
  up<T, RT, NT>(a, blockIdx.x * 16 * RT, lds);
}

// ------------------------------------------------------------ host

FewWs few_layout(const FewDims& d) {
  FewWs w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t es = d.bf16 ? 2 : 4, second = d.bf16 ? 2 : 0;
  w.logits = take((size_t)d.T * d.E * 4);
  w.mask = take((size_t)d.X * 8);
  w.active = take((size_t)d.X * 4);
  w.first = take((size_t)d.X * 4);
  w.count = take(64);
  w.gate = take((size_t)d.T * d.X * 4);
  w.z = take((size_t)d.T * d.L * es);
  w.z_lo = take((size_t)d.T * d.L * second);
  w.hs = take((size_t)d.T * d.S * d.HS * es);
  w.hs_lo = take((size_t)d.T * d.S * d.HS * second);
  w.h = take((size_t)d.T * d.k * d.H * es);
  w.h_lo = take((size_t)d.T * d.k * d.H * second);
  w.c = take((size_t)d.T * d.L * es);
  w.c_lo = take((size_t)d.T * d.L * second);
  // The down product: two row tiles share the reads of the tokens' hidden
  // values (16 tokens with MX-FP4 experts: 60 us, one tile or four 77; 64 tokens:
  // 315 us, one 337), one where there would be too few workgroups; shares as
  // many as give every CU two workgroups and every wave of a share something to do.
  const int64_t most = d.X < d.T * d.k ? d.X : d.T * d.k;
  const int64_t pieces = most * tiles_of(d.H, d.mx ? DOWN_K_MX : d.bf16 ? DOWN_K_ACT : DOWN_K_F32), most_parts = (pieces + NW - 1) / NW;
  w.down_rt = 2;
  while (w.down_rt > 1 && tiles_of(d.L, 16 * w.down_rt) * most_parts < 2 * FEW_CUS) w.down_rt /= 2;
  w.tiles = tiles_of(d.L, 16 * w.down_rt);
  int64_t parts = (2 * FEW_CUS + w.tiles - 1) / w.tiles;
  if (parts > most_parts) parts = most_parts;
  w.parts = parts < 1 ? 1 : (int)parts;
  w.part = take((size_t)(w.parts > 1 ? w.parts : 0) * d.T * d.L * 4);
  w.arrived = take((size_t)w.tiles * 4);
  w.total = off;
  return w;
}

// f(type tag, weight tag, token tiles) for the layer's types and tokens.
template <class F>
hipError_t few_dispatch(const FewDims& d, F f) {
  auto tiles = [&](auto t, auto w) {
    if (d.T <= 16) f(t, w, std::integral_constant<int, 1>());
    else if (d.T <= 32) f(t, w, std::integral_constant<int, 2>());
    else f(t, w, std::integral_constant<int, 4>());
  };
  if (!d.bf16) tiles(float(), WF32());
  else if (d.mx) tiles(bf16_t(), WMx());
  else tiles(bf16_t(), WBf16());
  return hipGetLastError();
}

hipError_t launch_few_project(const FewArgs& a, hipStream_t st) {
  return few_dispatch(a.d, [&](auto t, auto, auto nt) {
    launch((few_project<decltype(t), decltype(nt)::value>), dim3((unsigned)(tiles_of(a.d.E, 16) + tiles_of(a.d.L, 16))),
           dim3(NTHREADS), 0, st, a);
  });
}

hipError_t launch_few_select(const FewArgs& a, hipStream_t st) {
  return few_dispatch(a.d, [&](auto t, auto, auto nt) {
    const dim3 grid((unsigned)(1 + a.d.S * tiles_of(a.d.HS, 16)));
    constexpr int NT = decltype(nt)::value;
    if (a.d.E <= 512) launch((few_select_shared<decltype(t), 8, NT>), grid, dim3(NTHREADS), 0, st, a);
    else launch((few_select_shared<decltype(t), 32, NT>), grid, dim3(NTHREADS), 0, st, a);
  });
}

hipError_t launch_few_gate_up(const FewArgs& a, hipStream_t st) {
  const unsigned most = (unsigned)(a.d.X < a.d.T * a.d.k ? a.d.X : a.d.T * a.d.k);
  return few_dispatch(a.d, [&](auto t, auto w, auto nt) {
    constexpr int NT = decltype(nt)::value > 2 ? 2 : decltype(nt)::value;
    // A wave to itself for 16 units where that gives every CU 16 of them (110
    // MX-FP4 experts of 1536 x 2048: 90 us, sharing K 128; 284 bf16 experts: 516
    // and 554), else K is shared: one token's 8 experts are only 768 such tiles.
    if ((int64_t)most * tiles_of(a.d.H, 16) >= 16 * FEW_CUS)
      launch((few_gate_up<decltype(t), decltype(w), 1, NT>), dim3(most * tiles_of(a.d.H, GU_WAVES * 16)), dim3(GU_WAVES * 64),
             0, st, a);
    else
      launch((few_gate_up<decltype(t), decltype(w), NW, NT>), dim3(most * tiles_of(a.d.H, 16)), dim3(NTHREADS), 0, st, a);
  });
}

hipError_t launch_few_down(const FewArgs& a, hipStream_t st) {
  return few_dispatch(a.d, [&](auto t, auto w, auto nt) {
    constexpr int NT = decltype(nt)::value > 2 ? 2 : decltype(nt)::value;
    auto go = [&](auto rt) {
      constexpr int RT = decltype(rt)::value;
      launch((few_down<decltype(t), decltype(w), RT, NT>), dim3((unsigned)(a.parts * a.tiles)), dim3(NTHREADS),
             (uint32_t)(NW * a.d.T * 16 * RT * 4), st, a);
    };
    if (a.down_rt == 2) go(std::integral_constant<int, 2>());
    else go(std::integral_constant<int, 1>());
  });
}

hipError_t launch_few_up(const FewArgs& a, hipStream_t st) {
  return few_dispatch(a.d, [&](auto t, auto, auto nt) {
    auto go = [&](auto rt) {
      constexpr int RT = decltype(rt)::value;
      launch((few_up<decltype(t), RT, decltype(nt)::value>), dim3((unsigned)tiles_of(a.d.D, 16 * RT)), dim3(NTHREADS), 0, st, a);
    };
    // One row tile a workgroup while every CU has at most one of those, else two, which share each read of the tokens'
    // rows (two parts of 16 bits a value), but for one or two tokens, whose rows are little.  One and two tiles, bf16:
    // 4096 wide, 8 tokens 10.6 and 14.0 us, 64 tokens 28.9 and 32.4; 6144 wide, one token 20.1 and 20.3, 4 tokens 23.5 and
    // 20.9, 16: 36.6 and 26.1, 64: 87.6 and 52.3; fp32, 4096 wide, 64 tokens 35.2 and 49.2, 6144 wide 108 and 81.
    if (tiles_of(a.d.D, 16) > FEW_CUS && a.d.T > 2) go(std::integral_constant<int, 2>());
    else go(std::integral_constant<int, 1>());
  });
}

}  // namespace moe
