// The choice of experts from router logits under a rule (softmax or sigmoid
// scores, a balance bias that counts for the choice alone, groups of experts,
// the k best, weights renormalised over them), and the logits' gradient (gfx950).
//
// The order is that of the scores as 64-bit arithmetic has them.  It is found
// in fp32: every comparison that decides something (neighbours among the k + 1
// best, the groups around the last one kept) has to differ by more than the
// fp32 scores can be off, or the token is ordered again from fp64 scores.
// Without a bias the k best are ordered by the logits themselves, which both
// scores are monotone in, so that there nothing is off.

#include "block.h"

namespace moe {

namespace {

constexpr int SOFTMAX = 0;

// Order-preserving key: a larger value has a larger key, -0 that of +0; 0 is below every value's.
__device__ __forceinline__ uint32_t rank_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float rank_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
constexpr uint32_t OUT_KEY = 0x007fffffu;  // of -infinity: an expert that is out

// Largest value of the wave, in every lane: rotations inside each row of 16
// lanes, then the four rows' maxima as scalars.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp_move<0x128>(v));
  v = max(v, dpp_move<0x124>(v));
  v = max(v, dpp_move<0x122>(v));
  v = max(v, dpp_move<0x121>(v));
  const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
  const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
  return max(a, b);
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, off);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ uint64_t rank_key64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double rank_value64(uint64_t key) {
  return __longlong_as_double((long long)((key >> 63) ? (key & ~(1ull << 63)) : ~key));
}
constexpr uint64_t OUT_KEY64 = 0x000fffffffffffffull;

struct GroupDiv {  // expert -> group; exact below 2048
  float inv;
  __device__ int of(int e) const { return (int)(((float)e + 0.5f) * inv); }
};

// One token in fp64: its k picks, pick r in lane r.  Nearly every token is
// settled by the fp32 scores, so this is written for few registers.
template <int EPL>
__device__ __forceinline__ int select_exactly(const SelectRule& r, const float* row, const float* balance, int E, int k,
                                           GroupDiv div) {
  const int lane = lane_id();
  double top = 0, inv_sum = 1;
  if (r.score == SOFTMAX) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 64) m = fmaxf(m, row[e]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    top = m;
    double s = 0;
    for (int e = lane; e < E; e += 64) s += exp((double)row[e] - top);
    inv_sum = 1.0 / wave_sum(s);
  }
  auto key_of = [&](int e) -> uint64_t {
    if (e >= E) return 0;
    const float l = row[e];
    if (l == -INFINITY) return OUT_KEY64;
    const double s = r.score == SOFTMAX ? exp((double)l - top) * inv_sum : 1.0 / (1.0 + exp(-(double)l));
    return rank_key64(balance ? s + (double)balance[e] : s);
  };
  uint64_t kept = ~0ull;
  if (r.top_groups < r.groups) {
    // lane g ends up with the score of group g
    uint64_t mine = 0;
    for (int g = 0; g < r.groups; ++g) {
      uint64_t a = 0, b = 0;  // this lane's two best of the group
      for (int j = 0; j < EPL; ++j) {
        const int e = lane + 64 * j;
        if (e < E && div.of(e) == g) {
          const uint64_t x = key_of(e);
          if (x > a) { b = a; a = x; }
          else if (x > b) b = x;
        }
      }
      const uint64_t first = wave_max64(a);
      const uint64_t owner = __ballot(a == first);
      const uint64_t second = wave_max64(lane == __ffsll((unsigned long long)owner) - 1 ? b : a);
      uint64_t score = first;
      if (r.group_best > 1 && second > OUT_KEY64) score = rank_key64(rank_value64(first) + rank_value64(second));
      if (lane == g) mine = score;
    }
    int better = 0;
    for (int g = 0; g < r.groups; ++g) {
      const uint64_t other = __shfl((unsigned long long)mine, g);
      better += other > mine || (other == mine && g < lane);
    }
    kept = __ballot(lane < r.groups && better < r.top_groups);
  }
  uint32_t picked = 0;  // bit j: this lane's expert lane + 64 j
  int my = 0;
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    int at = 0;
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 64 * j;
      if (e >= E || (picked >> j & 1)) continue;
      uint64_t x = balance ? key_of(e) : rank_key64((double)row[e]);
      if (!(kept >> div.of(e) & 1)) x = OUT_KEY64;
      if (x > best) { best = x; at = j; }
    }
    const uint64_t top_key = wave_max64(best);
    int e = best == top_key ? lane + 64 * at : 1 << 30;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) e = min(e, __shfl_xor(e, off));
    if ((e & 63) == lane) picked |= 1u << (e >> 6);
    // an expert that is out is marked by its sign
    if (lane == i) my = top_key == OUT_KEY64 ? ~e : e;
  }
  return my;
}

// One wave per token.  A lane has the experts lane + 64 j; EPL = how many.
template <int EPL>
__global__ void __launch_bounds__(256)
select_rule_kernel(SelectRule r, const float* __restrict__ logits, int64_t ld, const float* __restrict__ balance, int64_t T,
                   int E, int k, int32_t* __restrict__ idx, float* __restrict__ w) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = lane_id();
  if (t >= T) return;
  const float* row = logits + t * ld;
  const GroupDiv div{(float)r.groups / (float)E};
  const bool grouped = r.top_groups < r.groups;
  const bool scores = grouped || balance;  // else the logits rank
  float l[EPL], v[EPL];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    l[j] = e < E ? row[e] : -INFINITY;
    bad |= !(l[j] == l[j]);
  }
  float top = 0.f, inv_sum = 1.f;
  if (r.score == SOFTMAX) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = fmaxf(m, l[j]);
    top = rank_value(wave_max(rank_key(m)));
    bad |= top == INFINITY;
    if (scores || !r.renorm) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) s += l[j] == -INFINITY ? 0.f : expf(l[j] - top);
      inv_sum = 1.0f / wave_sum(s);
    }
  }
  auto score_of = [&](float x) {
    if (x == -INFINITY) return 0.f;
    return r.score == SOFTMAX ? expf(x - top) * inv_sum : 1.0f / (1.0f + expf(-x));
  };
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 64 * j;
    v[j] = l[j];
    if (scores && l[j] != -INFINITY) {
      v[j] = score_of(l[j]);
      if (balance) v[j] += balance[e];
      bad |= !(v[j] == v[j]);
    }
  }
  if (__any(bad)) {  // no order: the first k experts, their weights NaN
    if (lane < k) {
      idx[t * k + lane] = lane;
      w[t * k + lane] = NAN;
    }
    return;
  }
  uint32_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) key[j] = lane + 64 * j < E ? rank_key(v[j]) : 0u;
  // the largest score bounds how far scores are off (a few units in the last place)
  const float unit = 0x1p-20f * (r.score == SOFTMAX ? inv_sum : 1.0f);
  bool close = false;
  if (grouped) {
    uint32_t mine = 0;
    for (int g = 0; g < r.groups; ++g) {
      uint32_t a = 0, b = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const uint32_t x = lane + 64 * j < E && div.of(lane + 64 * j) == g ? key[j] : 0u;
        b = max(b, min(a, x));
        a = max(a, x);
      }
      const uint32_t first = wave_max(a);
      const uint64_t owner = __ballot(a == first);
      const uint32_t second = wave_max(lane == __ffsll((unsigned long long)owner) - 1 ? b : a);
      uint32_t s = first;
      if (r.group_best > 1 && second > OUT_KEY) s = rank_key(rank_value(first) + rank_value(second));
      if (lane == g) mine = s;
    }
    int better = 0;
    for (int g = 0; g < r.groups; ++g) {
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, g);
      better += other > mine || (other == mine && g < lane);
    }
    const uint64_t kept = __ballot(lane < r.groups && better < r.top_groups);
    // the last group kept and the first one dropped; two that are out tie by index
    const int last = __ffsll((unsigned long long)__ballot(lane < r.groups && better == r.top_groups - 1)) - 1;
    const int next = __ffsll((unsigned long long)__ballot(lane < r.groups && better == r.top_groups)) - 1;
    const uint32_t klast = (uint32_t)__builtin_amdgcn_readlane((int)mine, last);
    const uint32_t knext = (uint32_t)__builtin_amdgcn_readlane((int)mine, next);
    if (knext > OUT_KEY) {
      const float a = rank_value(klast), b = rank_value(knext);
      close |= !(a - b > 2 * unit + 0x1p-20f * (fabsf(a) + fabsf(b)));
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (lane + 64 * j >= E) continue;
      if (!balance) key[j] = rank_key(l[j]);
      if (!(kept >> div.of(lane + 64 * j) & 1)) key[j] = OUT_KEY;
    }
  }
  // k rounds of a maximum over the wave, and one more to see how near the next one is
  int my = 0;
  uint32_t before = 0;
  const int rounds = balance && k < E ? k + 1 : k;
  for (int i = 0; i < rounds; ++i) {
    uint32_t m = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = max(m, key[j]);
    m = wave_max(m);
    if (balance && i > 0 && m > OUT_KEY) {
      const float a = rank_value(before), b = rank_value(m);
      close |= !(a - b > unit + 0x1p-20f * (fabsf(a) + fabsf(b)));
    }
    before = m;
    int e = 0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint64_t who = __ballot(key[j] == m);
      if (who && !found) {
        e = 64 * j + __ffsll((unsigned long long)who) - 1;
        found = true;
      }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + 64 * j == e) key[j] = 0u;
    if (lane == i) my = m == OUT_KEY ? ~e : e;
  }
  if (close) my = select_exactly<EPL>(r, row, balance, E, k, div);
  const bool out = my < 0;
  const int e = out ? ~my : my;
  float x = -INFINITY;
  if (lane < k && !out) x = row[e];
  float s;
  if (r.score == SOFTMAX && r.renorm) {  // relative to the largest that was chosen
    const float m = rank_value(wave_max(rank_key(x)));
    s = x == -INFINITY ? 0.f : expf(x - m);
  } else {
    s = score_of(x);
  }
  if (r.renorm) {
    const float sum = wave_sum(s);
    s = sum > 0.f ? s / sum : 0.f;
  }
  if (lane < k) {
    idx[t * k + lane] = e;
    w[t * k + lane] = s * r.scale;
  }
}

// ------------------------------------------------------------ gradient
//
// With m = sum_i w_i dw_i / scale over the chosen experts,
//   sigmoid, renormalised   dl_i = w_i (1 - sigmoid(l_i)) (dw_i - m)
//   sigmoid                 dl_i = w_i (1 - sigmoid(l_i)) dw_i
//   softmax, renormalised   dl_i = w_i (dw_i - m)
//   softmax                 dl_e = w_e dw_e [e chosen] - scale m p_e   (p: the softmax over all)
// and 0 elsewhere.  One wave per token; each pick's term is added in the lane
// that writes its expert, so picks of one expert add up in order.

template <int V>
__global__ void __launch_bounds__(256)
select_backward_kernel(SelectRule r, const float* __restrict__ dw, const float* __restrict__ w,
                       const int32_t* __restrict__ idx, const float* __restrict__ logits, int64_t ld, int64_t T, int E,
                       int k, float* __restrict__ dlogits, int64_t ldd) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = lane_id();
  if (t >= T) return;
  const float* row = logits + t * ld;
  int e = -1;
  float wi = 0.f, di = 0.f;
  if (lane < k) {
    e = idx[t * k + lane];
    wi = w[t * k + lane];
    di = dw[t * k + lane];
  }
  if (e < 0 || e >= E) { e = -1; wi = 0.f; di = 0.f; }
  // a weight of 0 (an expert that is out) takes no part, whatever its gradient
  const float wd = wi == 0.f ? 0.f : wi * di;
  const float sum = wave_sum(wd);
  const bool dense = r.score == SOFTMAX && !r.renorm;
  float term = wd;
  if (r.renorm) term = wi == 0.f ? 0.f : wi * (di - sum / r.scale);
  if (r.score != SOFTMAX && wi != 0.f) term *= 1.0f / (1.0f + expf(row[e]));
  float top = 0.f, factor = 0.f;
  if (dense) {
    float m = -INFINITY;
    for (int c = lane; c < E; c += 64) m = fmaxf(m, row[c]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    top = m;
    float s = 0.f;
    for (int c = lane; c < E; c += 64) s += row[c] == -INFINITY ? 0.f : expf(row[c] - top);
    s = wave_sum(s);
    factor = s > 0.f ? -sum / s : 0.f;
  }
  float* out = dlogits + t * ldd;
  for (int c0 = 0; c0 < E; c0 += 64 * V) {
    const int c = c0 + lane * V;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = 0.f;
      if (dense && c + i < E && row[c + i] != -INFINITY) v[i] = factor * expf(row[c + i] - top);
    }
    for (int p = 0; p < k; ++p) {
      const int ep = __builtin_amdgcn_readlane(e, p);
      const float tp = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(term), p));
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i == ep) v[i] += tp;
    }
    if constexpr (V == 4) {
      if (c < E) *(float4*)(out + c) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      if (c < E) out[c] = v[0];
    }
  }
}

// A launch has fewer than 2^32 threads.
template <class F>
hipError_t by_tokens(int64_t T, F f) {
  constexpr int64_t most = 1ll << 24;
  for (int64_t t = 0; t < T; t += most) {
    const int64_t n = T - t < most ? T - t : most;
    f(t, n, dim3((unsigned)((n + 3) / 4)));
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_select_rule(const SelectRule& r, const float* logits, int64_t ld, const float* balance, int64_t T, int E,
                              int k, int32_t* idx, float* w, hipStream_t st) {
  const int epl = (E + 63) / 64;
  return by_tokens(T, [&](int64_t t, int64_t n, dim3 grid) {
    const float* l = logits + t * ld;
    int32_t* i = idx + t * k;
    float* o = w + t * k;
#define SEL(N) launch(select_rule_kernel<N>, grid, dim3(256), 0, st, r, l, ld, balance, n, E, k, i, o)
    if (epl <= 1) SEL(1);
    else if (epl <= 2) SEL(2);
    else if (epl <= 4) SEL(4);
    else if (epl <= 6) SEL(6);
    else if (epl <= 8) SEL(8);
    else if (epl <= 16) SEL(16);
    else SEL(32);
#undef SEL
  });
}

hipError_t launch_select_backward(const SelectRule& r, const float* dw, const float* w, const int32_t* idx,
                                  const float* logits, int64_t ld, int64_t T, int E, int k, float* dlogits, int64_t ldd,
                                  hipStream_t st) {
  const bool wide = E % 4 == 0 && ldd % 4 == 0 && (uintptr_t)dlogits % 16 == 0;
  return by_tokens(T, [&](int64_t t, int64_t n, dim3 grid) {
    const int64_t at = t * k;
    if (wide)
      launch(select_backward_kernel<4>, grid, dim3(256), 0, st, r, dw + at, w + at, idx + at, logits + t * ld, ld, n, E, k,
             dlogits + t * ldd, ldd);
    else
      launch(select_backward_kernel<1>, grid, dim3(256), 0, st, r, dw + at, w + at, idx + at, logits + t * ld, ld, n, E, k,
             dlogits + t * ldd, ldd);
  });
}

}  // namespace moe
