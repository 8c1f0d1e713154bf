// The choice of experts from router logits under a rule (softmax or sigmoid
// scores, a balance bias that counts for the choice alone, groups of experts,
// the k best, weights renormalised over them), and the logits' gradient (gfx950).
//
// The order is that of the scores as 64-bit arithmetic has them (ranks nearer
// than its own rounding, a few 2^-53 of them, in either order).  It is found
// in fp32: every comparison that decides something (neighbours among the k + 1
// best, the groups around the last one kept) has to differ by more than the
// fp32 scores can be off.  Where neighbours do not (about one token in 2000), the
// k + 1 best are put in order by their fp64 scores; where that leaves open which
// they are, all experts by theirs.  Groups that do not differ are chosen by fp64
// scores, and the experts in them as before.
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

// Sums over the wave in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](uint32_t moved) { v += __uint_as_float(moved); };
  add(dpp_move<0xB1>(__float_as_uint(v)));
  add(dpp_move<0x4E>(__float_as_uint(v)));
  add(dpp_move<0x141>(__float_as_uint(v)));
  add(dpp_move<0x140>(__float_as_uint(v)));
  auto row = [&](int lane) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_move64(uint64_t x) {
  return ((uint64_t)dpp_move<CTRL>((uint32_t)(x >> 32)) << 32) | dpp_move<CTRL>((uint32_t)x);
}
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  v = larger(v, dpp_move64<0x128>(v));
  v = larger(v, dpp_move64<0x124>(v));
  v = larger(v, dpp_move64<0x122>(v));
  v = larger(v, dpp_move64<0x121>(v));
  auto row = [&](int lane) {
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
  };
  return larger(larger(row(0), row(16)), larger(row(32), row(48)));
}
__device__ __forceinline__ uint64_t rank_key64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double rank_value64(uint64_t key) {
  return __longlong_as_double((long long)((key >> 63) ? (key & ~(1ull << 63)) : ~key));
}
constexpr uint64_t OUT_KEY64 = 0x000fffffffffffffull;

// e^x to about an ulp (results below 2^-126 are 0): the argument's product with
// log2 e keeps its rounding error, which the power of two is corrected by.
__device__ __forceinline__ float exp_of(float x) {
  x = fminf(fmaxf(x, -200.0f), 200.0f);
  const float hi = x * 1.44269504f;
  const float lo = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269504f, -hi));
  return __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.693147181f, 1.0f);
}

struct GroupDiv {  // expert -> group; exact below 2048
  float inv;
  __device__ int of(int e) const { return (int)(((float)e + 0.5f) * inv); }
};

// The scores of one token's logits in fp64 (the softmax's sum by the whole wave).
struct Score64 {
  bool softmax;
  double top, inv_sum;
  __device__ Score64(const SelectRule& r, const float* row, int E) : softmax(r.score == SOFTMAX), top(0), inv_sum(1) {
    if (!softmax) return;
    const int lane = lane_id();
    float m = -INFINITY;
    for (int e = lane; e < E; e += 64) m = fmaxf(m, row[e]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    top = m;
    double s = 0;
    for (int e = lane; e < E; e += 64) s += exp((double)row[e] - top);
    inv_sum = 1.0 / wave_sum(s);
  }
  // The key of expert e's rank.
  __device__ uint64_t key(const float* row, const float* balance, int e) const {
    const double l = row[e];
    const double s = softmax ? exp(l - top) * inv_sum : 1.0 / (1.0 + exp(-l));
    return l == -INFINITY ? OUT_KEY64 : rank_key64(balance ? s + (double)balance[e] : s);
  }
};

// One token's ranks in fp64; the lanes have the experts as in the kernel below.
template <int EPL>
__device__ __forceinline__ void keys64(const SelectRule& r, const float* row, const float* balance, int E, uint64_t (&key)[EPL]) {
  const int e0 = lane_id() * EPL;
  const Score64 scores(r, row, E);
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    key[j] = scores.key(row, balance, min(e0 + j, E - 1));
    if (e0 + j >= E) key[j] = 0;
    // two at a time: side by side they take hundreds of registers
    if (j & 1) __builtin_amdgcn_sched_barrier(0);
  }
}

// The groups that stay by those ranks, a bit each.
template <int EPL>
__device__ __forceinline__ uint64_t groups64(const SelectRule& r, GroupDiv div, const uint64_t (&key)[EPL]) {
  const int lane = lane_id(), e0 = lane * EPL;
  uint64_t mine = 0;  // lane g: the score of group g
  for (int g = 0; g < r.groups; ++g) {
    uint64_t a = 0, b = 0;  // this lane's two best of the group
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const uint64_t x = div.of(e0 + j) == g ? key[j] : 0;
      if (x > a) { b = a; a = x; }
      else if (x > b) b = x;
    }
    const uint64_t first = wave_max64(a);
    const int owner = __ffsll((unsigned long long)__ballot(a == first)) - 1;
    const uint64_t second = wave_max64(lane == owner ? b : a);
    uint64_t score = first;
    if (r.group_best > 1 && second > OUT_KEY64) score = rank_key64(rank_value64(first) + rank_value64(second));
    if (lane == g) mine = score;
  }
  int better = 0;
  for (int g = 0; g < r.groups; ++g) {
    const uint64_t other = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), g) << 32) |
                           (uint32_t)__builtin_amdgcn_readlane((int)mine, g);
    better += other > mine || (other == mine && g < lane);
  }
  return __ballot(lane < r.groups && better < r.top_groups);
}

// One token's k picks by its ranks in fp64 among the experts of the groups in
// `kept` (group g in bit g step): pick r in lane r, an expert that is out as its
// complement.
template <int EPL>
__device__ __forceinline__ int picks64(GroupDiv div, uint64_t kept, int step, int E, int k, uint64_t (&key)[EPL]) {
  const int lane = lane_id(), e0 = lane * EPL;
#pragma unroll
  for (int j = 0; j < EPL; ++j)
    if (e0 + j < E && !(kept >> (div.of(e0 + j) * step) & 1)) key[j] = OUT_KEY64;
  int my = 0;
  for (int i = 0; i < k; ++i) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (key[j] > best) { best = key[j]; at = j; }
    const uint64_t top_key = wave_max64(best);
    const int owner = __ffsll((unsigned long long)__ballot(best == top_key)) - 1;
    const int e = owner * EPL + __builtin_amdgcn_readlane(at, owner);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j == e) key[j] = 0;
    if (lane == i) my = top_key <= OUT_KEY64 ? ~e : e;
  }
  return my;
}

// Largest value of the wave as a scalar: rotations inside each row of 16 lanes,
// then row 0 (2) into row 1 (3) and rows 0 and 1 into 2 and 3.
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
  v = max(v, dpp_move<0x128>(v));
  v = max(v, dpp_move<0x124>(v));
  v = max(v, dpp_move<0x122>(v));
  v = max(v, dpp_move<0x121>(v));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Descending order of N registers: Batcher's odd-even merge sort of the next
// power of two, without the exchanges that would reach past N.
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
  constexpr int P = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : 32;
#pragma unroll
  for (int p = 1; p < P; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < P; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if ((i + j) / (2 * p) == (i + j + q) / (2 * p) && i + j + q < N) {
            const uint32_t a = v[i + j], b = v[i + j + q];
            v[i + j] = max(a, b);
            v[i + j + q] = min(a, b);
          }
}

// The two largest of this lane's and another lane's pair.
__device__ __forceinline__ void merge_two(uint32_t& a, uint32_t& b, uint32_t a2, uint32_t b2) {
  b = max(max(b, b2), min(a, a2));
  a = max(a, a2);
}

// A lane's values e0 .. e0 + EPL - 1 of a row of E, 16 or 8 bytes at a time where
// it has that many, at any alignment; those past the row are any of its values.
// 16,384 rows of 1001 experts 25 us, with values one at a time 37.
template <int EPL>
__device__ __forceinline__ void lane_values(const float* row, int e0, int E, float (&l)[EPL]) {
  constexpr int W = EPL % 4 == 0 ? 4 : EPL % 2 == 0 ? 2 : 1;  // (E > 64 where W > 1)
#pragma unroll
  for (int j = 0; j < EPL; j += W) {
    const float* at = row + min(e0 + j, E - W);
    if constexpr (W == 4) {
      const i32x4_any d = *(const i32x4_any*)at;
#pragma unroll
      for (int i = 0; i < 4; ++i) l[j + i] = __int_as_float(d[i]);
    } else if constexpr (W == 2) {
      const i32x2_any d = *(const i32x2_any*)at;
      l[j] = __int_as_float(d[0]);
      l[j + 1] = __int_as_float(d[1]);
    } else {
      l[j] = *at;
    }
  }
  if (W > 1 && E % W) {  // a piece that crosses the row's end was loaded up to it
#pragma unroll
    for (int j = 0; j < EPL; j += W) {
      const int n = e0 + j - (E - W);
#pragma unroll
      for (int by = 1; by < W; ++by)
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {  // one place down, up to n times
          const float stay = l[j + i], moved = l[j + i + 1];
          l[j + i] = n >= by ? moved : stay;
        }
    }
  }
}

// One wave per token.  A lane has the experts EPL lane .. EPL lane + EPL - 1, so
// that of equal keys the lower lane's, and in a lane the lower register's, is
// the lower expert's.  Each lane sorts its keys once; a round of the choice is
// then a maximum over the lanes' first keys (6 DPP steps), the lane that holds
// it, and a shift of that lane's keys.  Which expert a key was is looked up
// once at the end.
//
// Bound by instructions (390 a wave for 8 of 384 without groups and bias), not by
// the 4 E bytes a token: 65,536 tokens of 384 experts 39-42 us (the bytes 22 at a
// copy's rate), with sigmoid scores, a bias and 4 of 8 groups 67; 8192 tokens 7.5
// and 12.4, 12 to 18 in groups over draws of the logits; one token 3.2 and 4.8, the
// length of the chain.  All ranks of 8192 tokens equal: 24 us, in groups 50.
// Two tokens a wave (32 lanes with 12 experts each) took 8 % less for 65,536
// tokens without groups, 8 % more in groups, and 80 % more for 8192 in groups.
template <int EPL>
__global__ void __launch_bounds__(256)
select_rule_kernel(SelectRule r, const float* __restrict__ logits, int64_t ld, const float* __restrict__ balance, int64_t T,
                   int E, int k, int32_t* __restrict__ idx, float* __restrict__ w) {
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), e0 = lane * EPL;
  if (t >= T) return;
  const float* row = logits + t * ld;
  const bool grouped = r.top_groups < r.groups;
  const bool full = E == 64 * EPL;  // else lanes past the last expert read it again and drop what they read
  float l[EPL];
  lane_values<EPL>(row, e0, E, l);
  if (!full) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j >= E) l[j] = -INFINITY;
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) bad |= !(l[j] == l[j]);
  float top = 0.f, inv_sum = 1.f;
  if (r.score == SOFTMAX) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = fmaxf(m, l[j]);
    top = rank_value(wave_top(rank_key(m)));
    bad |= top == INFINITY;
    if (grouped || balance || !r.renorm) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) s += l[j] == -INFINITY ? 0.f : exp_of(l[j] - top);
      inv_sum = 1.0f / wave_sum(s);
    }
  }
  // orig: the keys that rank; the scores where a bias is added to them, else the logits
  uint32_t orig[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) orig[j] = rank_key(l[j]);
  uint32_t score[EPL];
  if (grouped || balance) {
    float bias[EPL];
    if (balance) lane_values<EPL>(balance, e0, E, bias);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      float v = r.score == SOFTMAX ? __expf(l[j] - top) * inv_sum : __builtin_amdgcn_rcpf(1.0f + __expf(-l[j]));
      if (balance) v += bias[j];
      if (l[j] == -INFINITY) v = -INFINITY;
      bad |= !(v == v);
      score[j] = rank_key(v);
    }
  }
  if (__any(bad)) {  // no order: the first k experts, their weights NaN
    if (lane < k) {
      idx[t * k + lane] = lane;
      w[t * k + lane] = NAN;
    }
    return;
  }
  if (balance) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) orig[j] = score[j];
  }
  if (!full) {  // below every expert's key
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (e0 + j >= E) orig[j] = score[j] = 0u;
  }
  // How far two scores' difference may be off.  Sigmoid: exp, its argument (times
  // a derivative of 1/4 at most), sum and reciprocal give 3 2^-24 a score; softmax:
  // of the largest score, exp and its argument 3 2^-24, the sum EPL + 8.
  const float unit = r.score == SOFTMAX ? inv_sum * ((EPL + 12) * 0x1p-23f) : 0x1p-21f;
  const GroupDiv div{(float)r.groups / (float)E};
  uint64_t kept = ~0ull;  // groups that stay: group g in bit g kept_step
  int kept_step = 1;
  if (grouped) {
    // Groups of whole lanes, a power of two of them, are reduced side by side
    // in their lanes; others one after the other, group g's score in lane g.
    const int per = E / r.groups, seg = per / EPL;
    const bool aligned = seg * EPL == per && (seg & (seg - 1)) == 0;
    const int gid = aligned ? lane >> (__ffs(seg) - 1) : lane, stride = aligned ? seg : 1;
    uint32_t a = 0, b = 0;
    if (aligned) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        b = max(b, min(a, score[j]));
        a = max(a, score[j]);
      }
      if (seg > 1) merge_two(a, b, dpp_move<0xB1>(a), dpp_move<0xB1>(b));
      if (seg > 2) merge_two(a, b, dpp_move<0x4E>(a), dpp_move<0x4E>(b));
      if (seg > 4) merge_two(a, b, dpp_move<0x141>(a), dpp_move<0x141>(b));
      if (seg > 8) merge_two(a, b, dpp_move<0x140>(a), dpp_move<0x140>(b));
      if (seg > 16) merge_two(a, b, (uint32_t)__shfl_xor((int)a, 16), (uint32_t)__shfl_xor((int)b, 16));
      if (seg > 32) merge_two(a, b, (uint32_t)__shfl_xor((int)a, 32), (uint32_t)__shfl_xor((int)b, 32));
    } else {
      for (int g = 0; g < r.groups; ++g) {
        uint32_t x = 0, y = 0;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const uint32_t s = div.of(e0 + j) == g ? score[j] : 0u;
          y = max(y, min(x, s));
          x = max(x, s);
        }
        const uint32_t first = wave_top(x);
        const int owner = __ffsll((unsigned long long)__ballot(x == first)) - 1;
        const uint32_t second = wave_top(lane == owner ? y : x);
        if (lane == g) { a = first; b = second; }
      }
    }
    uint32_t mine = a;
    if (r.group_best > 1 && b > OUT_KEY) mine = rank_key(rank_value(a) + rank_value(b));
    int better = 0;
    for (int g = 0; g < r.groups; ++g) {
      const uint32_t other = (uint32_t)__builtin_amdgcn_readlane((int)mine, g * stride);
      better += other > mine || (other == mine && g < gid);
    }
    // the last group kept and the first one dropped; two that are out tie by index
    const int last = __ffsll((unsigned long long)__ballot(gid < r.groups && better == r.top_groups - 1)) - 1;
    const int next = __ffsll((unsigned long long)__ballot(gid < r.groups && better == r.top_groups)) - 1;
    const uint32_t klast = (uint32_t)__builtin_amdgcn_readlane((int)mine, last);
    const uint32_t knext = (uint32_t)__builtin_amdgcn_readlane((int)mine, next);
    const float x = rank_value(klast), y = rank_value(knext);
    bool keep;  // this lane's experts, where groups are of whole lanes
    if (knext > OUT_KEY && !(x - y > 2 * unit + 0x1p-22f * (fabsf(x) + fabsf(y)))) {
      uint64_t exact[EPL];
      keys64<EPL>(r, row, balance, E, exact);
      kept = groups64<EPL>(r, div, exact);
      keep = kept >> (gid & 63) & 1;
    } else {
      keep = gid < r.groups && better < r.top_groups;
      kept = __ballot(keep);
      kept_step = stride;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (!(aligned ? keep : kept >> (div.of(e0 + j) & 63) & 1)) orig[j] = min(orig[j], OUT_KEY);
  }
  // k rounds, and two more to see how near the next keys are
  uint32_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) key[j] = orig[j];
  sort_down<EPL>(key);
  int from = 0, chosen = 0;  // lane i: the lane that held pick i, and its key
  const int rounds = balance ? min(k + 2, E) : k;
  for (int i = 0; i < rounds; ++i) {
    const uint32_t m = wave_top(key[0]);
    const int owner = __ffsll((unsigned long long)__ballot(key[0] == m)) - 1;
    from = lane == i ? owner : from;
    chosen = lane == i ? (int)m : chosen;
    const bool pop = lane == owner;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {  // (values, not places, to choose from: an array indexed by `pop` would be spelled out)
      const uint32_t stay = key[j], next = j + 1 < EPL ? key[j + 1] : 0u;
      key[j] = pop ? next : stay;
    }
  }
  const uint32_t mk = (uint32_t)chosen;
  bool near = false, open = false;  // the first k + 1 may be in another order; which they are is open
  if (balance) {
    const uint32_t after = (uint32_t)__shfl_down(chosen, 1);
    if (lane + 1 < rounds && after > OUT_KEY) {
      const float x = rank_value(mk), y = rank_value(after);
      near = !(x - y > unit + 0x1p-23f * (fabsf(x) + fabsf(y)));
    }
    const uint64_t nears = __ballot(near);  // bit i: picks i and i + 1 may be the other way round
    near = nears & ((1ull << k) - 1);
    open = (nears >> (k - 1) & 3) == 3;
  }
  int e;
  bool out;
  if (open) {
    uint64_t exact[EPL];
    keys64<EPL>(r, row, balance, E, exact);
    const int my = picks64<EPL>(div, kept, kept_step, E, k, exact);
    out = my < 0;
    e = out ? ~my : my;
  } else {
    // a lane's equal keys were taken in the order of its registers
    int nth = 0;
    const int from1 = __shfl_up(from, 1), chosen1 = __shfl_up(chosen, 1);
    if (__any(lane > 0 && lane <= k && from1 == from && chosen1 == chosen))
      for (int d = 1; d <= k; ++d) {
        const int from_d = __shfl(from, lane - d), chosen_d = __shfl(chosen, lane - d);
        nth += lane >= d && from_d == from && chosen_d == chosen;
      }
    int at = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if ((uint32_t)__shfl((int)orig[j], from) == mk) {
        at = nth == 0 ? j : at;
        --nth;
      }
    }
    e = from * EPL + at;
    out = mk <= OUT_KEY;
    if (near) {  // the first k + 1 in their order
      const Score64 scores(r, row, E);
      const int n = min(k + 1, E);
      const uint64_t mine = out ? OUT_KEY64 : scores.key(row, balance, lane < n ? e : 0);
      int place = 0;
      for (int p = 0; p < n; ++p) {
        const uint64_t other = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), p) << 32) |
                               (uint32_t)__builtin_amdgcn_readlane((int)mine, p);
        place += other > mine || (other == mine && __builtin_amdgcn_readlane(e, p) < e);
      }
      const int moved = __builtin_amdgcn_ds_permute((lane < n ? place : lane) * 4, out ? ~e : e);
      out = moved < 0;
      e = out ? ~moved : moved;
    }
  }
  float x = -INFINITY;
  if (lane < k && !out) x = row[e];
  // a hardware reciprocal where a quotient is wanted: within an ulp
  // Scores that are divided by their sum count relative to the largest chosen
  // one: of any size, what the logits' differences say of them.
  float s;
  if (r.score == SOFTMAX && r.renorm) {
    s = exp_of(x - rank_value(wave_top(rank_key(x))));
  } else if (r.score == SOFTMAX) {
    s = exp_of(x - top) * inv_sum;
  } else if (r.renorm) {  // 1 / (1 + e^-x) times e^-c, c the largest chosen logit, at most 0: then no term of the largest is above 1
    const float c = fminf(rank_value(wave_top(rank_key(x))), 0.f);
    s = __builtin_amdgcn_rcpf(exp_of(c) + exp_of(c - x));
  } else {
    s = __builtin_amdgcn_rcpf(1.0f + exp_of(-x));
  }
  s = x == -INFINITY ? 0.f : s;
  if (r.renorm) {
    const float sum = wave_sum(s);
    s = sum > 0.f ? s * __builtin_amdgcn_rcpf(sum) : 0.f;
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
// and 0 elsewhere.  One wave per token: its row of terms is laid out in LDS
// (zeros, then each pick's term) and stored whole, so that the time is that of
// writing the row (8192 x 384: 4.5-5.5 us; with each term compared into its lane
// 7.8).  The softmax without renormalisation reads its logits three times, 4 bytes
// a lane: 11.5 us, 65,536 tokens 70 (their bytes 42 at a copy's rate).
// Picks of one expert are added up in their order; that there
// are some shows where a pick does not read its own mark back.

// LDS written by the wave's lanes so far may be read by its other lanes.
__device__ __forceinline__ void wave_lds() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

template <int V>
__global__ void __launch_bounds__(256)
select_backward_kernel(SelectRule r, const float* __restrict__ dw, const float* __restrict__ w,
                       const int32_t* __restrict__ idx, const float* __restrict__ logits, int64_t ld, int64_t T, int E,
                       int k, float* __restrict__ dlogits, int64_t ldd) {
  extern __shared__ float lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;
  const float* row = logits + t * ld;
  const int width = (E + 64 * V - 1) / (64 * V) * (64 * V);
  float* terms = lds + wave * width;
  int e = -1;
  float wi = 0.f, di = 0.f;
  if (lane < k) {
    e = idx[t * k + lane];
    wi = w[t * k + lane];
    di = dw[t * k + lane];
  }
  if (e < 0 || e >= E) { e = -1; wi = 0.f; di = 0.f; }
  const bool dense = r.score == SOFTMAX && !r.renorm;
  for (int c = lane * V; c < width; c += 64 * V) {
    if constexpr (V == 4) *(float4*)(terms + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    else terms[c] = 0.f;
  }
  // a weight of 0 (an expert that is out) takes no part, whatever its gradient
  const float wd = wi == 0.f ? 0.f : wi * di;
  const float sum = wave_sum(wd);
  float term = wd;
  if (r.renorm) term = wi == 0.f ? 0.f : wi * (di - sum / r.scale);
  if (r.score != SOFTMAX && wi != 0.f) term *= __builtin_amdgcn_rcpf(1.0f + exp_of(row[e]));
  wave_lds();
  if (e >= 0) terms[e] = __int_as_float(lane);
  wave_lds();
  const bool mine = e < 0 || __float_as_int(terms[e]) == lane;
  wave_lds();
  if (__all(mine)) {
    if (e >= 0) terms[e] = term;
  } else {  // each expert's first pick adds up all of them
    float all = 0.f;
    int first = lane;
    for (int p = k - 1; p >= 0; --p)
      if (__builtin_amdgcn_readlane(e, p) == e) first = p;
    for (int p = 0; p < k; ++p) {
      const float tp = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(term), p));
      if (__builtin_amdgcn_readlane(e, p) == e) all += tp;
    }
    if (e >= 0 && first == lane) terms[e] = all;
  }
  wave_lds();
  float top = 0.f, factor = 0.f;
  if (dense) {
    float m = -INFINITY;
    for (int c = lane; c < E; c += 64) m = fmaxf(m, row[c]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    top = m;
    float s = 0.f;
    for (int c = lane; c < E; c += 64) s += row[c] == -INFINITY ? 0.f : exp_of(row[c] - top);
    s = wave_sum(s);
    factor = s > 0.f ? -sum / s : 0.f;
  }
  float* out = dlogits + t * ldd;
  for (int c = lane * V; c < E; c += 64 * V) {
    float v[V];
    if constexpr (V == 4) {
      const float4 d = *(const float4*)(terms + c);
      v[0] = d.x; v[1] = d.y; v[2] = d.z; v[3] = d.w;
    } else {
      v[0] = terms[c];
    }
    if (dense) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (row[c + i] != -INFINITY) v[i] += factor * exp_of(row[c + i] - top);
    }
    if constexpr (V == 4) *(float4*)(out + c) = make_float4(v[0], v[1], v[2], v[3]);
    else out[c] = v[0];
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
  const int lane_values = wide ? 256 : 64, lds = 4 * 4 * ((E + lane_values - 1) / lane_values * lane_values);
  return by_tokens(T, [&](int64_t t, int64_t n, dim3 grid) {
    const int64_t at = t * k;
    if (wide)
      launch(select_backward_kernel<4>, grid, dim3(256), lds, st, r, dw + at, w + at, idx + at, logits + t * ld, ld, n, E, k,
             dlogits + t * ldd, ldd);
    else
      launch(select_backward_kernel<1>, grid, dim3(256), lds, st, r, dw + at, w + at, idx + at, logits + t * ld, ld, n, E, k,
             dlogits + t * ldd, ldd);
  });
}

}  // namespace moe
