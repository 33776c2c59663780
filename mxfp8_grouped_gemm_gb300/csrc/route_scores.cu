// Routing by scores: softmax or sigmoid scores of all experts, a selection bias,
// groups of experts, top-k, renormalised weights; and the gradient.
//
// With s the scores, c = s + bias ranks the experts (bias and groups choose, the
// weights are made of s alone):
//   weight_j = scale s_j [/ sum over the chosen s_i]
// A group's score is the sum of its two largest c (or its largest); experts
// outside the best groups do not take part.  Without a bias and without sums
// over groups the order of c is that of the logits, and these are compared.
//
// The ids are those of scores in 64 bits, so that they depend on no rounding:
// the kernel ranks by fp32 scores, whose error it can bound, and a token in
// which a decision lies within that bound is ranked again in fp64 by its warp.
// With sigmoids spread over (0, 1) that is about one token in two thousand.
//
// LPT lanes take a token, eight consecutive experts a lane, so the lowest lane
// has the lowest ids.  Each lane sorts its eight in registers (19 exchanges);
// then a round picks the largest head, and its lane moves up by one.
//
// Measured, launch included: 65536 x 256, top-8, sigmoid, bias, 4 of 8 groups 40
// us, without groups 33, by logits 29; 8191 x 64 softmax 4.3 us.  Bound by
// instructions (424 a warp and token with groups, 293 by logits) at two thirds of
// the issue slots, 24 warps an SM; the logits' stream would take 10 us.  Its
// gradient 21 us, bound by HBM (118 MB: a chosen logit is a 64-byte access).
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kVals = 8;                // experts per lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

enum { SOFTMAX = 0, SIGMOID = 1 };

struct RouteParams {
  const float* logits;
  const float* bias;
  int T, E, k;
  int score;
  int groups, top_groups, group_top;
  int size;             // experts of a group
  int lanes_of_group;   // size / 8 where groups are whole lanes, a power of two; else 0
  int spread;           // else: lanes that scan a group together, a power of two
  int renorm;
  float scale;
  int32_t* ids;
  float* probs;
};

template <int LPT>
__device__ __forceinline__ unsigned group_mask(int lane) {
  return LPT == 32 ? kAll : ((1u << LPT) - 1u) << (lane & ~(LPT - 1));
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LPT == 32) {
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v));
  } else {
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// The sigmoid of a weight: relative error at most 6 x 2^-24.
__device__ __forceinline__ float sigmoid_of(float z) {
  const float t = expf(-fabsf(z));
  return (z >= 0.f ? 1.f : t) / (1.f + t);
}

// The weight of a chosen logit (-inf: 0), of a token whose choices lie in kp
// neighbouring lanes.  A renormalised sigmoid's are taken relative to the largest
// chosen, which keeps them from vanishing together.
__device__ __forceinline__ float weight_of(const RouteParams& P, float z, int kp, float top, float inv) {
  float low = z;
  if (P.renorm)
    for (int off = kp >> 1; off > 0; off >>= 1) low = fmaxf(low, __shfl_xor_sync(kAll, low, off));
  float w;
  if (z == -INFINITY) w = 0.f;
  else if (P.score == SOFTMAX) w = expf(z - (P.renorm ? low : top));
  else w = P.renorm && low < 0.f ? expf(z - low) / (1.f + expf(z)) : sigmoid_of(z);
  if (!P.renorm) return w * (P.score == SOFTMAX ? P.scale * inv : P.scale);
  float total = w;
  for (int off = kp >> 1; off > 0; off >>= 1) total += __shfl_xor_sync(kAll, total, off);
  return total == 0.f ? 0.f : w * (P.scale / total);
}

// ------------------------------------------------------------------ 64 bits --
// Keys that order like the numbers, -0 with +0 and NaN with -inf; 0 is less
// than all of them and stands for "not there".
__device__ __forceinline__ uint64_t key_of(double v) {
  v = v == v ? v + 0.0 : -INFINITY;
  const int64_t b = __double_as_longlong(v);
  return static_cast<uint64_t>(b ^ ((b >> 63) | INT64_MIN));
}
__device__ __forceinline__ double of_key(uint64_t k) {
  const int64_t b = static_cast<int64_t>(k);
  return __longlong_as_double(b ^ ((~b >> 63) | INT64_MIN));
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// --------------------------------------------------------------------- fp32 --
// e^d and 1 / d by the hardware's approximations: relative errors 2^-22.5 (and
// |d| 1.5 x 2^-24 from the rounding of d log2 e), and 2^-23.
__device__ __forceinline__ float exp_fast(float d) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * 1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float rcp_fast(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}
// A lane's list: eight and the -inf behind them, at a stride that keeps 16-byte
// stores of neighbouring lanes in different banks.
constexpr int kList = 12;

// One round: of the lanes whose head is the largest (`best`), the one without
// another `ahead` of it writes (best, its number) to `to` and takes its next, at
// the `end` -inf again.
// All by predicate: as a branch the round took 28 instructions, so it is 11.
__device__ __forceinline__ void take(float& head, uint32_t& list, uint32_t end, uint32_t to, float best, int number,
                                     unsigned ahead) {
  asm volatile(
      "{\n .reg .pred eq, p;\n .reg .b32 who;\n"
      " setp.eq.f32 eq, %0, %3;\n"
      " vote.sync.ballot.b32 who, eq, 0xffffffff;\n"
      " and.b32 who, who, %5;\n"
      " setp.eq.and.u32 p, who, 0, eq;\n"
      " @p st.shared.v2.b32 [%2], {%6, %4};\n"
      " @p add.u32 %1, %1, 4;\n @p min.u32 %1, %1, %7;\n"
      " @p ld.shared.f32 %0, [%1];\n}"
      : "+f"(head), "+r"(list)
      : "r"(to), "f"(best), "r"(number), "r"(ahead), "r"(__float_as_uint(best)), "r"(end)
      : "memory");
}

// Descending, by a network of 19 exchanges, the fewest for eight (Knuth, The Art of
// Computer Programming 3, section 5.3.4, gives the count).
__device__ __forceinline__ void sort8(float (&h)[kVals]) {
  constexpr int net[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                              {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int n = 0; n < 19; ++n) {
    const float a = h[net[n][0]], b = h[net[n][1]];
    h[net[n][0]] = fmaxf(a, b);
    h[net[n][1]] = fminf(a, b);
  }
}
// a >= b and a2 >= b2 become the two largest of the four.
__device__ __forceinline__ void top_two(float& a, float& b, float a2, float b2) {
  b = fmaxf(fminf(a, a2), fmaxf(b, b2));
  a = fmaxf(a, a2);
}

// |v|, the largest finite number in place of infinity (whose distance to any other
// number still passes every bound made of it).
__device__ __forceinline__ float size_of(float v) { return fminf(fabsf(v), FLT_MAX); }
// Half of what |a| + |b| is above |a + b|: for the two largest c of a group, a >= b
// (0 without a second).
__device__ __forceinline__ float apart_of(float a, float b) { return b != -INFINITY ? fmaxf(fminf(a, -b), 0.f) : 0.f; }

struct Kept {
  float worst, next;    // scores of the last group kept and of the best one left out
  float apart;          // largest apart_of, of sums
  uint32_t experts;     // of the lane's eight, those in groups that are kept
  bool close;           // groups of equal scores on both sides
};

// The best groups of any size, from a token's experts in shared memory.
// `scratch`: `room` floats of shared memory of the token's own.
template <int LPT>
__device__ __forceinline__ Kept kept_groups(const RouteParams& P, const float* row_c, float* scratch, int room, int lane) {
  const int gl = lane % LPT;
  const unsigned mask = group_mask<LPT>(lane);
  Kept out{-INFINITY, -INFINITY, 0.f, 0u, false};
  __syncwarp();
  // entry x = gl + LPT r of the lanes' list: group x / spread, scanned with step `spread`
  float score[kVals];
  bool first[kVals];
#pragma unroll
  for (int r = 0; r < kVals; ++r) {
    score[r] = -INFINITY;
    first[r] = false;
    if (r * LPT < P.groups * P.spread) {
      const int x = gl + LPT * r, g = x / P.spread, sub = x % P.spread;
      float a = -INFINITY, b = -INFINITY;
      if (g < P.groups) {
        for (int e = sub; e < P.size; e += P.spread) top_two(a, b, row_c[g * P.size + e], -INFINITY);
      }
      for (int off = 1; off < P.spread; off <<= 1) {
        const float a2 = __shfl_xor_sync(kAll, a, off), b2 = __shfl_xor_sync(kAll, b, off);
        top_two(a, b, a2, b2);
      }
      score[r] = P.group_top == 2 && b != -INFINITY ? a + b : a;
      if (P.group_top == 2) out.apart = fmaxf(out.apart, apart_of(a, b));
      first[r] = g < P.groups && sub == 0;
    }
  }
  out.apart = lanes_max<LPT>(out.apart);
  float cur[kVals];
#pragma unroll
  for (int r = 0; r < kVals; ++r) cur[r] = score[r];
  for (int m = 0; m <= P.top_groups; ++m) {
    float best = cur[0];
#pragma unroll
    for (int r = 1; r < kVals; ++r) best = fmaxf(best, cur[r]);
    out.next = lanes_max<LPT>(best);
    if (m == P.top_groups) break;
    out.worst = out.next;
#pragma unroll
    for (int r = 0; r < kVals; ++r)
      if (cur[r] == out.worst) cur[r] = -INFINITY;
  }
  int kept = 0;
#pragma unroll
  for (int r = 0; r < kVals; ++r) kept += __popc(__ballot_sync(kAll, first[r] && score[r] >= out.worst) & mask);
  out.close = kept != P.top_groups;
  // the scores to shared memory, where every lane finds those of its experts
  for (int lo = 0; lo < P.groups; lo += room) {
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kVals; ++r) {
      const int g = (gl + LPT * r) / P.spread;
      if (first[r] && g >= lo && g < lo + room) scratch[g - lo] = score[r];
    }
    __syncwarp();
    for (int i = 0; i < kVals; ++i) {
      const int e = gl * kVals + i, g = e / P.size;
      if (e < P.E && g >= lo && g < lo + room && scratch[g - lo] >= out.worst) out.experts |= 1u << i;
    }
  }
  __syncwarp();
  return out;
}

// What ranks the experts: the logits, whose order is exact, or scores (with a
// bias, or sums over groups).
enum { BY_LOGIT = 0, BY_SIGMOID = 1, BY_SOFTMAX = 2 };
// Groups: all take part, each is a power of two of whole lanes, any size.
enum { NO_GROUPS = 0, LANE_GROUPS = 1, ANY_GROUPS = 2 };

constexpr float kU = 1.f / 16777216.f;  // 2^-24

// Absolute error of c in fp32 (see below) for scores of at most `most` (1, or the
// softmax's largest) and a |c| of at most `at`.  Both c + error and c - error grow
// with c, so what holds for a decision's two numbers holds for all behind them,
// experts with a bias of -1e9 among them.
template <int BY>
__device__ __forceinline__ float error_of(float most, float at) {
  if constexpr (BY == BY_LOGIT) return 0.f;
  else if constexpr (BY == BY_SIGMOID) return kU * (4.1f + at);
  else return kU * (37.f * most + at);
}
// What an expert that may have to go ahead of one with c = `edge` lies below it at
// most: both errors, and the rounding of the difference.
template <int BY>
__device__ __forceinline__ float slack_of(float most, float edge) {
  return 2.1f * (error_of<BY>(most, size_of(edge)) + kU * size_of(edge)) + 1e-37f;
}

// The warp's largest key (expert 8 lane + i) among those that `in` names, ties
// to the lowest expert; every lane gets the expert.  0: none.
__device__ __forceinline__ uint64_t warp_best(const uint64_t (&key)[kVals], uint32_t in, int lane, int* expert) {
  uint64_t m = 0;
  int idx = 0;
#pragma unroll
  for (int i = kVals - 1; i >= 0; --i) {
    if ((in >> i & 1u) && key[i] >= m) m = key[i], idx = i;
  }
  const uint32_t hi = static_cast<uint32_t>(m >> 32), best_hi = __reduce_max_sync(kAll, hi);
  const uint32_t lo = hi == best_hi ? static_cast<uint32_t>(m) : 0u, best_lo = __reduce_max_sync(kAll, lo);
  const uint64_t best = static_cast<uint64_t>(best_hi) << 32 | best_lo;
  const int owner = __ffs(__ballot_sync(kAll, m == best)) - 1;
  *expert = __shfl_sync(kAll, lane * kVals + idx, owner);
  return best;
}
// One token by the whole warp, everything in fp64: the j-th choice to win[j].y.
template <bool SCORED>
__device__ __noinline__ void rank_all(const RouteParams& P, const float* row, float2* win) {
  const int lane = threadIdx.x & 31;
  double c[kVals];
  uint32_t there = 0, live = 0;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const int e = lane * kVals + i;
    const float z = e < P.E ? row[e] : -INFINITY;
    if (e < P.E) there |= 1u << i;
    if (z != -INFINITY) live |= 1u << i;               // a NaN is on, and its score NaN
    c[i] = z;
    top = fmaxf(top, z);
  }
  if constexpr (SCORED) {
    top = lanes_max<32>(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const bool on = live >> i & 1u;
      if (P.score == SIGMOID) c[i] = on ? 1.0 / (1.0 + exp(-c[i])) : 0.0;
      else c[i] = on ? exp(c[i] - top) : 0.0;
      sum += c[i];
    }
    if (P.score == SOFTMAX) {
      sum = warp_sum(sum);
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (sum != 0.0) c[i] /= sum;
    }
    if (P.bias != nullptr) {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (there >> i & 1u) c[i] += static_cast<double>(P.bias[lane * kVals + i]);
    }
  }
  uint64_t key[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) key[i] = key_of((live >> i & 1u) ? c[i] : -INFINITY);
  if (P.top_groups < P.groups) {
    uint64_t score[kVals];                             // of group 8 lane + i
    uint32_t left = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) score[i] = 0;
    for (int g = 0; g < P.groups; ++g) {
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (static_cast<unsigned>(lane * kVals + i - g * P.size) < static_cast<unsigned>(P.size)) in |= 1u << i;
      int e;
      double a = of_key(warp_best(key, in, lane, &e));
      if (P.group_top == 2) {
        if (e / kVals == lane) in &= ~(1u << (e % kVals));
        const double b = of_key(warp_best(key, in, lane, &e));
        if (b != -INFINITY) a += b;
      }
      if (g / kVals == lane) {
        left |= 1u << (g % kVals);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if (i == g % kVals) score[i] = key_of(a);
      }
    }
    uint32_t kept = 0;                                 // of the lane's own experts
    for (int n = 0; n < P.top_groups; ++n) {
      int g;
      warp_best(score, left, lane, &g);
      if (g / kVals == lane) left &= ~(1u << (g % kVals));
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (static_cast<unsigned>(lane * kVals + i - g * P.size) < static_cast<unsigned>(P.size)) kept |= 1u << i;
    }
    there &= kept;
  }
  for (int j = 0; j < P.k; ++j) {
    int e;
    warp_best(key, there, lane, &e);
    if (e / kVals == lane) there &= ~(1u << (e % kVals));
    if (lane == j) win[j].y = __int_as_float(e);
  }
  __syncwarp();
}

// One token by the whole warp, its decisions in fp64: the j-th choice to
// win[j].y.  fp32 scores and their error bound name the few experts that a
// decision can hang on (each group's group_top largest, and the k largest, with
// what lies within the error of them); these are evaluated in fp64, one to a lane.
// Where they are more than lanes, or experts that are off have to fill the route,
// all are ranked: always where groups are undecided and more than 32 / group_top
// of them have group_top experts on (65536 x 256 with 32 groups takes 65 us for
// that, 41 with 16).  (All in fp64 for every such token cost 14 us of the 57 that
// 65536 x 256 took: a few dozen tokens, but the last to finish; they are 4 us now,
// 6 with the loops over candidates not unrolled and a division in them.)
//   row_c   fp32 c; -inf: off, NaN: its group does not take part
//   win     the choices by fp32 (the k-th bounds the others), then inverse sums
//   groups_close  the groups are to be decided as well: row_c has all of them
template <int BY, int GROUPS, int N>
__device__ __noinline__ void rank_close(const RouteParams& P, const float* row, const float* row_c, float2* win,
                                        uint8_t* list, float most, bool groups_close) {
  const int lane = threadIdx.x & 31;
  if (BY == BY_LOGIT || (GROUPS == ANY_GROUPS && groups_close)) return rank_all<BY != BY_LOGIT>(P, row, win);
  float c[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) c[i] = lane * kVals < N ? row_c[lane * kVals + i] : NAN;
  float top = 0.f;
  double sum = 1.0;
  if (BY == BY_SOFTMAX) {
    top = -INFINITY;
    for (int e = lane; e < P.E; e += 32) top = fmaxf(top, row[e]);
    top = lanes_max<32>(top);
    sum = 0.0;
#pragma unroll 1
    for (int e = lane; e < P.E; e += 32) sum += exp(static_cast<double>(row[e]) - top);
    sum = warp_sum(sum);
  }
  // First (groups_close) each group's largest, which decide the groups, then what
  // is at least as large as the k-th.
  bool by_group = GROUPS == LANE_GROUPS && groups_close;
  float kth = -INFINITY, from;
  if (by_group) {
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVals; ++i) top_two(a, b, c[i], -INFINITY);
    for (int off = 1; off < P.lanes_of_group; off <<= 1) {
      const float a2 = __shfl_xor_sync(kAll, a, off), b2 = __shfl_xor_sync(kAll, b, off);
      top_two(a, b, a2, b2);
    }
    const float edge = P.group_top == 2 ? b : a;
    from = edge - slack_of<BY>(most, edge);
  } else {
    kth = win[P.k - 1].x;
    __syncwarp();
    if (kth == -INFINITY) return rank_all<true>(P, row, win);
    from = kth - slack_of<BY>(most, kth);
  }
  int n, mine;
  uint64_t key;
#pragma unroll 1
  while (true) {
    // the experts with c at least `from`: their number; lane n gets the n-th and its key
    n = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const bool w = c[i] >= from && c[i] != -INFINITY;
      const unsigned who = __ballot_sync(kAll, w);
      const int at = n + __popc(who & ((1u << lane) - 1u));
      if (w && at < 32) list[at] = static_cast<uint8_t>(lane * kVals + i);
      n += __popc(who);
    }
    __syncwarp();
    if (n > 32) return rank_all<true>(P, row, win);
    mine = lane < n ? list[lane] : -1;
    const double z = row[lane < n ? mine : 0];
    const double x = exp(BY == BY_SIGMOID ? -z : z - top);
    double v = BY == BY_SIGMOID ? 1.0 / (1.0 + x) : x / sum;
    if (P.bias != nullptr && lane < n) v += static_cast<double>(P.bias[mine]);
    key = lane < n ? key_of(v) : 0;
    __syncwarp();
    if (!by_group) break;
    by_group = false;
    uint64_t best = 0, second = 0;                     // of group `lane`
    const int group = mine < 0 ? -1 : mine / kVals / P.lanes_of_group;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += 4) {
#pragma unroll
      for (int i = i0; i < i0 + 4; ++i) {              // past n: key 0, group -1
        const uint64_t u = __shfl_sync(kAll, key, i);
        if (__shfl_sync(kAll, group, i) == lane) {
          second = max(second, min(best, u));
          best = max(best, u);
        }
      }
    }
    const uint64_t score = P.group_top == 2 && second != 0 ? key_of(of_key(best) + of_key(second)) : best;
    int ahead = 0;
#pragma unroll 1
    for (int g0 = 0; g0 < P.groups; g0 += 4) {
#pragma unroll
      for (int g = g0; g < g0 + 4; ++g) {              // past the last: score 0, and behind
        const uint64_t u = __shfl_sync(kAll, score, g);
        ahead += u > score || (u == score && g < lane);
      }
    }
    const unsigned kept = __ballot_sync(kAll, lane < P.groups && ahead < P.top_groups);
    const bool in = lane / P.lanes_of_group < 32 && (kept >> (lane / P.lanes_of_group) & 1u);
    int live = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      if (!in) c[i] = NAN;
      live += c[i] > -INFINITY;
    }
    if (static_cast<int>(__reduce_add_sync(kAll, live)) < P.k) return rank_all<true>(P, row, win);
    // the k-th largest value of what is left (values that stand twice count once, which leaves more candidates)
#pragma unroll 1
    for (int j = 0; j < P.k; ++j) {
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (j == 0 || c[i] < kth) m = fmaxf(m, c[i]);
      kth = lanes_max<32>(m);
    }
    if (kth == -INFINITY) return rank_all<true>(P, row, win);
    from = kth - slack_of<BY>(most, kth);
  }
  int ahead = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 4) {
#pragma unroll
    for (int i = i0; i < i0 + 4; ++i) {                // past n: key 0
      const uint64_t u = __shfl_sync(kAll, key, i);
      const int o = __shfl_sync(kAll, mine, i);
      ahead += u > key || (u == key && o < mine);
    }
  }
  if (lane < n && ahead < P.k) win[ahead].y = __int_as_float(mine);
  __syncwarp();
}

// A warp takes NB tokens: first LPT lanes to a token rank its experts and pick k
// heads, which leaves (value, lane) pairs in shared memory; then KP lanes to a
// token, one to a choice, find the ids and make the weights (KP: k rounded up to
// a power of two), so that this part's cost is shared by 32 / KP tokens.
//
// Error of a score, in units of 2^-24: a sigmoid s = 1 / (1 + t) moves by s (1 -
// s) <= 1/4 of t's relative error, which is 1.5 |z| + 2.83 (|z| s (1 - s) <=
// 0.224), and by 3 s in addition and reciprocal: 4.1 in all; relative to s, with
// |z| <= 88, 138.  A softmax: e^d (d <= 0) is off by (2.5 |d| + 2.83) e^d <= 3.8,
// the sum by 30 of itself (the mean of |d| over a softmax of 256 is below 5.6; 13
// additions), reciprocal and product 3: 37 of the largest score; relative to a
// score, with |d| <= 88, 256.  c = s + bias adds a rounding of c, 2^-24 |c|: of the
// numbers compared, not of the largest bias (by which one bias of -1e9 sent every
// token to 64 bits, 65536 x 256 took 1050 us).
template <int LPT, int BY, int GROUPS>
__global__ void __launch_bounds__(kThreads, 3) route_scores_kernel(const __grid_constant__ RouteParams P) {
  constexpr bool SCORED = BY != BY_LOGIT;
  constexpr int TPW = 32 / LPT;                                 // tokens at a time
  constexpr int NB = TPW > 4 ? TPW : 4;                         // tokens of the warp
  constexpr int MOST = LPT * kVals < 32 ? LPT * kVals : 32;     // choices of a token
  constexpr float kTiny = 1e-37f;                               // below that scores have no relative error
  struct __align__(16) Shared {
    float c[NB][LPT * kVals];           // what ranks a token's experts
    float h[32][kList];                 // the same, each lane's in descending order, then -inf
    // a token's choices; then the best value left out and whether to rank again; the softmax's maximum and 1 / sum
    float2 win[NB][MOST + 2];
  };
  __shared__ Shared s_all[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const unsigned mask = group_mask<LPT>(lane), ahead = mask & ((1u << lane) - 1u);
  Shared& S = s_all[warp];
  S.h[lane][kVals] = -INFINITY;
  const bool softmax = P.score == SOFTMAX;
  const bool ragged = P.E < LPT * kVals;

  __shared__ __align__(16) float s_bias[SCORED ? LPT * kVals : 4];
  float reach = 0.f;                                            // largest |bias|
  float apart = 0.f;                                            // at least apart_of every group of whole lanes
  if constexpr (SCORED) {
    for (int e = threadIdx.x; e < LPT * kVals; e += kThreads) {
      float b = P.bias != nullptr && e < P.E ? P.bias[e] : 0.f;
      s_bias[e] = b != b ? -INFINITY : b;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const float b = fabsf(s_bias[gl * kVals + i]);
      if (b < INFINITY) reach = fmaxf(reach, b);
    }
    reach = lanes_max<LPT>(reach);
    if (GROUPS == LANE_GROUPS && P.group_top == 2) {
      // s lies in [0, 1], and c between the least bias and 1 + the largest: found for each token, it took 4 us of 43
      float lo = 0.f, hi = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        const float b = s_bias[gl * kVals + i];
        if (fabsf(b) < INFINITY) lo = fminf(lo, b), hi = fmaxf(hi, b);
      }
      for (int off = 1; off < P.lanes_of_group; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(kAll, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, off));
      }
      apart = lanes_max<LPT>(fmaxf(fminf(1.f + hi, -lo), 0.f));
    }
  }

  // the warp's share of the tokens, NB at a time
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps, me = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t end = (me + 1) * P.T / warps;
  int64_t t0 = me * P.T / warps;
  unsigned undecided = 0;                                       // tokens of the set that fp32 cannot decide
  float z[kVals];
  const auto load = [&](int64_t t) {                            // past the share: some token of it
    const float* row = P.logits + min(t, end - 1) * P.E;
    if (P.E % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kVals; i += 4) {
        const int e = gl * kVals + i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < P.E) v = *reinterpret_cast<const float4*>(row + e);
        z[i] = v.x, z[i + 1] = v.y, z[i + 2] = v.z, z[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) z[i] = gl * kVals + i < P.E ? row[gl * kVals + i] : 0.f;
    }
  };
  if (t0 < end) load(t0 + grp);
#pragma unroll 1
  while (true) {
#pragma unroll 1
  for (; t0 < end; t0 += NB) {
  const int ntok = static_cast<int>(min(static_cast<int64_t>(NB), end - t0));
  __syncwarp();                                                 // the last tokens' rows have been read
#pragma unroll 1
  for (int n0 = 0; n0 < ntok; n0 += TPW) {
    const int n = n0 + grp;
    float2* win = S.win[n];
    float* row_c = S.c[n];
    float probe = 0.f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) probe = fmaf(z[i], 0.f, probe);
    const bool odd = __any_sync(kAll, probe != probe);          // an infinity or a NaN among the warp's logits

    float h[kVals];                                             // what ranks the experts
    float top = 0.f, inv = 1.f;
    if (BY == BY_SOFTMAX || (BY == BY_LOGIT && softmax && !P.renorm)) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (!ragged || gl * kVals + i < P.E) top = fmaxf(top, z[i]);
      top = lanes_max<LPT>(top);
      if (top == -INFINITY) top = 0.f;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        h[i] = !ragged || gl * kVals + i < P.E ? exp_fast(z[i] - top) : 0.f;
        sum += h[i];
      }
      sum = lanes_sum<LPT>(sum);
      inv = sum == 0.f ? 0.f : 1.f / sum;
    }
    if constexpr (BY == BY_LOGIT) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) h[i] = z[i];
    } else {
#pragma unroll
      for (int i = 0; i < kVals; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(s_bias + gl * kVals + i);
        const float bias[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int m = i; m < i + 4; ++m)
          h[m] = BY == BY_SIGMOID ? rcp_fast(1.f + exp_fast(-z[m])) + bias[m - i] : fmaf(h[m], inv, bias[m - i]);
      }
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (z[i] == -INFINITY || h[i] != h[i]) h[i] = -INFINITY;
    }
    if (ragged) {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (gl * kVals + i >= P.E) h[i] = -INFINITY;
    }
    load(t0 + n + TPW);                                         // on its way while this token is ranked
#pragma unroll
    for (int i = 0; i < kVals; i += 4)
      *reinterpret_cast<float4*>(row_c + gl * kVals + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    sort8(h);
    bool close = false;                                         // a decision that fp32 cannot take

    if constexpr (GROUPS != NO_GROUPS) {
      float worst = -INFINITY, next;
      uint32_t out;                                             // of the lane's experts, those that take no part
      if constexpr (GROUPS == LANE_GROUPS) {
        float a = h[0], b = h[1];
        for (int off = 1; off < P.lanes_of_group; off <<= 1) {
          const float a2 = __shfl_xor_sync(kAll, a, off), b2 = __shfl_xor_sync(kAll, b, off);
          top_two(a, b, a2, b2);
        }
        const float score = P.group_top == 2 && b != -INFINITY ? a + b : a;
        float cur = score;
#pragma unroll 4
        for (int r = 0; r < P.top_groups; ++r) {
          worst = lanes_max<LPT>(cur);
          if (cur == worst) cur = -INFINITY;
        }
        next = lanes_max<LPT>(cur);
        const bool keep = score >= worst, first = (gl & (P.lanes_of_group - 1)) == 0 && gl * kVals < P.E;
        if (__popc(__ballot_sync(kAll, keep && first) & mask) != P.top_groups) close = true;     // equal scores
        out = keep ? 0u : 0xffu;
        if (!keep) h[0] = -INFINITY;                            // and no more comes behind it (end_of_list)
      } else {
        const Kept kept = kept_groups<LPT>(P, row_c, reinterpret_cast<float*>(win), 2 * (MOST + 2), lane);
        worst = kept.worst;
        next = kept.next;
        apart = kept.apart;
        close = kept.close;
        out = ~kept.experts;
#pragma unroll
        for (int i = 0; i < kVals; ++i) h[i] = (kept.experts >> i & 1u) ? row_c[gl * kVals + i] : -INFINITY;
        sort8(h);
      }
      if (worst == -INFINITY) close = true;                     // groups without an expert left
      if constexpr (SCORED) {
        // a sum's error: two numbers' and the rounding of the sum; |a| + |b| is at most |a + b| + 2 apart.  Both sums'
        // are 4 times that of one number with a |c| of at + apart
        const float at = fmaxf(size_of(worst), size_of(next));
        const float scores = 4.02f * (error_of<BY>(BY == BY_SOFTMAX ? inv : 1.f, 0.f) + kU * apart);
        if (!(fminf(worst, FLT_MAX) - next > fmaf(4.02f * kU, at, scores))) close = true;
      }
      // experts that take no part are found neither by their values nor by rank_close
      if (SCORED && GROUPS == LANE_GROUPS && !close && out != 0) {
#pragma unroll
        for (int i = 0; i < kVals; i += 4)
          *reinterpret_cast<float4*>(row_c + gl * kVals + i) = make_float4(NAN, NAN, NAN, NAN);
      }
      if (GROUPS == ANY_GROUPS && !close) {
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if (out >> i & 1u) row_c[gl * kVals + i] = NAN;
      }
    }

    // the rounds: the lowest lane with the largest head gives it, and takes its next from shared memory
    float* list = S.h[lane];
#pragma unroll
    for (int i = 0; i < kVals; i += 4)
      *reinterpret_cast<float4*>(list + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    float head = h[0];
    const uint32_t end_of_list = smem_u32(list) + 4 * kVals;
    uint32_t at = GROUPS == LANE_GROUPS && h[0] == -INFINITY ? end_of_list : smem_u32(list);
    const uint32_t to = smem_u32(win);
#pragma unroll 4
    for (int j = 0; j < P.k; ++j) take(head, at, end_of_list, to + 8 * j, lanes_max<LPT>(head), gl, ahead);
    const float left = SCORED ? lanes_max<LPT>(head) : -INFINITY;
    if (gl == 0) {
      win[P.k] = make_float2(left, close ? 1.f : 0.f);
      win[P.k + 1] = make_float2(top, inv);
    }
  }
  __syncwarp();

  int kp_log = 0;
  while ((1 << kp_log) < P.k) ++kp_log;
  const int kp = 1 << kp_log;
#pragma unroll 1
  for (int n0 = 0; n0 < ntok; n0 += 32 >> kp_log) {
    const int j = lane & (kp - 1), n = n0 + (lane >> kp_log);
    const bool here = n < ntok && j < P.k;
    const int nn = n < ntok ? n : 0, jj = here ? j : 0;
    const float* row = P.logits + (t0 + nn) * P.E;
    const float2* win = S.win[nn];
    const float v = win[jj].x, top = win[P.k + 1].x, inv = win[P.k + 1].y;
    const int o = __float_as_int(win[jj].y);
    const bool groups_close = win[P.k].y != 0.f;
    bool close = groups_close || v == -INFINITY;                // or fewer than k experts are left
    int skip = 0;
    if constexpr (SCORED) {
      // an absolute bound on the error of a score, and one relative to it (which is at most |c| + reach)
      const float abs_err = BY == BY_SOFTMAX ? 37.f * kU * inv : 4.1f * kU;
      const float rel_err = BY == BY_SOFTMAX ? 256.f * kU : 138.f * kU;
      const float w = win[jj + 1].x, at = fmaxf(size_of(v), size_of(w));
      if (!(v - w > 2.01f * (fminf(abs_err, rel_err * (at + reach)) + kU * at) + kTiny)) close = true;
    } else {
      // equal logits of one lane, chosen one after another
      while (skip < jj && win[jj - 1 - skip].x == v && __float_as_int(win[jj - 1 - skip].y) == o) ++skip;
    }
    const float* row_c = S.c[nn] + o * kVals;
    float c[kVals];
#pragma unroll
    for (int i = 0; i < kVals; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(row_c + i);
      c[i] = q.x, c[i + 1] = q.y, c[i + 2] = q.z, c[i + 3] = q.w;
    }
    int idx = 0;
#pragma unroll
    for (int i = kVals - 1; i >= 0; --i)
      if (c[i] == v) idx = i;
    if (!SCORED && skip != 0) {
      for (idx = 0; idx < kVals - 1; ++idx)
        if (row_c[idx] == v && skip-- == 0) break;
    }
    int sel = o * kVals + idx;
    unsigned who = __ballot_sync(kAll, here && close);
    while (who != 0) {
      const int place = (__ffs(who) - 1) >> kp_log;             // the token's among the 32 / kp
      who &= ~((kp == 32 ? kAll : (1u << kp) - 1u) << (place << kp_log));
      undecided |= 1u << (n0 + place);
    }
    const float w = weight_of(P, here ? row[sel] : -INFINITY, kp, top, inv);
    if (here) {
      P.ids[(t0 + n) * P.k + j] = sel;
      P.probs[(t0 + n) * P.k + j] = w;
    }
  }
  if (undecided != 0) break;
  }
  if (undecided == 0) return;
  do {
    const int n = __ffs(undecided) - 1;
    undecided &= undecided - 1;
    const float* row = P.logits + (t0 + n) * P.E;
    float2* win = S.win[n];
    __syncwarp();
    const float2 stat = win[P.k + 1];
    rank_close<BY, GROUPS, LPT * kVals>(P, row, S.c[n], win, reinterpret_cast<uint8_t*>(S.h), stat.y,
                                        win[P.k].y != 0.f);
    const int sel = __float_as_int(win[lane < P.k ? lane : 0].y);
    const float w = weight_of(P, lane < P.k ? row[sel] : -INFINITY, 32, stat.x, stat.y);
    if (lane < P.k) {
      P.ids[(t0 + n) * P.k + lane] = sel;
      P.probs[(t0 + n) * P.k + lane] = w;
    }
  } while (undecided != 0);
  t0 += NB;
  }
}

struct RouteBwdParams {
  const float* logits;
  const int32_t* ids;
  const float* probs;
  const float* dprobs;
  const float* dlogits_in;
  float* dlogits;
  int T, E, k;
  int score, renorm;
  float inv_scale;
  int32_t* status;
};

// A warp takes NB tokens.  KP lanes to a token, one to a choice, make the chosen
// experts' gradients; LPT lanes to a token lay down what every expert gets, in
// rows of shared memory, where the choices are added; and the rows leave in
// 16-byte pieces.  (With LPT lanes to a token for the choices as well, 65536 x 256
// took 31 us.)
template <int LPT>
__global__ void __launch_bounds__(kThreads, 4) route_scores_bwd_kernel(const __grid_constant__ RouteBwdParams P) {
  constexpr int TPW = 32 / LPT;
  constexpr int NB = TPW > 4 ? TPW : 4;
  constexpr int MOST = LPT * kVals < 32 ? LPT * kVals : 32;
  __shared__ __align__(16) float s_row[kWarps][NB][LPT * kVals];
  __shared__ __align__(8) float2 s_pick[kWarps][NB][MOST];      // expert (-1: none) and gradient of a choice
  __shared__ float s_inner[kWarps][NB];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * NB;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(NB), P.T - t0));
  if (ntok <= 0) return;
  const bool dense = P.score == SOFTMAX && !P.renorm, vec = P.E % 4 == 0;
  int kp_log = 0;
  while ((1 << kp_log) < P.k) ++kp_log;
  const int kp = 1 << kp_log;

#pragma unroll 1
  for (int n0 = 0; n0 < ntok; n0 += 32 >> kp_log) {
    const int j = lane & (kp - 1), n = n0 + (lane >> kp_log);
    const bool here = n < ntok && j < P.k;
    const int64_t at = (t0 + n) * P.k + j;
    int e = here ? P.ids[at] : -1;
    const float p = here ? P.probs[at] : 0.f, dp = here ? P.dprobs[at] : 0.f;
    const bool valid = static_cast<unsigned>(e) < static_cast<unsigned>(P.E);
    float z = 0.f;
    if (P.score == SIGMOID && valid) z = P.logits[(t0 + n) * P.E + e];
    if (here && !valid) report(P.status, MXG_ERR_EXPERT_ID);
    // sum of p_i (dp_i - dp_0), or of p_i dp_i where the weights are not renormalised
    const float first = P.renorm ? __shfl_sync(kAll, dp, lane & ~(kp - 1)) : 0.f;
    float inner = here ? p * (dp - first) : 0.f;
    for (int off = kp >> 1; off > 0; off >>= 1) inner += __shfl_xor_sync(kAll, inner, off);
    float g = p * ((dp - first) - (P.renorm ? inner * P.inv_scale : 0.f));
    if (P.score == SIGMOID) g *= sigmoid_of(-z);
    // an id that stands twice: the first adds up all of them, in their order
    const unsigned same = __match_any_sync(kAll, here && valid ? (lane >> kp_log) * 256 + e : -1 - lane);
    if (__any_sync(kAll, (same & (same - 1)) != 0)) {
      float sum = 0.f;
      for (int l = 0; l < 32; ++l) {
        const float o = __shfl_sync(kAll, g, l);
        if (same >> l & 1u) sum += o;
      }
      g = sum;
      if ((same & ((1u << lane) - 1u)) != 0) e = -1;
    }
    if (here) s_pick[warp][n][j] = make_float2(__int_as_float(valid ? e : -1), g);
    if (here && j == 0) s_inner[warp][n] = inner;
  }
  __syncwarp();

  const auto expert = [&](int i) { return vec ? 4 * (gl + LPT * (i >> 2)) + (i & 3) : gl + LPT * i; };
  const auto load = [&](const float* row, float fill, float (&v)[kVals]) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < kVals; i += 4) {
        float4 q = make_float4(fill, fill, fill, fill);
        if (expert(i) < P.E) q = *reinterpret_cast<const float4*>(row + expert(i));
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) v[i] = expert(i) < P.E ? row[expert(i)] : fill;
    }
  };
#pragma unroll 1
  for (int n0 = 0; n0 < ntok; n0 += TPW) {
    const int n = n0 + grp;
    const int64_t row = (t0 + (n < ntok ? n : 0)) * P.E;
    float d[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) d[i] = 0.f;
    if (P.dlogits_in != nullptr) load(P.dlogits_in + row, 0.f, d);
    if (dense) {
      float z[kVals], top = -INFINITY, sum = 0.f;
      load(P.logits + row, -INFINITY, z);
#pragma unroll
      for (int i = 0; i < kVals; ++i) top = fmaxf(top, z[i]);
      top = lanes_max<LPT>(top);
      if (top == -INFINITY) top = 0.f;
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        z[i] = expf(z[i] - top);
        sum += z[i];
      }
      sum = lanes_sum<LPT>(sum);
      const float f = sum == 0.f ? 0.f : s_inner[warp][n < ntok ? n : 0] / sum;
#pragma unroll
      for (int i = 0; i < kVals; ++i) d[i] = fmaf(-z[i], f, d[i]);
    }
    float* mine = s_row[warp][n];
    if (vec) {
#pragma unroll
      for (int i = 0; i < kVals; i += 4)
        *reinterpret_cast<float4*>(mine + expert(i)) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) mine[expert(i)] = d[i];
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int n0 = 0; n0 < ntok; n0 += 32 >> kp_log) {
    const int j = lane & (kp - 1), n = n0 + (lane >> kp_log);
    if (n < ntok && j < P.k) {
      const float2 pick = s_pick[warp][n][j];
      const int e = __float_as_int(pick.x);
      if (e >= 0) s_row[warp][n][e] += pick.y;
    }
  }
  __syncwarp();
#pragma unroll 1
  for (int n0 = 0; n0 < ntok; n0 += TPW) {
    const int n = n0 + grp;
    if (n >= ntok) break;
    float* out = P.dlogits + (t0 + n) * P.E;
    const float* mine = s_row[warp][n];
    if (vec) {
#pragma unroll
      for (int i = 0; i < kVals; i += 4)
        if (expert(i) < P.E) *reinterpret_cast<float4*>(out + expert(i)) = *reinterpret_cast<const float4*>(mine + expert(i));
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (expert(i) < P.E) out[expert(i)] = mine[expert(i)];
    }
  }
}

int lanes_per_token(int E) {
  int l = 1;
  while (l * kVals < E) l *= 2;
  return l;
}

// Calls f with the number as a compile-time one.
template <typename F>
void with_lanes(int E, F f) {
  switch (lanes_per_token(E)) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 8: f(std::integral_constant<int, 8>{}); break;
    case 16: f(std::integral_constant<int, 16>{}); break;
    default: f(std::integral_constant<int, 32>{}); break;
  }
}
template <typename F>
void with_three(int n, F f) {
  switch (n) {
    case 0: f(std::integral_constant<int, 0>{}); break;
    case 1: f(std::integral_constant<int, 1>{}); break;
    default: f(std::integral_constant<int, 2>{}); break;
  }
}

// Blocks for T tokens, each warp taking what its lanes hold at once.
unsigned token_blocks(int T, int E) {
  const int64_t per = static_cast<int64_t>(kWarps) * (32 / lanes_per_token(E));
  return static_cast<unsigned>((T + per - 1) / per);
}

int route_shape(int T, int E, int k, int score, float scale) {
  if (T <= 0 || E <= 0 || k <= 0) return MXG_ERR_ARG;
  if (score != MXG_SCORE_SOFTMAX && score != MXG_SCORE_SIGMOID) return MXG_ERR_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MXG_ERR_ARG;
  if (k > E || E > 256 || k > 32) return MXG_ERR_SHAPE;
  return MXG_OK;
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" int mxg_route_scores_fwd(const mxg_route_scores_fwd_args* A, void* stream) {
  if (!A || !A->logits || !A->ids || !A->probs) return MXG_ERR_ARG;
  const int T = A->T, E = A->E, k = A->k, groups = A->groups, top_groups = A->top_groups, group_top = A->group_top;
  if (const int err = route_shape(T, E, k, A->score, A->scale)) return err;
  if (groups <= 0 || top_groups <= 0 || (group_top != 1 && group_top != 2)) return MXG_ERR_ARG;
  if (groups > E || E % groups != 0 || top_groups > groups) return MXG_ERR_SHAPE;
  const int size = E / groups;
  if (k > top_groups * size || (groups > 1 && group_top > size)) return MXG_ERR_SHAPE;
  if (!api::aligned32(A->logits) || !api::aligned32(A->bias) || !api::aligned32(A->ids) || !api::aligned32(A->probs))
    return MXG_ERR_ALIGN;
  api::NvtxRange nvtx("mxg.route_scores_fwd");
  const int lanes = lanes_per_token(E);
  RouteParams p{A->logits, A->bias, T,    E, k, A->score,            groups,   top_groups, group_top,
                size,      0,       1,    A->renormalize != 0, A->scale, A->ids,   A->probs};
  const int whole = size % kVals == 0 ? size / kVals : 0;
  if ((whole & (whole - 1)) == 0) p.lanes_of_group = whole;
  while (2 * p.spread * groups <= lanes) p.spread *= 2;
  const bool scored = A->bias != nullptr || (top_groups < groups && group_top == 2);
  const int by = !scored ? BY_LOGIT : A->score == SIGMOID ? BY_SIGMOID : BY_SOFTMAX;
  const int kind = top_groups == groups ? NO_GROUPS : p.lanes_of_group != 0 ? LANE_GROUPS : ANY_GROUPS;
  // all that fit at once (three blocks an SM), fewer where a warp would get less than a set of tokens
  const unsigned most = 3 * 152, need = token_blocks(T, E), grid = need < most ? need : most;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  with_lanes(E, [&](auto l) {
    with_three(by, [&](auto b) {
      with_three(kind, [&](auto g) { route_scores_kernel<l.value, b.value, g.value><<<grid, kThreads, 0, st>>>(p); });
    });
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}

extern "C" int mxg_route_scores_bwd(const mxg_route_scores_bwd_args* A, void* stream) {
  if (!A || !A->logits || !A->ids || !A->probs || !A->dprobs || !A->dlogits || !A->dev_status) return MXG_ERR_ARG;
  const int T = A->T, E = A->E;
  if (const int err = route_shape(T, E, A->k, A->score, A->scale)) return err;
  if (!api::aligned32(A->logits) || !api::aligned32(A->ids) || !api::aligned32(A->probs) ||
      !api::aligned32(A->dprobs) || !api::aligned32(A->dlogits_in) || !api::aligned32(A->dlogits))
    return MXG_ERR_ALIGN;
  api::NvtxRange nvtx("mxg.route_scores_bwd");
  const RouteBwdParams p{A->logits, A->ids, A->probs, A->dprobs, A->dlogits_in,        A->dlogits,      T,
                         E,         A->k,   A->score, A->renormalize != 0, 1.f / A->scale, A->dev_status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  with_lanes(E, [&](auto l) {
    constexpr int at_once = 32 / l.value, set = kWarps * (at_once > 4 ? at_once : 4);
    route_scores_bwd_kernel<l.value><<<static_cast<unsigned>((static_cast<int64_t>(T) + set - 1) / set), kThreads, 0, st>>>(p);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}
