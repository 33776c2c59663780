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
#include <climits>
#include <cmath>
#include <type_traits>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"

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
  int reps;             // tokens a lane group takes one after another
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
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}

// The choice for one token by the whole warp, all in fp64: lane j gets the j-th id.
template <bool SCORED>
__device__ __noinline__ int route_exact(const RouteParams& P, int64_t t) {
  const int lane = threadIdx.x & 31;
  const float* row = P.logits + t * P.E;
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
  int id = 0;                                          // k <= 32: lane j keeps the j-th choice
  for (int j = 0; j < P.k; ++j) {
    int e;
    warp_best(key, there, lane, &e);
    if (e / kVals == lane) there &= ~(1u << (e % kVals));
    if (lane == j) id = e;
  }
  return id;
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
// The sigmoid of a weight: relative error at most 6 x 2^-24.
__device__ __forceinline__ float sigmoid_of(float z) {
  const float t = expf(-fabsf(z));
  return (z >= 0.f ? 1.f : t) / (1.f + t);
}

// Descending.
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

// LPT lanes per token.  SCORED: ranked by scores (with a bias, or sums over
// groups), else by the logits, whose order is exact.
//
// Error of a score, in units of 2^-24: a sigmoid s = 1 / (1 + t) moves by s (1 -
// s) <= 1/4 of t's relative error, which is 1.5 |z| + 2.83 (|z| s (1 - s) <=
// 0.224), and by 3 s in addition and reciprocal: 4.1 in all; relative to s, with
// |z| <= 88, 138.  A softmax: e^d (d <= 0) is off by (2.5 |d| + 2.83) e^d <= 3.8,
// the sum by 30 of itself (the mean of |d| over a softmax of 256 is below 5.6; 13
// additions), reciprocal and product 3: 37 of the largest score; relative to a
// score, with |d| <= 88, 256.  c = s + bias adds a rounding of c.
template <int LPT, bool SCORED, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) route_scores_kernel(const RouteParams P) {
  constexpr int TPW = 32 / LPT;
  constexpr int SEL = 32 / LPT < kVals ? 32 / LPT : kVals;      // choices a lane keeps
  constexpr int MOST = LPT * kVals < 32 ? LPT * kVals : 32;     // choices of a token
  constexpr float kU = 1.f / 16777216.f;                        // 2^-24
  constexpr float kTiny = 1e-37f;                               // below that scores have no relative error
  __shared__ __align__(16) float s_c[kWarps][32 * kVals];
  __shared__ __align__(8) float2 s_v[kWarps][TPW][MOST + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const unsigned mask = group_mask<LPT>(lane);
  const bool softmax = P.score == SOFTMAX;
  const bool ragged = P.E < LPT * kVals;
  float* row_c = s_c[warp] + grp * LPT * kVals;
  float2* win = s_v[warp][grp];

  float bias[kVals];
  float reach = 0.f;                                            // largest |bias|
  if constexpr (SCORED) {
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int e = gl * kVals + i;
      bias[i] = P.bias != nullptr && e < P.E ? P.bias[e] : 0.f;
      if (bias[i] != bias[i]) bias[i] = -INFINITY;
      if (fabsf(bias[i]) < INFINITY) reach = fmaxf(reach, fabsf(bias[i]));
    }
    reach = lanes_max<LPT>(reach);
  }

  int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * P.reps * TPW + grp;
  for (int n = 0; n < P.reps; ++n, t += TPW) {
    if (t - grp >= P.T) return;                                 // the whole warp
    const bool in = t < P.T;
    const float* row = P.logits + (in ? t : 0) * P.E;
    float z[kVals];
    if constexpr (VEC) {
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
    float probe = 0.f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) probe = fmaf(z[i], 0.f, probe);
    const bool odd = __any_sync(kAll, probe != probe);          // an infinity or a NaN among the warp's logits

    // h: what ranks the experts
    float h[kVals];
    float top = 0.f, inv = 1.f;
    if (softmax && (SCORED || !P.renorm)) {
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
    if constexpr (SCORED) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) h[i] = (softmax ? h[i] * inv : rcp_fast(1.f + exp_fast(-z[i]))) + bias[i];
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) h[i] = z[i];
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
    __syncwarp();                                               // the last token's rows have been read
#pragma unroll
    for (int i = 0; i < kVals; i += 4)
      *reinterpret_cast<float4*>(row_c + gl * kVals + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
    sort8(h);
    // an absolute bound on the error of a score, and one relative to it (its size is at most |c| + reach)
    const float abs_err = softmax ? 37.f * kU * inv : 4.1f * kU;
    const float rel_err = softmax ? 256.f * kU : 138.f * kU;
    bool close = false;                                         // a decision that fp32 cannot take

    if (P.top_groups < P.groups) {
      float worst = -INFINITY, next;
      if (P.lanes_of_group != 0) {
        float a = h[0], b = h[1];
        for (int off = 1; off < P.lanes_of_group; off <<= 1) {
          const float a2 = __shfl_xor_sync(kAll, a, off), b2 = __shfl_xor_sync(kAll, b, off);
          top_two(a, b, a2, b2);
        }
        const float score = P.group_top == 2 && b != -INFINITY ? a + b : a;
        float cur = score;
        for (int r = 0; r < P.top_groups; ++r) {
          worst = lanes_max<LPT>(cur);
          if (cur == worst) cur = -INFINITY;
        }
        next = lanes_max<LPT>(cur);
        const bool keep = score >= worst, first = gl % P.lanes_of_group == 0 && gl * kVals < P.E;
        if (__popc(__ballot_sync(kAll, keep && first) & mask) != P.top_groups) close = true;     // equal scores
        if (!keep) {
#pragma unroll
          for (int i = 0; i < kVals; ++i) h[i] = -INFINITY;
        }
      } else {
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
            first[r] = g < P.groups && sub == 0;
          }
        }
        float cur[kVals];
#pragma unroll
        for (int r = 0; r < kVals; ++r) cur[r] = score[r];
        for (int m = 0; m <= P.top_groups; ++m) {
          float best = cur[0];
#pragma unroll
          for (int r = 1; r < kVals; ++r) best = fmaxf(best, cur[r]);
          next = lanes_max<LPT>(best);
          if (m == P.top_groups) break;
          worst = next;
#pragma unroll
          for (int r = 0; r < kVals; ++r)
            if (cur[r] == worst) cur[r] = -INFINITY;
        }
        int kept = 0;
#pragma unroll
        for (int r = 0; r < kVals; ++r)
          kept += __popc(__ballot_sync(kAll, first[r] && score[r] >= worst) & mask);
        if (kept != P.top_groups) close = true;
        // the scores to shared memory, where every lane finds those of its experts
        float* s_score = reinterpret_cast<float*>(s_v[warp]);
        const int per = TPW * (MOST + 1) * 2 / TPW;             // floats of a token
        float own[kVals];
        for (int lo = 0; lo < P.groups; lo += per) {
          __syncwarp();
#pragma unroll
          for (int r = 0; r < kVals; ++r) {
            const int g = (gl + LPT * r) / P.spread;
            if (first[r] && g >= lo && g < lo + per) s_score[grp * per + g - lo] = score[r];
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kVals; ++i) {
            const int g = (gl * kVals + i) / P.size;
            if (g >= lo && g < lo + per && g < P.groups) own[i] = s_score[grp * per + g - lo];
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kVals; ++i) h[i] = gl * kVals + i < P.E && own[i] >= worst ? row_c[gl * kVals + i] : -INFINITY;
        sort8(h);
      }
      if (worst == -INFINITY) close = true;                     // groups without an expert left
      if constexpr (SCORED) {
        // two scores and the rounding of c twice and of the sum
        const float err = 2.f * abs_err + 4.f * kU * (softmax ? inv + reach : 1.f + reach);
        if (!(worst - next > 2.f * err)) close = true;
      }
    }

    // the rounds; with scores one more, which shows the best of the experts left out
    __syncwarp();
    for (int j = 0; j < P.k + (SCORED ? 1 : 0); ++j) {
      const float best = lanes_max<LPT>(h[0]);
      const int owner = __ffs(__ballot_sync(kAll, h[0] == best) & mask) - 1;
      if (lane == owner) {
        win[j] = make_float2(best, __int_as_float(gl));
#pragma unroll
        for (int i = 0; i + 1 < kVals; ++i) h[i] = h[i + 1];
        h[kVals - 1] = -INFINITY;
      }
    }
    __syncwarp();
    int sel[SEL];
#pragma unroll
    for (int r = 0; r < SEL; ++r) {
      const int j = gl + r * LPT;
      sel[r] = 0;
      if (j < P.k) {
        const float v = win[j].x;
        const int o = __float_as_int(win[j].y);
        if (v == -INFINITY) close = true;                       // fewer than k experts are left
        int skip = 0;
        if constexpr (SCORED) {
          const float w = win[j + 1].x;
          const float size = fmaxf(fabsf(v), w == -INFINITY ? 0.f : fabsf(w)) + reach;
          if (!(v - w > 2.f * (fminf(abs_err, rel_err * size) + kU * size) + kTiny)) close = true;
        } else {
          // equal logits of one lane, chosen one after another
          while (skip < j && win[j - 1 - skip].x == v && __float_as_int(win[j - 1 - skip].y) == o) ++skip;
        }
        float c[kVals];
#pragma unroll
        for (int i = 0; i < kVals; i += 4) {
          const float4 q = *reinterpret_cast<const float4*>(row_c + o * kVals + i);
          c[i] = q.x, c[i + 1] = q.y, c[i + 2] = q.z, c[i + 3] = q.w;
        }
        int idx = 0;
        if constexpr (SCORED) {
#pragma unroll
          for (int i = kVals - 1; i >= 0; --i)
            if (c[i] == v) idx = i;
        } else {
#pragma unroll
          for (int i = kVals - 1; i >= 0; --i) {
            int ahead = 0;
#pragma unroll
            for (int m = 0; m < i; ++m) ahead += c[m] == v;
            if (c[i] == v && ahead == skip) idx = i;
          }
        }
        sel[r] = o * kVals + idx;
      }
    }
    unsigned again = __ballot_sync(kAll, in && close);
    while (again != 0) {
      const int l = __ffs(again) - 1;
      again &= ~group_mask<LPT>(l);
      const int id = route_exact<SCORED>(P, t - grp + l / LPT);
#pragma unroll
      for (int r = 0; r < SEL; ++r) {
        const int e = __shfl_sync(kAll, id, gl + r * LPT);
        if (grp == l / LPT && gl + r * LPT < P.k) sel[r] = e;
      }
    }

    // weights; those of a renormalised sigmoid by the largest chosen, which keeps them from vanishing together
    float w[SEL], zc[SEL];
    float low = -INFINITY;
#pragma unroll
    for (int r = 0; r < SEL; ++r) {
      zc[r] = gl + r * LPT < P.k ? row[sel[r]] : -INFINITY;
      low = fmaxf(low, zc[r]);
    }
    if (P.renorm) low = lanes_max<LPT>(low);
    float total = 0.f;
#pragma unroll
    for (int r = 0; r < SEL; ++r) {
      if (zc[r] == -INFINITY) {
        w[r] = 0.f;
      } else if (softmax) {
        w[r] = expf(zc[r] - (P.renorm ? low : top));
      } else {
        w[r] = P.renorm && low < 0.f ? expf(zc[r] - low) / (1.f + expf(zc[r])) : sigmoid_of(zc[r]);
      }
      total += w[r];
    }
    float factor = P.scale;
    if (P.renorm) {
      total = lanes_sum<LPT>(total);
      factor = total == 0.f ? 0.f : P.scale / total;
    } else if (softmax) {
      factor = P.scale * inv;
    }
    if (in) {
#pragma unroll
      for (int r = 0; r < SEL; ++r) {
        const int j = gl + r * LPT;
        if (j < P.k) {
          P.ids[t * P.k + j] = sel[r];
          P.probs[t * P.k + j] = w[r] * factor;
        }
      }
    }
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

// dlogits of a token by LPT lanes.  The lanes build the row in shared memory, the
// chosen experts' lanes add theirs there, and it leaves in 16-byte pieces.
template <int LPT, bool VEC>
__global__ void __launch_bounds__(kThreads) route_scores_bwd_kernel(const RouteBwdParams P) {
  constexpr int TPW = 32 / LPT;
  constexpr int SEL = 32 / LPT < kVals ? 32 / LPT : kVals;
  __shared__ __align__(16) float s_row[kWarps][32 * kVals];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * TPW + grp;
  if (t - grp >= P.T) return;
  const bool in = t < P.T;
  const int64_t row = (in ? t : 0) * P.E, pick = (in ? t : 0) * P.k;
  float* mine = s_row[warp] + grp * LPT * kVals;
  const auto expert = [&](int i) { return VEC ? 4 * (gl + LPT * (i >> 2)) + (i & 3) : gl + LPT * i; };
  const auto load = [&](const float* p, float fill, float (&v)[kVals]) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kVals; i += 4) {
        float4 q = make_float4(fill, fill, fill, fill);
        if (expert(i) < P.E) q = *reinterpret_cast<const float4*>(p + row + expert(i));
        v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) v[i] = expert(i) < P.E ? p[row + expert(i)] : fill;
    }
  };
  int id[SEL];
  float p[SEL], dp[SEL];
#pragma unroll
  for (int r = 0; r < SEL; ++r) {
    const int j = gl + r * LPT;
    id[r] = j < P.k ? P.ids[pick + j] : -1;
    p[r] = j < P.k ? P.probs[pick + j] : 0.f;
    dp[r] = j < P.k ? P.dprobs[pick + j] : 0.f;
  }
  float d[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) d[i] = 0.f;
  if (P.dlogits_in != nullptr) load(P.dlogits_in, 0.f, d);
  // sum of p_i (dp_i - dp_0), or of p_i dp_i where the weights are not renormalised
  const float first = P.renorm ? __shfl_sync(kAll, dp[0], grp * LPT) : 0.f;
  float inner = 0.f;
#pragma unroll
  for (int r = 0; r < SEL; ++r)
    if (gl + r * LPT < P.k) inner = fmaf(p[r], dp[r] - first, inner);
  inner = lanes_sum<LPT>(inner);
  if (P.score == SOFTMAX && !P.renorm) {
    float z[kVals], top = -INFINITY, sum = 0.f;
    load(P.logits, -INFINITY, z);
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
    const float f = sum == 0.f ? 0.f : inner / sum;
#pragma unroll
    for (int i = 0; i < kVals; ++i) d[i] = fmaf(-z[i], f, d[i]);
  }
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kVals; i += 4)
      *reinterpret_cast<float4*>(mine + expert(i)) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i) mine[expert(i)] = d[i];
  }
  __syncwarp();
  const float mean = P.renorm ? inner * P.inv_scale : 0.f;
#pragma unroll
  for (int r = 0; r < SEL; ++r) {
    const int e = id[r];
    const bool chosen = gl + r * LPT < P.k, valid = static_cast<unsigned>(e) < static_cast<unsigned>(P.E);
    if (in && chosen && !valid) report(P.status, MXG_ERR_EXPERT_ID);
    float g = p[r] * ((dp[r] - first) - mean);
    if (P.score == SIGMOID && chosen && valid) g *= sigmoid_of(-P.logits[row + e]);
    // an id that stands twice adds in its order
    const int tag = chosen && valid ? grp * 256 + e : -1 - lane;
    const unsigned same = __match_any_sync(kAll, tag);
    unsigned turn = __popc(same & ((1u << lane) - 1u));
    const unsigned turns = __reduce_max_sync(kAll, turn);
    for (unsigned n = 0; n <= turns; ++n) {
      if (tag >= 0 && turn == n) mine[e] += g;
      __syncwarp();
    }
  }
  if (in) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kVals; i += 4)
        if (expert(i) < P.E)
          *reinterpret_cast<float4*>(P.dlogits + row + expert(i)) = *reinterpret_cast<const float4*>(mine + expert(i));
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (expert(i) < P.E) P.dlogits[row + expert(i)] = mine[expert(i)];
    }
  }
}

int lanes_per_token(int E) {
  int l = 1;
  while (l * kVals < E) l *= 2;
  return l;
}

// Calls f(lanes per token, 16-byte rows).
template <typename F>
void with_lanes(int E, F f) {
  const auto vec = [&](auto l) {
    if (E % 4 == 0) f(l, std::true_type{});
    else f(l, std::false_type{});
  };
  switch (lanes_per_token(E)) {
    case 1: vec(std::integral_constant<int, 1>{}); break;
    case 2: vec(std::integral_constant<int, 2>{}); break;
    case 4: vec(std::integral_constant<int, 4>{}); break;
    case 8: vec(std::integral_constant<int, 8>{}); break;
    case 16: vec(std::integral_constant<int, 16>{}); break;
    default: vec(std::integral_constant<int, 32>{}); break;
  }
}

unsigned token_blocks(int T, int E, int reps) {
  const int64_t per = static_cast<int64_t>(kWarps) * (32 / lanes_per_token(E)) * reps;
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

extern "C" int mxg_route_scores_fwd(const float* logits, const float* bias, int T, int E, int k, int score, int groups,
                                    int top_groups, int group_top, int renormalize, float scale, int32_t* ids,
                                    float* probs, void* stream) {
  if (!logits || !ids || !probs) return MXG_ERR_ARG;
  if (const int err = route_shape(T, E, k, score, scale)) return err;
  if (groups <= 0 || top_groups <= 0 || (group_top != 1 && group_top != 2)) return MXG_ERR_ARG;
  if (groups > E || E % groups != 0 || top_groups > groups) return MXG_ERR_SHAPE;
  const int size = E / groups;
  if (k > top_groups * size || (groups > 1 && group_top > size)) return MXG_ERR_SHAPE;
  if (!api::aligned32(logits) || !api::aligned32(bias) || !api::aligned32(ids) || !api::aligned32(probs))
    return MXG_ERR_ALIGN;
  api::NvtxRange nvtx("mxg.route_scores_fwd");
  const int lanes = lanes_per_token(E);
  RouteParams p{logits, bias, T, E, k, score, groups, top_groups, group_top, size, 0, 1, renormalize != 0, scale, 1, ids,
                probs};
  const int whole = size % kVals == 0 ? size / kVals : 0;
  if ((whole & (whole - 1)) == 0) p.lanes_of_group = whole;
  while (2 * p.spread * groups <= lanes) p.spread *= 2;
  if (T >= 16384) p.reps = 4;
  const bool scored = bias != nullptr || (top_groups < groups && group_top == 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  with_lanes(E, [&](auto l, auto v) {
    const unsigned grid = token_blocks(T, E, p.reps);
    if (scored) route_scores_kernel<l.value, true, v.value><<<grid, kThreads, 0, st>>>(p);
    else route_scores_kernel<l.value, false, v.value><<<grid, kThreads, 0, st>>>(p);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}

extern "C" int mxg_route_scores_bwd(const float* logits, const int32_t* ids, const float* probs, const float* dprobs,
                                    const float* dlogits_in, int T, int E, int k, int score, int renormalize,
                                    float scale, float* dlogits, int32_t* dev_status, void* stream) {
  if (!logits || !ids || !probs || !dprobs || !dlogits || !dev_status) return MXG_ERR_ARG;
  if (const int err = route_shape(T, E, k, score, scale)) return err;
  if (!api::aligned32(logits) || !api::aligned32(ids) || !api::aligned32(probs) || !api::aligned32(dprobs) ||
      !api::aligned32(dlogits_in) || !api::aligned32(dlogits))
    return MXG_ERR_ALIGN;
  api::NvtxRange nvtx("mxg.route_scores_bwd");
  const RouteBwdParams p{logits, ids,   probs, dprobs,           dlogits_in,   dlogits,   T,
                         E,      k,     score, renormalize != 0, 1.f / scale, dev_status};
  with_lanes(E, [&](auto l, auto v) {
    route_scores_bwd_kernel<l.value, v.value>
        <<<token_blocks(T, E, 1), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}
