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
// which a decision lies within that bound is routed again in fp64 by its warp.
// With scores spread over (0, 1) that is about one token in a thousand.
//
// LPT lanes take a token, eight consecutive experts a lane.  A choice is a round
// of maxima over order-preserving integer keys: eight per lane, one across the
// lanes; the lowest lane with the largest key owns the lowest such id.
#include <cfloat>
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

enum { SOFTMAX = 0, SIGMOID = 1 };

struct RouteParams {
  const float* logits;
  const float* bias;
  int T, E, k;
  int score;
  int groups, top_groups, group_top;
  int renorm;
  float scale;
  int32_t* ids;
  float* probs;
};

// Keys that order like the numbers: -inf lowest (0x007fffff), above 0, which
// stands for "not there"; NaN ranks with -inf, -0 with +0.
__device__ __forceinline__ uint32_t key_of(float v) {
  v = v == v ? v + 0.f : -INFINITY;
  const uint32_t b = __float_as_uint(v);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (static_cast<uint32_t>(static_cast<int32_t>(~k) >> 31) | 0x80000000u));
}
constexpr uint32_t kOffKey = 0x007fffffu;      // key_of(-inf)

template <int LPT>
__device__ __forceinline__ unsigned group_mask(int lane) {
  return LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1u) << (lane & ~(LPT - 1));
}
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (LPT == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// ------------------------------------------------------------------ 64 bits --
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The largest of the warp's c[i] (expert lane + 32 i) that `there` still holds;
// ties to the lower expert.  Every lane gets the expert and the value.
__device__ __forceinline__ int warp_best(const double (&c)[kVals], uint32_t there, int lane, double* value) {
  double bv = 0.0;
  int bi = INT_MAX;
#pragma unroll
  for (int i = 0; i < kVals; ++i)
    if ((there >> i & 1u) && (bi == INT_MAX || c[i] > bv)) bv = c[i], bi = lane + 32 * i;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const double ov = __shfl_xor_sync(0xffffffffu, bv, off);
    const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
    if (oi != INT_MAX && (bi == INT_MAX || ov > bv || (ov == bv && oi < bi))) bv = ov, bi = oi;
  }
  *value = bv;
  return bi;
}

// The choice for one token by the whole warp, all in fp64: lane j gets the j-th id.
__device__ __noinline__ int route_exact(const RouteParams& P, int64_t t) {
  const int lane = threadIdx.x & 31;
  const float* row = P.logits + t * P.E;
  double s[kVals], c[kVals];
  uint32_t there = 0, live = 0;
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < P.E ? static_cast<double>(row[e]) : -INFINITY;
    if (e < P.E) there |= 1u << i;
    if (s[i] == s[i]) top = fmax(top, s[i]);
  }
  top = warp_max(top);
  if (top == -INFINITY) top = 0.0;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const bool on = s[i] != -INFINITY;                       // a NaN is on, and its score NaN
    s[i] = P.score == SIGMOID ? 1.0 / (1.0 + exp(-s[i])) : exp(s[i] - top);
    if (!on) s[i] = 0.0;
    if (on) live |= 1u << i;
    sum += s[i];
  }
  if (P.score == SOFTMAX) {
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (sum != 0.0) s[i] /= sum;
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const int e = lane + 32 * i;
    c[i] = e < P.E && P.bias != nullptr ? s[i] + static_cast<double>(P.bias[e]) : s[i];
    if (!(live >> i & 1u) || c[i] != c[i]) c[i] = -INFINITY;
  }
  if (P.top_groups < P.groups) {
    const int size = P.E / P.groups;
    double score[kVals];                                     // of group lane + 32 i
    uint32_t left = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) score[i] = -INFINITY;
    for (int g = 0; g < P.groups; ++g) {
      uint32_t in = 0;
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if ((there >> i & 1u) && (lane + 32 * i) / size == g) in |= 1u << i;
      double a, b = -INFINITY;
      const int first = warp_best(c, in, lane, &a);
      if (P.group_top == 2) {
        if ((first & 31) == lane) in &= ~(1u << (first >> 5));
        warp_best(c, in, lane, &b);
      }
      if (b != -INFINITY) a += b;
      if ((g & 31) == lane) {
        left |= 1u << (g >> 5);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if (i == g >> 5) score[i] = a;
      }
    }
    uint32_t kept = 0;                                       // of the lane's own elements
    for (int n = 0; n < P.top_groups; ++n) {
      double v;
      const int g = warp_best(score, left, lane, &v);
      if ((g & 31) == lane) left &= ~(1u << (g >> 5));
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if ((there >> i & 1u) && (lane + 32 * i) / size == g) kept |= 1u << i;
    }
    there = kept;
  }
  // k <= 32: lane j keeps the j-th choice
  int id = 0;
  for (int j = 0; j < P.k; ++j) {
    double v;
    const int e = warp_best(c, there, lane, &v);
    if ((e & 31) == lane) there &= ~(1u << (e >> 5));
    if (lane == j) id = e;
  }
  return id;
}

// --------------------------------------------------------------------- fp32 --
// Sigmoid, relative error at most 2^-21 (expf 2 ulp, an addition, a quotient).
__device__ __forceinline__ float sigmoid_of(float z) {
  const float t = expf(-fabsf(z));
  return (z >= 0.f ? 1.f : t) / (1.f + t);
}

constexpr float kTiny = 1e-37f;         // scores below the normal numbers have no relative error

// LPT lanes per token.  SCORED: ranked by scores (with a bias, or sums over
// groups), else by the logits.
template <int LPT, bool SCORED>
__global__ void __launch_bounds__(kThreads) route_scores_kernel(const RouteParams P) {
  constexpr int TPW = 32 / LPT;
  constexpr int SEL = 32 / LPT < kVals ? 32 / LPT : kVals;      // choices a lane keeps
  __shared__ float s_row[SCORED ? kWarps * TPW * LPT * kVals : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * TPW + grp;
  if (t - grp >= P.T) return;                                   // the whole warp
  const bool in = t < P.T;
  const float* row = P.logits + (in ? t : 0) * P.E;
  float z[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const int e = gl * kVals + i;
    z[i] = e < P.E ? row[e] : -INFINITY;
  }
  float top = -INFINITY, sum = 0.f, inv = 1.f;
  float s[kVals];                                               // scores, where they are needed for every expert
  const bool softmax = P.score == SOFTMAX;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < kVals; ++i) top = fmaxf(top, z[i]);
    top = lanes_max<LPT>(top);
    if (top == -INFINITY) top = 0.f;
    if (SCORED || !P.renorm) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        s[i] = expf(z[i] - top);
        sum += s[i];
      }
      sum = lanes_sum<LPT>(sum);
      inv = sum == 0.f ? 0.f : 1.f / sum;
    }
  }
  uint32_t key[kVals];
  bool close = false;                                           // a decision within the error bound
  float reach = 0.f;                                            // largest |bias|
  // relative errors of a score: the sigmoid's (see there); the softmax's is 2.75 of 2^-21 from exponential, sum and
  // quotient, and up to 88 of 2^-24 from the rounding of z - top, which the exponential magnifies
  constexpr float kU = 1.f / 2097152.f;
  const float u = softmax ? 14.f * kU : 1.1f * kU;
  if constexpr (SCORED) {
    float c[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int e = gl * kVals + i;
      const float b = P.bias != nullptr && e < P.E ? P.bias[e] : 0.f;
      if (fabsf(b) < INFINITY) reach = fmaxf(reach, fabsf(b));
      s[i] = softmax ? s[i] * inv : sigmoid_of(z[i]);
      c[i] = z[i] == -INFINITY ? -INFINITY : s[i] + b;
      if (c[i] != c[i]) c[i] = -INFINITY;
      key[i] = e < P.E ? key_of(c[i]) : 0u;
    }
    reach = lanes_max<LPT>(reach);
    if (P.top_groups < P.groups) {
      const int size = P.E / P.groups;
      float* mine = s_row + (warp * TPW + grp) * LPT * kVals;
#pragma unroll
      for (int i = 0; i < kVals; ++i) mine[gl * kVals + i] = c[i];
      __syncwarp();
      // scores of groups gl, gl + LPT, ...
      float score[kVals];
      float most = 0.f;
#pragma unroll
      for (int n = 0; n < kVals; ++n) {
        const int g = gl + n * LPT;
        float a = -INFINITY, b = -INFINITY;
        if (g < P.groups) {
          for (int i = 0; i < size; ++i) {
            const float v = mine[g * size + i];
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
        }
        if (a != -INFINITY) most = fmaxf(most, fabsf(a));
        score[n] = P.group_top == 2 && b != -INFINITY ? a + b : a;
      }
      most = lanes_max<LPT>(most);
      __syncwarp();
#pragma unroll
      for (int n = 0; n < kVals; ++n)
        if (gl + n * LPT < P.groups) mine[gl + n * LPT] = score[n];
      __syncwarp();
      // a group stays if fewer than top_groups are ahead of it
      uint32_t keep = 0;
      float worst = INFINITY, next = -INFINITY;
      for (int g = 0; g < P.groups; ++g) {
        const float v = mine[g];
        int ahead = 0;
        for (int h = 0; h < P.groups; ++h) {
          const float w = mine[h];
          ahead += w > v || (w == v && h < g);
        }
        if (ahead < P.top_groups) {
          worst = fminf(worst, v);
#pragma unroll
          for (int i = 0; i < kVals; ++i)
            if ((gl * kVals + i) / size == g) keep |= 1u << i;
        } else {
          next = fmaxf(next, v);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (!(keep >> i & 1u)) key[i] = 0u;
      // each score is a sum of at most two, each off by u (|c| + reach), and rounded
      const float err = (2.f * u + 0.5f * kU) * (most + reach) + kTiny;
      close = next != -INFINITY && worst - next <= 2.f * err;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i) key[i] = gl * kVals + i < P.E ? key_of(z[i]) : 0u;
    if (P.top_groups < P.groups) {                              // group_top 1: by the groups' largest logits
      const int size = P.E / P.groups;
      uint32_t keep = 0, gone = 0;
      for (int n = 0; n < P.top_groups; ++n) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if (!(gone >> i & 1u)) m = max(m, key[i]);
        const uint32_t best = lanes_max<LPT>(m);
        const unsigned who = __ballot_sync(0xffffffffu, m == best) & group_mask<LPT>(lane);
        const int owner = __ffs(who) - 1;
        int e = 0;
#pragma unroll
        for (int i = kVals - 1; i >= 0; --i)
          if (!(gone >> i & 1u) && key[i] == best) e = gl * kVals + i;
        e = __shfl_sync(0xffffffffu, e, owner);
#pragma unroll
        for (int i = 0; i < kVals; ++i)
          if ((gl * kVals + i) / size == e / size) {
            keep |= 1u << i;
            gone |= 1u << i;
          }
      }
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (!(keep >> i & 1u)) key[i] = 0u;
    }
  }
  // k rounds, and one more that shows the best of the experts left out
  int sel[SEL];
#pragma unroll
  for (int r = 0; r < SEL; ++r) sel[r] = 0;
  float before = INFINITY;
  for (int j = 0; j < P.k + (SCORED ? 1 : 0); ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < kVals; ++i) m = max(m, key[i]);
    const uint32_t best = lanes_max<LPT>(m);
    if constexpr (SCORED) {
      if (best > kOffKey) {
        const float v = of_key(best);
        // a score is at most |c| + reach, and c rounds once
        if (before - v <= 2.f * (u + 0.125f * kU) * (fmaxf(fabsf(before), fabsf(v)) + reach) + kTiny) close = true;
        before = v;
      }
      if (j == P.k) break;
    }
    const unsigned who = __ballot_sync(0xffffffffu, m == best) & group_mask<LPT>(lane);
    const int owner = __ffs(who) - 1;
    int idx = 0;
#pragma unroll
    for (int i = kVals - 1; i >= 0; --i)
      if (key[i] == best) idx = i;
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (lane == owner && i == idx) key[i] = 0u;
    const int e = __shfl_sync(0xffffffffu, gl * kVals + idx, owner);
#pragma unroll
    for (int r = 0; r < SEL; ++r)
      if (j == gl + r * LPT) sel[r] = e;
  }
  if constexpr (SCORED) {
    unsigned again = __ballot_sync(0xffffffffu, in && close && gl == 0);
    while (again != 0) {
      const int l = __ffs(again) - 1;
      again &= again - 1;
      const int id = route_exact(P, __shfl_sync(0xffffffffu, t, l));
#pragma unroll
      for (int r = 0; r < SEL; ++r) {
        const int e = __shfl_sync(0xffffffffu, id, gl + r * LPT);
        if (grp == l / LPT && gl + r * LPT < P.k) sel[r] = e;
      }
    }
  }
  // weights; a renormalised sigmoid is scaled by the power that keeps the largest from vanishing
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

// dlogits of a token by LPT lanes, lane gl holding experts gl + LPT i.
template <int LPT>
__global__ void __launch_bounds__(kThreads) route_scores_bwd_kernel(const RouteBwdParams P) {
  constexpr int TPW = 32 / LPT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * TPW + grp;
  if (t - grp >= P.T) return;
  const bool in = t < P.T;
  const int64_t row = (in ? t : 0) * P.E, pick = (in ? t : 0) * P.k;
  float d[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const int e = gl + LPT * i;
    d[i] = P.dlogits_in != nullptr && in && e < P.E ? P.dlogits_in[row + e] : 0.f;
  }
  // sum of p_i (dp_i - dp_0), or of p_i dp_i where the weights are not renormalised
  const float first = P.renorm ? P.dprobs[pick] : 0.f;
  float inner = 0.f;
  for (int j = gl; j < P.k; j += LPT) inner = fmaf(P.probs[pick + j], P.dprobs[pick + j] - first, inner);
  inner = lanes_sum<LPT>(inner);
  if (P.score == SOFTMAX && !P.renorm) {
    float z[kVals], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int e = gl + LPT * i;
      z[i] = e < P.E ? P.logits[row + e] : -INFINITY;
      top = fmaxf(top, z[i]);
    }
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
  const float mean = P.renorm ? inner * P.inv_scale : 0.f;
  for (int j = 0; j < P.k; ++j) {
    const int e = P.ids[pick + j];
    if (static_cast<unsigned>(e) >= static_cast<unsigned>(P.E)) {
      if (in && gl == 0) report(P.status, MXG_ERR_EXPERT_ID);
      continue;
    }
    if (e % LPT != gl) continue;
    float g = P.probs[pick + j] * ((P.dprobs[pick + j] - first) - mean);
    if (P.score == SIGMOID) g *= sigmoid_of(-P.logits[row + e]);
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (e / LPT == i) d[i] += g;
  }
  if (in) {
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int e = gl + LPT * i;
      if (e < P.E) P.dlogits[row + e] = d[i];
    }
  }
}

int lanes_per_token(int E) {
  int l = 1;
  while (l * kVals < E) l *= 2;
  return l;
}

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
  const RouteParams p{logits, bias, T, E, k, score, groups, top_groups, group_top, renormalize != 0, scale, ids, probs};
  const bool scored = bias != nullptr || (top_groups < groups && group_top == 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  with_lanes(E, [&](auto l) {
    if (scored) route_scores_kernel<l.value, true><<<token_blocks(T, E), kThreads, 0, st>>>(p);
    else route_scores_kernel<l.value, false><<<token_blocks(T, E), kThreads, 0, st>>>(p);
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
  with_lanes(E, [&](auto l) {
    route_scores_bwd_kernel<l.value><<<token_blocks(T, E), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}
