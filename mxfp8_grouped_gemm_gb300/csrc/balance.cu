// Balance loss of the router and its gradient.
//
// BioNeMo Uses Grouped Kernels and MXFP8, Fig. 1: a router sends each token to
// a few of the experts.  With p = softmax of a token's logits over all E
// experts, c_e the number of times expert e was chosen, P_e the sum of p_te
// and n the number of tokens that count (token_mask),
//   loss          = coef E sum_e (c_e / (k n)) (P_e / n)
//   dlogits[t, e] = dloss coef E / n  p_te (f_e - sum_i p_ti f_i),  f = c / (k n)
// (the counts carry no gradient).  f is near 1 / E once the router is
// balanced and the bracket a small difference of near-equal numbers, so it is
// taken on the deviations instead: f_e = (1 + d_e) / E with the integer
// numerator of d_e = (E c_e - k n) / (k n) exact, and since the p of a token
// sum to one the bracket is (d_e - sum_i p_ti d_i) / E.
//
// A token's logits are read by a group of LPT lanes, eight experts per lane
// (LPT = the power of two that covers E), so one warp handles 32 / LPT tokens
// at a time and every lane keeps its experts' sums in registers.
#include <climits>
#include <cmath>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"

namespace mxg {
namespace {

constexpr int kBlThreads = 256;
constexpr int kBlWarps = kBlThreads / 32;
constexpr int kBlVals = 8;               // experts per lane
constexpr int kBlMaxBlocks = 152;        // partial sums of the forward: one block per SM

// The group's softmax of one token: z[i] = logit of expert lane_in_group + LPT i
// (-inf past E) becomes the probability.  A row without a finite logit gives
// zeros; NaN (or +inf, as inf - inf) gives NaN in the whole row.
template <int LPT>
__device__ __forceinline__ void group_softmax(float (&z)[kBlVals]) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < kBlVals; ++i) top = fmaxf(top, z[i]);
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top == -INFINITY) top = 0.f;       // fmaxf skips NaN: a row of NaN and -inf keeps its NaN below
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) {
    z[i] = expf(z[i] - top);
    sum += z[i];
  }
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) z[i] *= inv;
}

template <int LPT>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, int gl, bool live,
                                            float (&z)[kBlVals]) {
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) {
    const int e = gl + LPT * i;
    z[i] = live && e < E ? row[e] : -INFINITY;
  }
}

// Sums of the probabilities and counts of the chosen ids over the block's
// tokens, one partial per block and expert.
template <int LPT>
__global__ void __launch_bounds__(kBlThreads) balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E,
    int k, float* __restrict__ part, int32_t* __restrict__ part_counts, int32_t* __restrict__ part_tokens,
    int32_t* status) {
  __shared__ float s_sum[kBlWarps][256];
  __shared__ int s_cnt[256];
  __shared__ int s_tok;
  constexpr int TPW = 32 / LPT;          // tokens a warp takes at once
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  for (int e = threadIdx.x; e < E; e += kBlThreads) s_cnt[e] = 0;
  if (threadIdx.x == 0) s_tok = 0;
  __syncthreads();
  float acc[kBlVals];
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) acc[i] = 0.f;
  int tokens = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kBlWarps * TPW;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kBlWarps + warp) * TPW; t0 < T; t0 += step) {
    const int64_t t = t0 + grp;
    const bool live = t < T && (mask == nullptr || mask[t] != 0);
    float z[kBlVals];
    load_logits<LPT>(logits + t * E, E, gl, live, z);
    group_softmax<LPT>(z);
#pragma unroll
    for (int i = 0; i < kBlVals; ++i) acc[i] += z[i];
    if (live) {
      tokens += gl == 0;
      for (int j = gl; j < k; j += LPT) {
        const int e = ids[t * k + j];
        if (e < 0 || e >= E) report(status, MXG_ERR_EXPERT_ID);
        else atomicAdd(&s_cnt[e], 1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) {
#pragma unroll
    for (int off = 16; off >= LPT; off >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
    if (grp == 0 && gl + LPT * i < E) s_sum[warp][gl + LPT * i] = acc[i];
  }
  if (tokens != 0) atomicAdd(&s_tok, tokens);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kBlThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBlWarps; ++w) s += s_sum[w][e];
    part[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    part_counts[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
  }
  if (threadIdx.x == 0) part_tokens[blockIdx.x] = s_tok;
}

// The partials in block order, the counts and the loss.
__global__ void __launch_bounds__(256) balance_finish_kernel(const float* __restrict__ part,
                                                            const int32_t* __restrict__ part_counts,
                                                            const int32_t* __restrict__ part_tokens, int nblk, int E,
                                                            int k, float coef, float* __restrict__ loss,
                                                            int32_t* __restrict__ counts,
                                                            float* __restrict__ prob_sums,
                                                            int32_t* __restrict__ n_tokens) {
  __shared__ float s_term[256];
  __shared__ int s_n;
  const int e = threadIdx.x;
  if (e == 0) {
    int n = 0;
    for (int b = 0; b < nblk; ++b) n += part_tokens[b];
    s_n = n;
    *n_tokens = n;
  }
  float sum = 0.f;
  int c = 0;
  if (e < E) {
    for (int b = 0; b < nblk; ++b) {
      sum += part[static_cast<int64_t>(b) * E + e];
      c += part_counts[static_cast<int64_t>(b) * E + e];
    }
    prob_sums[e] = sum;
    counts[e] = c;
  }
  __syncthreads();
  const float n = static_cast<float>(s_n);
  s_term[e] = e < E && s_n > 0 ? (static_cast<float>(c) / (static_cast<float>(k) * n)) * (sum / n) : 0.f;
  __syncthreads();
  for (int off = 128; off > 0; off >>= 1) {
    if (e < off) s_term[e] += s_term[e + off];
    __syncthreads();
  }
  if (e == 0) *loss = coef * static_cast<float>(E) * s_term[0];
}

template <int LPT>
__global__ void __launch_bounds__(kBlThreads) balance_bwd_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ n_tokens, int T, int E, int k, float coef, const float* __restrict__ dloss,
    const int32_t* __restrict__ ids, const float* __restrict__ probs, const float* __restrict__ dprobs,
    float* __restrict__ dlogits, int32_t* status) {
  constexpr int TPW = 32 / LPT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const int n = *n_tokens;
  const float up = n > 0 ? (dloss != nullptr ? *dloss : 1.f) * coef / static_cast<float>(n) : 0.f;
  // deviations of the lane's experts: (E c - k n) / (k n), the numerator exact
  float dev[kBlVals];
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) {
    const int e = gl + LPT * i;
    const int64_t kn = static_cast<int64_t>(k) * n;
    dev[i] = e < E && n > 0 ? static_cast<float>(static_cast<int64_t>(E) * counts[e] - kn) / static_cast<float>(kn)
                            : 0.f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kBlWarps * TPW;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kBlWarps + warp) * TPW; t0 < T; t0 += step) {
    const int64_t t = t0 + grp;
    const bool in = t < T;
    const bool live = in && (mask == nullptr || mask[t] != 0);
    float z[kBlVals];
    load_logits<LPT>(logits + t * E, E, gl, live, z);
    group_softmax<LPT>(z);
    float mean = 0.f;
#pragma unroll
    for (int i = 0; i < kBlVals; ++i) mean = fmaf(z[i], dev[i], mean);
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, off);
#pragma unroll
    for (int i = 0; i < kBlVals; ++i) z[i] = live ? up * z[i] * (dev[i] - mean) : 0.f;
    if (probs != nullptr) {
      // the route's gradient at the chosen experts: q_j (dq_j - sum_i q_i dq_i)
      float inner = 0.f;
      for (int j = gl; j < k; j += LPT)
        if (in) inner = fmaf(probs[t * k + j], dprobs[t * k + j], inner);
#pragma unroll
      for (int off = LPT / 2; off > 0; off >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, off);
      if (in) {
        for (int j = 0; j < k; ++j) {
          const int e = ids[t * k + j];
          if (e < 0 || e >= E) {
            if (gl == 0) report(status, MXG_ERR_EXPERT_ID);
          } else if (e % LPT == gl) {
            const float q = probs[t * k + j];
            const float d = q * (dprobs[t * k + j] - inner);
#pragma unroll
            for (int i = 0; i < kBlVals; ++i)
              if (e / LPT == i) z[i] += d;
          }
        }
      }
    }
    if (in) {
#pragma unroll
      for (int i = 0; i < kBlVals; ++i)
        if (gl + LPT * i < E) dlogits[t * E + gl + LPT * i] = z[i];
    }
  }
}

int lanes_per_token(int E) {
  int l = 1;
  while (l * kBlVals < E) l *= 2;
  return l;
}

// Blocks of a pass over T tokens: enough for one trip each, at most `most`.
int balance_blocks(int T, int E, int most) {
  const int64_t per = static_cast<int64_t>(kBlWarps) * (32 / lanes_per_token(E));
  const int64_t n = (T + per - 1) / per;
  return static_cast<int>(n < most ? n : most);
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

int64_t part_floats(int T, int E) { return api::align_up(4ll * balance_blocks(T, E, kBlMaxBlocks) * E, api::kAlign); }

int balance_shape(int T, int E, int k) {
  if (T <= 0 || E <= 0 || k <= 0) return MXG_ERR_ARG;
  if (E > 256 || k > 32 || k > E || static_cast<int64_t>(T) * k > INT32_MAX) return MXG_ERR_SHAPE;
  return MXG_OK;
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" size_t mxg_balance_loss_workspace_bytes(int T, int E) {
  if (T <= 0 || E <= 0 || E > 256) return 0;
  return static_cast<size_t>(2 * part_floats(T, E) + api::align_up(4ll * kBlMaxBlocks, api::kAlign));
}

extern "C" int mxg_balance_loss_fwd(const float* logits, const int32_t* ids, const uint8_t* token_mask, int T, int E,
                                    int k, float coef, float* loss, int32_t* counts, float* prob_sums,
                                    int32_t* n_tokens, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                    void* stream) {
  if (!logits || !ids || !loss || !counts || !prob_sums || !n_tokens || !workspace || !dev_status) return MXG_ERR_ARG;
  if (const int err = balance_shape(T, E, k)) return err;
  if (!api::aligned32(logits) || !api::aligned32(ids) || !api::aligned32(counts) || !api::aligned32(prob_sums) ||
      !api::aligned32(workspace))
    return MXG_ERR_ALIGN;
  if (workspace_bytes < mxg_balance_loss_workspace_bytes(T, E)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.balance_loss_fwd");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int nblk = balance_blocks(T, E, kBlMaxBlocks);
  float* part = api::at<float>(workspace, 0);
  int32_t* part_counts = api::at<int32_t>(workspace, part_floats(T, E));
  int32_t* part_tokens = api::at<int32_t>(workspace, 2 * part_floats(T, E));
  with_lanes(E, [&](auto l) {
    balance_partial_kernel<l.value><<<nblk, kBlThreads, 0, s>>>(logits, ids, token_mask, T, E, k, part, part_counts,
                                                                part_tokens, dev_status);
  });
  count_launch();
  balance_finish_kernel<<<1, 256, 0, s>>>(part, part_counts, part_tokens, nblk, E, k, coef, loss, counts, prob_sums,
                                          n_tokens);
  count_launch();
  return api::cuda_status(cudaGetLastError());
}

extern "C" int mxg_balance_loss_bwd(const float* logits, const uint8_t* token_mask, const int32_t* counts,
                                    const int32_t* n_tokens, int T, int E, int k, float coef, const float* dloss,
                                    const int32_t* ids, const float* probs, const float* dprobs, float* dlogits,
                                    int32_t* dev_status, void* stream) {
  if (!logits || !counts || !n_tokens || !dlogits || !dev_status) return MXG_ERR_ARG;
  const int route = (ids != nullptr) + (probs != nullptr) + (dprobs != nullptr);
  if (route != 0 && route != 3) return MXG_ERR_ARG;      // the route's gradient needs all three
  if (const int err = balance_shape(T, E, k)) return err;
  if (!api::aligned32(logits) || !api::aligned32(counts) || !api::aligned32(ids) || !api::aligned32(probs) ||
      !api::aligned32(dprobs) || !api::aligned32(dlogits))
    return MXG_ERR_ALIGN;
  api::NvtxRange nvtx("mxg.balance_loss_bwd");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  with_lanes(E, [&](auto l) {
    balance_bwd_kernel<l.value><<<balance_blocks(T, E, 152 * 8), kBlThreads, 0, s>>>(
        logits, token_mask, counts, n_tokens, T, E, k, coef, dloss, ids, probs, dprobs, dlogits, dev_status);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}
