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
// at a time and every lane keeps its experts' sums in registers.  Where E is a
// multiple of four (VEC) a lane's experts are two 16-byte pieces of the row.
// Both passes are bound by the logits stream, and below a megabyte or so by
// the latency of the launch and of one trip to memory.  Where the stream is
// long the forward's instructions count beside it (65536 x 256: 10 us of reads;
// the softmax's arithmetic is some 130 instructions a warp and token), so it
// steps pointers instead of multiplying 64-bit indices, takes a full warp's
// maximum in one instruction and its own exponential and reciprocal: 23.0 ->
// 18.9 us with the finish.  Fetching the next tokens ahead of the softmax
// changes nothing (32 warps an SM do that).  Measured, launch included: forward
// 65536 x 256 18.9 us (3.6 TB/s), 77 x 5 6.2; backward 8192 x 64 with the
// route's gradient 9.3 us, 30011 x 60 9.3 (an empty kernel's graph: about 6).
#include <climits>
#include <cmath>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kBlVals = 8;               // experts per lane
constexpr int kBlFwdThreads = 1024;
constexpr int kBlFwdWarps = kBlFwdThreads / 32;
constexpr int kBlMaxBlocks = 152;        // partial sums of the forward: one block per SM
constexpr int kBlFinBlocks = 8;          // of 32 experts
constexpr int kBlBwdThreads = 256;
constexpr int kBlBwdWarps = kBlBwdThreads / 32;

// Expert of value i of lane gl of a group, and the inverse.
template <int LPT, bool VEC>
__device__ __forceinline__ int expert_of(int gl, int i) {
  return VEC ? 4 * (gl + LPT * (i >> 2)) + (i & 3) : gl + LPT * i;
}
template <int LPT, bool VEC>
__device__ __forceinline__ int lane_of(int e) {
  return (VEC ? e >> 2 : e) % LPT;
}
template <int LPT, bool VEC>
__device__ __forceinline__ int value_of(int e) {
  return VEC ? ((e >> 2) / LPT) * 4 + (e & 3) : e / LPT;
}

// e^d for d <= 0 (NaN stays): 2 to the power of d log2 e, the product taken in
// two pieces y + lo since a power magnifies y's rounding by y, and 2^lo = 1 + lo
// ln 2 for the tiny piece.  The relative error is below 2^-22 (ex2's 2^-22.5 and
// one rounding).  What is below fp32's normal numbers (d < -87.33) becomes zero,
// and so arguments can be kept above -200, where -inf would make lo NaN.  Fewer
// instructions than expf, which has to serve all arguments.
__device__ __forceinline__ float exp_neg(float d) {
  constexpr double kLog2e = 1.4426950408889634;
  constexpr float kHi = static_cast<float>(kLog2e), kLo = static_cast<float>(kLog2e - kHi);
  float e;
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(-200.f));
  const float y = d * kHi;
  const float lo = fmaf(d, kLo, fmaf(d, kHi, -y));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  return fmaf(e, lo * 0.693147181f, e);
}

// The group's softmax of one token: z[i] = logit of expert lane_in_group + LPT i
// (-inf past E) becomes the probability.  A row without a finite logit gives
// zeros; NaN (or +inf, as inf - inf) gives NaN in the whole row.
template <int LPT>
__device__ __forceinline__ void group_softmax(float (&z)[kBlVals]) {
  float top = z[0];
#pragma unroll
  for (int i = 1; i < kBlVals; ++i) top = fmaxf(top, z[i]);
  if constexpr (LPT == 32) {
    asm volatile("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(top));     // skips NaN like fmaxf
  } else {
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  if (top == -INFINITY) top = 0.f;       // fmaxf skips NaN: a row of NaN and -inf keeps its NaN below
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) z[i] = exp_neg(z[i] - top);
  float sum = ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
#pragma unroll
  for (int off = LPT / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  float inv;                             // of 1 <= sum <= 256, within 1 ulp
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sum));
  if (sum == 0.f) inv = 0.f;
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) z[i] *= inv;
}

template <int LPT, bool VEC>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, int gl, bool live,
                                            float (&z)[kBlVals]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kBlVals; i += 4) {
      const int e = expert_of<LPT, VEC>(gl, i);
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (live && e < E) v = *reinterpret_cast<const float4*>(row + e);
      z[i] = v.x;
      z[i + 1] = v.y;
      z[i + 2] = v.z;
      z[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kBlVals; ++i) {
      const int e = expert_of<LPT, VEC>(gl, i);
      z[i] = live && e < E ? row[e] : -INFINITY;
    }
  }
}

// Expert's share of the loss (before coef E).
__device__ __forceinline__ float balance_term(float prob_sum, int count, int k, int n) {
  const float nf = static_cast<float>(n);
  return n > 0 ? (static_cast<float>(count) / (static_cast<float>(k) * nf)) * (prob_sum / nf) : 0.f;
}

// The counts and the loss from s_sum / s_cnt / n (whole block, at least 256
// threads; the sums and counts of all experts are in shared memory).
__device__ __forceinline__ void balance_finish(const float* s_sum, const int* s_cnt, int n, float* s_term, int E,
                                               int k, float coef, float* loss, int32_t* counts, float* prob_sums,
                                               int32_t* n_tokens) {
  const int e = threadIdx.x;
  if (e < 256) {
    float term = 0.f;
    if (e < E) {
      prob_sums[e] = s_sum[e];
      counts[e] = s_cnt[e];
      term = balance_term(s_sum[e], s_cnt[e], k, n);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xffffffffu, term, off);
    if ((e & 31) == 0) s_term[e >> 5] = term;
  }
  __syncthreads();
  if (e == 0) {
    float t = 0.f;
    for (int i = 0; i < 8; ++i) t += s_term[i];
    *loss = coef * static_cast<float>(E) * t;
    *n_tokens = n;
  }
}

// Sums of the probabilities and counts of the chosen ids over the block's
// tokens: one partial per block and expert, or, when one block covers all
// tokens, the results.
template <int LPT, bool VEC>
__global__ void __launch_bounds__(kBlFwdThreads) balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E,
    int k, float coef, float* __restrict__ part, int32_t* __restrict__ part_counts, int32_t* __restrict__ part_tokens,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob_sums,
    int32_t* __restrict__ n_tokens, int32_t* status) {
  __shared__ float s_sum[kBlFwdWarps][256];
  __shared__ float s_term[8];
  __shared__ int s_cnt[256];
  __shared__ int s_tok;
  constexpr int TPW = 32 / LPT;          // tokens a warp takes at once
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  for (int e = threadIdx.x; e < E; e += kBlFwdThreads) s_cnt[e] = 0;
  if (threadIdx.x == 0) s_tok = 0;
  __syncthreads();
  float acc[kBlVals];
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) acc[i] = 0.f;
  int tokens = 0;
  // T k fits 31 bits, so token numbers (up to T + two steps) fit 32; the pointers step along
  const uint32_t step = gridDim.x * kBlFwdWarps * TPW, end = static_cast<uint32_t>(T);
  uint32_t t = (blockIdx.x * kBlFwdWarps + warp) * TPW + grp;
  const float* row = logits + static_cast<int64_t>(t) * E;
  const int32_t* id = ids + static_cast<int64_t>(t) * k + gl;
  const int64_t row_step = static_cast<int64_t>(step) * E, id_step = static_cast<int64_t>(step) * k;
  for (; t - grp < end; t += 2 * step, row += 2 * row_step, id += 2 * id_step) {
    // two tokens per group in flight
    float z[2][kBlVals];
    bool live[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      live[u] = t + u * step < end && (mask == nullptr || mask[t + u * step] != 0);
      load_logits<LPT, VEC>(row + u * row_step, E, gl, live[u], z[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (live[u]) {
        tokens += gl == 0;
        for (int j = gl; j < k; j += LPT) {
          const int e = id[u * id_step + j - gl];
          if (static_cast<unsigned>(e) >= static_cast<unsigned>(E)) report(status, MXG_ERR_EXPERT_ID);
          else atomicAdd(&s_cnt[e], 1);
          if (LPT == 32) break;          // k is at most 32
        }
      }
      __syncwarp();
      group_softmax<LPT>(z[u]);
#pragma unroll
      for (int i = 0; i < kBlVals; ++i) acc[i] += z[u][i];
    }
  }
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) {
#pragma unroll
    for (int off = 16; off >= LPT; off >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
    const int e = expert_of<LPT, VEC>(gl, i);
    if (grp == 0 && e < E) s_sum[warp][e] = acc[i];
  }
  if (tokens != 0) atomicAdd(&s_tok, tokens);
  __syncthreads();
  if (threadIdx.x < E) {
    const int e = threadIdx.x;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBlFwdWarps; ++w) s += s_sum[w][e];
    if (gridDim.x > 1) {
      part[static_cast<int64_t>(blockIdx.x) * E + e] = s;
      part_counts[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
    } else {
      s_sum[0][e] = s;                   // read and written by this thread only
    }
  }
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) part_tokens[blockIdx.x] = s_tok;
    return;
  }
  __syncthreads();
  balance_finish(s_sum[0], s_cnt, s_tok, s_term, E, k, coef, loss, counts, prob_sums, n_tokens);
}

// The partials, 32 experts a block: 32 threads share an expert, each adding
// every 32nd block in order, then their sums in order.  The eight blocks are one
// cluster and each hands its experts' share of the loss to block 0 through
// shared memory.  (With a ticket in global memory instead, the last block
// reading all sums again, 65536 x 256 took 2.2 us more; by a single block 6.)
__global__ void __cluster_dims__(kBlFinBlocks, 1, 1) __launch_bounds__(1024)
balance_finish_kernel(const float* __restrict__ part, const int32_t* __restrict__ part_counts,
                      const int32_t* __restrict__ part_tokens, int nblk, int E, int k, float coef,
                      float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob_sums,
                      int32_t* __restrict__ n_tokens) {
  __shared__ float s_sum[1024];
  __shared__ int s_cnt[1024];
  __shared__ float s_term[kBlFinBlocks];  // block 0's: every block's share
  __shared__ int s_n;
  if (threadIdx.x == 0) s_n = 0;
  cluster_sync();                         // block 0 is there to be written to
  dependency_wait();
  const int el = threadIdx.x & 31, e = blockIdx.x * 32 + el, r = threadIdx.x >> 5;
  float s = 0.f;
  int c = 0;
  if (e < E) {
#pragma unroll
    for (int i = 0; i < (kBlMaxBlocks + 31) / 32; ++i) {
      const int b = r + 32 * i;
      if (b < nblk) {
        s += part[static_cast<int64_t>(b) * E + e];
        c += part_counts[static_cast<int64_t>(b) * E + e];
      }
    }
  }
  s_sum[threadIdx.x] = s;
  s_cnt[threadIdx.x] = c;
  int n = threadIdx.x < nblk ? part_tokens[threadIdx.x] : 0;
  n = __reduce_add_sync(0xffffffffu, n);
  if (el == 0 && n != 0) atomicAdd(&s_n, n);
  __syncthreads();
  if (r == 0) {
    float term = 0.f;
    if (e < E) {
      for (int i = 1; i < 32; ++i) {
        s += s_sum[i * 32 + el];
        c += s_cnt[i * 32 + el];
      }
      prob_sums[e] = s;
      counts[e] = c;
      term = balance_term(s, c, k, s_n);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) term += __shfl_xor_sync(0xffffffffu, term, off);
    if (el == 0) st_shared_cluster_f32(map_to_rank(smem_u32(&s_term[blockIdx.x]), 0), term);
  }
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    float t = 0.f;
    for (int i = 0; i < kBlFinBlocks; ++i) t += s_term[i];
    *loss = coef * static_cast<float>(E) * t;
    *n_tokens = s_n;
  }
}

template <int LPT, bool VEC>
__global__ void __launch_bounds__(kBlBwdThreads) balance_bwd_kernel(
    const float* __restrict__ logits, const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ n_tokens, int T, int E, int k, float coef, const float* __restrict__ dloss,
    const int32_t* __restrict__ ids, const float* __restrict__ probs, const float* __restrict__ dprobs,
    float* __restrict__ dlogits, int32_t* status) {
  constexpr int TPW = 32 / LPT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % LPT, grp = lane / LPT;
  const uint32_t step = gridDim.x * kBlBwdWarps * TPW, end = static_cast<uint32_t>(T);
  uint32_t t = (blockIdx.x * kBlBwdWarps + warp) * TPW + grp;
  const int64_t row_step = static_cast<int64_t>(step) * E;
  int64_t row = static_cast<int64_t>(t) * E;
  // the first logits are on their way while the counts arrive
  bool in = t < end, live = in && (mask == nullptr || mask[t] != 0);
  float z[kBlVals];
  load_logits<LPT, VEC>(logits + row, E, gl, live, z);
  int cnt[kBlVals];
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) {
    const int e = expert_of<LPT, VEC>(gl, i);
    cnt[i] = e < E ? counts[e] : 0;
  }
  const int n = *n_tokens;
  const float up = n > 0 ? (dloss != nullptr ? *dloss : 1.f) * coef / static_cast<float>(n) : 0.f;
  // deviations of the lane's experts: (E c - k n) / (k n), the numerator exact
  const int64_t kn = static_cast<int64_t>(k) * n;
  const float inv = n > 0 ? 1.f / static_cast<float>(kn) : 0.f;
  float dev[kBlVals];
#pragma unroll
  for (int i = 0; i < kBlVals; ++i) dev[i] = static_cast<float>(static_cast<int64_t>(E) * cnt[i] - kn) * inv;
  while (t - grp < end) {
    group_softmax<LPT>(z);
    float mean = 0.f;
#pragma unroll
    for (int i = 0; i < kBlVals; ++i) mean = fmaf(z[i], dev[i], mean);
#pragma unroll
    for (int off = LPT / 2; off > 0; off >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, off);
    float d[kBlVals];
#pragma unroll
    for (int i = 0; i < kBlVals; ++i) d[i] = live ? up * z[i] * (dev[i] - mean) : 0.f;
    const bool here = in, kept = live;
    const int64_t pick = static_cast<int64_t>(t) * k;
    float* dst = dlogits + row;
    t += step;
    row += row_step;
    in = t < end;
    live = in && (mask == nullptr || mask[t] != 0);
    load_logits<LPT, VEC>(logits + row, E, gl, live, z);
    if (probs != nullptr) {
      // the route's gradient at the chosen experts: q_j (dq_j - sum_i q_i dq_i)
      float inner = 0.f;
      for (int j = gl; j < k; j += LPT)
        if (here) inner = fmaf(probs[pick + j], dprobs[pick + j], inner);
#pragma unroll
      for (int off = LPT / 2; off > 0; off >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, off);
      if (here) {
        for (int j = 0; j < k; ++j) {
          const int e = ids[pick + j];
          if (e < 0 || e >= E) {
            if (gl == 0 && kept) report(status, MXG_ERR_EXPERT_ID);      // a dropped token may have no route
          } else if (lane_of<LPT, VEC>(e) == gl) {
            const float q = probs[pick + j];
            const float g = q * (dprobs[pick + j] - inner);
            const int v = value_of<LPT, VEC>(e);
#pragma unroll
            for (int i = 0; i < kBlVals; ++i)
              if (v == i) d[i] += g;
          }
        }
      }
      __syncwarp();
    }
    if (here) {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kBlVals; i += 4) {
          const int e = expert_of<LPT, VEC>(gl, i);
          if (e < E) *reinterpret_cast<float4*>(dst + e) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBlVals; ++i) {
          const int e = expert_of<LPT, VEC>(gl, i);
          if (e < E) dst[e] = d[i];
        }
      }
    }
  }
}

int lanes_per_token(int E) {
  int l = 1;
  while (l * kBlVals < E) l *= 2;
  return l;
}

// Blocks of `warps` warps for a pass over T tokens: enough for one trip each, at most `most`.
int balance_blocks(int T, int E, int warps, int most) {
  const int64_t per = static_cast<int64_t>(warps) * (32 / lanes_per_token(E));
  const int64_t n = (T + per - 1) / per;
  return static_cast<int>(n < most ? n : most);
}

template <bool VEC, typename F>
void with_lanes(int lanes, F f) {
  using V = std::integral_constant<bool, VEC>;
  switch (lanes) {
    case 1: f(std::integral_constant<int, 1>{}, V{}); break;
    case 2: f(std::integral_constant<int, 2>{}, V{}); break;
    case 4: f(std::integral_constant<int, 4>{}, V{}); break;
    case 8: f(std::integral_constant<int, 8>{}, V{}); break;
    case 16: f(std::integral_constant<int, 16>{}, V{}); break;
    default: f(std::integral_constant<int, 32>{}, V{}); break;
  }
}
template <typename F>
void with_layout(int E, F f) {
  if (E % 4 == 0) with_lanes<true>(lanes_per_token(E), f);
  else with_lanes<false>(lanes_per_token(E), f);
}

int fwd_blocks(int T, int E) { return balance_blocks(T, E, kBlFwdWarps, kBlMaxBlocks); }
int64_t part_floats(int T, int E) { return api::align_up(4ll * fwd_blocks(T, E) * E, api::kAlign); }

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
  const int nblk = fwd_blocks(T, E);
  float* part = api::at<float>(workspace, 0);
  int32_t* part_counts = api::at<int32_t>(workspace, part_floats(T, E));
  int32_t* part_tokens = api::at<int32_t>(workspace, 2 * part_floats(T, E));
  with_layout(E, [&](auto l, auto v) {
    balance_partial_kernel<l.value, v.value><<<nblk, kBlFwdThreads, 0, s>>>(
        logits, ids, token_mask, T, E, k, coef, part, part_counts, part_tokens, loss, counts, prob_sums, n_tokens,
        dev_status);
  });
  count_launch();
  MXG_TRY(cudaGetLastError());
  if (nblk == 1) return MXG_OK;
  MXG_TRY(launch_after(balance_finish_kernel, dim3(kBlFinBlocks), dim3(1024), 0, s, part, part_counts, part_tokens,
                       nblk, E, k, coef, loss, counts, prob_sums, n_tokens));
  return MXG_OK;
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
  with_layout(E, [&](auto l, auto v) {
    balance_bwd_kernel<l.value, v.value><<<balance_blocks(T, E, kBlBwdWarps, 152 * 8), kBlBwdThreads, 0, s>>>(
        logits, token_mask, counts, n_tokens, T, E, k, coef, dloss, ids, probs, dprobs, dlogits, dev_status);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}
