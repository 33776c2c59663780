// Backward of the router's linear layer for dense logit gradients.
//
// mxg_router_bwd takes the gradients of the k chosen logits of a token; a loss
// on the whole softmax (the balance loss) gives every logit one.  With
// G = dlogits [T][E]:
//   dx        = dx_in + G W_r      (bf16, rounded once)
//   dw_router = G^T x              (fp32, fixed-order sums over token chunks)
#include <climits>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"

namespace mxg {
namespace {

constexpr int kRlCols = 512;                  // hidden columns per CTA, two per thread
constexpr int kRlThreads = kRlCols / 2;
constexpr int kRlChunk = 256;                 // tokens per partial sum
constexpr int kRlGroup = 16;                  // experts per CTA of the dW pass

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__global__ void __launch_bounds__(kRlThreads) router_linear_dx_kernel(const uint32_t* __restrict__ w,
                                                                     const float* __restrict__ g,
                                                                     const uint32_t* dx_in, int T, int H, int E,
                                                                     uint32_t* dx) {
  const int hp = blockIdx.x * kRlThreads + threadIdx.x;
  if (hp >= H / 2) return;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    float lo = 0.f, hi = 0.f;
    for (int e = 0; e < E; ++e) {
      const float d = g[t * E + e];
      const uint32_t wv = w[static_cast<int64_t>(e) * (H / 2) + hp];
      lo = fmaf(d, lo16(wv), lo);
      hi = fmaf(d, hi16(wv), hi);
    }
    if (dx_in != nullptr) {
      const uint32_t v = dx_in[t * (H / 2) + hp];
      lo += lo16(v);
      hi += hi16(v);
    }
    dx[t * (H / 2) + hp] = pack_bf16x2(lo, hi);
  }
}

__global__ void __launch_bounds__(kRlThreads) router_linear_dw_kernel(const uint32_t* __restrict__ x,
                                                                     const float* __restrict__ g, int T, int H, int E,
                                                                     float* __restrict__ part) {
  __shared__ float s_g[kRlChunk][kRlGroup];
  const int hp = blockIdx.x * kRlThreads + threadIdx.x;
  const int e0 = blockIdx.z * kRlGroup;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kRlChunk;
  const int nt = static_cast<int>(T - t0 < kRlChunk ? T - t0 : kRlChunk);
  for (int i = threadIdx.x; i < nt * kRlGroup; i += kRlThreads) {
    const int e = e0 + i % kRlGroup;
    s_g[i / kRlGroup][i % kRlGroup] = e < E ? g[(t0 + i / kRlGroup) * E + e] : 0.f;
  }
  __syncthreads();
  if (hp >= H / 2) return;
  float2 acc[kRlGroup];
#pragma unroll
  for (int i = 0; i < kRlGroup; ++i) acc[i] = make_float2(0.f, 0.f);
  for (int t = 0; t < nt; ++t) {
    const uint32_t xv = x[(t0 + t) * (H / 2) + hp];
#pragma unroll
    for (int i = 0; i < kRlGroup; ++i) {
      acc[i].x = fmaf(s_g[t][i], lo16(xv), acc[i].x);
      acc[i].y = fmaf(s_g[t][i], hi16(xv), acc[i].y);
    }
  }
#pragma unroll
  for (int i = 0; i < kRlGroup; ++i)
    if (e0 + i < E)
      *reinterpret_cast<float2*>(part + (static_cast<int64_t>(blockIdx.y) * E + e0 + i) * H + 2 * hp) = acc[i];
}

__global__ void __launch_bounds__(256) router_linear_sum_kernel(const float* __restrict__ part, int chunks,
                                                               int64_t n, float* __restrict__ dw) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float s = 0.f;
  for (int c = 0; c < chunks; ++c) s += part[c * n + i];
  dw[i] = s;
}

int rl_chunks(int T) { return (T + kRlChunk - 1) / kRlChunk; }

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" size_t mxg_router_linear_bwd_workspace_bytes(int T, int H, int E) {
  if (T <= 0 || H <= 0 || E <= 0) return 0;
  return static_cast<size_t>(4ll * rl_chunks(T) * E * H);
}

extern "C" int mxg_router_linear_bwd(const uint16_t* x, const uint16_t* w_router, const float* dlogits,
                                     const uint16_t* dx_in, int T, int H, int E, uint16_t* dx, float* dw_router,
                                     void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (!x || !w_router || !dlogits || !dx || !dw_router || !workspace || !dev_status) return MXG_ERR_ARG;
  if (T <= 0 || H <= 0 || E <= 0) return MXG_ERR_ARG;
  if (H % 128 != 0 || E > 256) return MXG_ERR_SHAPE;
  if (!api::aligned32(x) || !api::aligned32(w_router) || !api::aligned32(dlogits) || !api::aligned32(dx_in) ||
      !api::aligned32(dx) || !api::aligned32(dw_router) || !api::aligned32(workspace))
    return MXG_ERR_ALIGN;
  if (workspace_bytes < mxg_router_linear_bwd_workspace_bytes(T, H, E)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.router_linear_bwd");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned cols = static_cast<unsigned>((H / 2 + kRlThreads - 1) / kRlThreads);
  router_linear_dx_kernel<<<dim3(cols, static_cast<unsigned>(T < 4096 ? T : 4096)), kRlThreads, 0, s>>>(
      reinterpret_cast<const uint32_t*>(w_router), dlogits, reinterpret_cast<const uint32_t*>(dx_in), T, H, E,
      reinterpret_cast<uint32_t*>(dx));
  count_launch();
  float* part = static_cast<float*>(workspace);
  router_linear_dw_kernel<<<dim3(cols, static_cast<unsigned>(rl_chunks(T)), static_cast<unsigned>((E + kRlGroup - 1) / kRlGroup)),
                            kRlThreads, 0, s>>>(reinterpret_cast<const uint32_t*>(x), dlogits, T, H, E, part);
  count_launch();
  const int64_t n = static_cast<int64_t>(E) * H;
  router_linear_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(part, rl_chunks(T), n, dw_router);
  count_launch();
  return api::cuda_status(cudaGetLastError());
}
