// Pieces shared by the two kernels of the orthogonalised momentum update
// (muon.cu, muon_resident.cu): the momentum, the norm, fp16 parts.
#pragma once
#include <cuda_fp16.h>

#include <cmath>

#include "common.cuh"
#include "ptx.cuh"

namespace mxg {

struct MomentumArgs {
  const void* grad;                       // bf16 or fp32 [batch][rows][cols]
  int grad_f32;
  const float* mom_in;                    // nullable
  float* mom_out;                         // nullable
  float mu;
  int nesterov;
  int64_t per;                            // elements of a matrix
};

namespace {

constexpr int kExpA = 12;                 // A and B are stored times 2^12
constexpr float kMostA = 15.99f;          // a 2^12 is B's diagonal for small singular values: fp16 ends at 65504

// ------------------------------------------------------------------ momentum
// Sum of squares that neither overflows nor underflows for any fp32 input:
// magnitudes below 2^-30 and from 2^46 are squared after scaling by a power of
// two (NaN compares false and stays in the middle sum).
struct SumSq {
  float lo, mid, hi;
  __device__ __forceinline__ void add(float v) {
    const float m = fabsf(v);
    if (m < 9.31322574615478515625e-10f) {             // 2^-30
      const float t = v * 18446744073709551616.f;      // 2^64
      lo = fmaf(t, t, lo);
    } else if (m >= 70368744177664.f) {                // 2^46
      const float t = v * 8.271806125530276749e-25f;   // 2^-80
      hi = fmaf(t, t, hi);
    } else {
      mid = fmaf(v, v, mid);
    }
  }
  // Eight values at once: where the largest magnitude needs no scaling, none of
  // them does (what underflows beside it does not count).  Few instructions:
  // code that runs once waits for its own fetch.
  __device__ __forceinline__ void add8(const float (&v)[8]) {
    float top = fabsf(v[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, fabsf(v[j]));
    if (top == 0.f || (top >= 9.31322574615478515625e-10f && top < 70368744177664.f)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) mid = fmaf(v[j], v[j], mid);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) add(v[j]);
    }
  }
  __device__ __forceinline__ double total() const {
    return static_cast<double>(lo) * 2.938735877055718770e-39 + static_cast<double>(mid) +
           static_cast<double>(hi) * 1.461501637330902918e48;   // 2^-128, 2^160
  }
};

constexpr int kMoThreads = 256;
constexpr int kMoVec = 8;                 // elements a thread takes at once

template <bool VEC>
__device__ __forceinline__ void load_f32(const float* p, int64_t i, int n, float (&v)[kMoVec]) {
  if constexpr (VEC) {
    uint32_t w[8];
    ld_global_v8(p + i, w);
#pragma unroll
    for (int j = 0; j < kMoVec; ++j) v[j] = __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kMoVec; ++j) v[j] = j < n ? p[i + j] : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load_grad(const MomentumArgs& P, int64_t i, int n, float (&v)[kMoVec]) {
  if (P.grad_f32) {
    load_f32<VEC>(static_cast<const float*>(P.grad), i, n, v);
  } else {
    const uint16_t* g = static_cast<const uint16_t*>(P.grad) + i;
    if constexpr (VEC) {
      const uint4 q = *reinterpret_cast<const uint4*>(g);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) v[j] = j < n ? bf16_bits_to_float(g[j]) : 0.f;
    }
  }
}

// Two values as fp16 (returned) and what the rounding left, as fp16 too.
__device__ __forceinline__ uint32_t split_half2(float a, float b, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// New momentum of eight elements (written when there is one), u to v.
template <bool VEC>
__device__ __forceinline__ void step_momentum(const MomentumArgs& P, int64_t i, int n, float (&u)[kMoVec]) {
  float m[kMoVec];
  load_grad<VEC>(P, i, n, u);
  if (P.mom_out == nullptr) return;
  if (P.mom_in != nullptr) {
    load_f32<VEC>(P.mom_in, i, n, m);
#pragma unroll
    for (int j = 0; j < kMoVec; ++j) m[j] = fmaf(P.mu, m[j], u[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kMoVec; ++j) m[j] = u[j];
  }
  if constexpr (VEC) {
    st_global_v8(P.mom_out + i, reinterpret_cast<const uint32_t*>(m));
  } else {
#pragma unroll
    for (int j = 0; j < kMoVec; ++j)
      if (j < n) P.mom_out[i + j] = m[j];
  }
#pragma unroll
  for (int j = 0; j < kMoVec; ++j) u[j] = P.nesterov ? fmaf(P.mu, m[j], u[j]) : m[j];
}

// u of eight elements (on 32 bytes of every buffer), and of one, from the new momentum.
__device__ __forceinline__ void momentum_u8(const MomentumArgs& P, int64_t i, float (&u)[kMoVec]) {
  if (P.mom_out == nullptr || P.nesterov) load_grad<true>(P, i, kMoVec, u);
  if (P.mom_out != nullptr) {
    float m[kMoVec];
    load_f32<true>(P.mom_out, i, kMoVec, m);
#pragma unroll
    for (int j = 0; j < kMoVec; ++j) u[j] = P.nesterov ? fmaf(P.mu, m[j], u[j]) : m[j];
  }
}
__device__ __forceinline__ float momentum_u1(const MomentumArgs& P, int64_t i) {
  const float g = P.grad_f32 ? static_cast<const float*>(P.grad)[i]
                             : bf16_bits_to_float(static_cast<const uint16_t*>(P.grad)[i]);
  if (P.mom_out == nullptr) return g;
  return P.nesterov ? fmaf(P.mu, P.mom_out[i], g) : P.mom_out[i];
}

// Whether B has a low part too (short side m of 65 to 128, long side n).  B's
// rounding is the largest error of an update from a few strong directions over
// noise (simulated, 96 x 3000: 1.8e-3 of X from B, 1.1e-3 from A, 0.7e-3 from X;
// the bf16 result's own rounding 1.66e-3).  Measured, times that rounding, one
// part and two: 96 x 958 1.49 1.24, 90 x 6000 1.70 1.28, 80 x 3000 1.61 1.30, but
// 128 x 6000 1.36 1.18 and 96 x 300 1.35 1.19, where one part is enough (two cost
// 8-10 % of the time).  At the edges, one part and (past them) two: 80 x 512 1.48,
// 80 x 513 1.21; 112 x 512 1.35, 112 x 513 1.17; 120 x 513 1.33, 119 x 513 1.16; 120 x
// 6000 1.38, 119 x 6000 1.18.
__host__ __device__ constexpr bool muon_b_low(int m, int n) { return m < 120 && n > 512; }

// u / |u| 2^ex is u times these three factors, in this order, so that no
// intermediate leaves fp32's range; n2 = |u|^2.
__device__ __forceinline__ void norm_factors(double n2, int ex, float (&f)[3]) {
  const double norm = sqrt(n2);
  if (norm == 0.0) {
    f[0] = f[1] = f[2] = 0.f;
  } else if (isfinite(norm)) {
    const int e = ilogb(norm);
    const int h = (ex - e) / 2;
    f[0] = scalbnf(1.f, h);
    f[1] = scalbnf(1.f, ex - e - h);
    f[2] = static_cast<float>(1.0 / scalbn(norm, -e));
  } else {
    f[0] = f[1] = 1.f;
    f[2] = static_cast<float>(1.0 / norm);
  }
}

}  // namespace

// The whole update of matrices that stay on the chip (muon_resident.cu):
// short side at most 128, long side at most kResidentMost.
constexpr int kResidentMost = 8192;
struct ResidentArgs {
  MomentumArgs mo;
  int batch, rows, cols, steps;
  int ex;                                 // X is held times 2^ex, A and B times 2^kExpA
  float alpha[3], alpha_last, beta, diag; // factors of the three products, as in muon.cu
  uint16_t* update;                       // bf16 [batch][rows][cols], nullable
  const uint16_t* w_in;
  uint16_t* w_out;                        // nullable: w_in * w_keep - lr * value
  float w_keep, lr;
  int32_t* status;
  // set by the launcher
  int m, n, tall, slice;                  // short and long side; columns of the long side per CTA
};
// CTAs that should take a matrix (short side m, long side n), 0: the tiled kernel is faster, or it does not fit.
int resident_cluster(int batch, int m, int n, bool split);
cudaError_t launch_muon_resident(ResidentArgs a, int cluster, bool split, cudaStream_t s);

}  // namespace mxg
