// Orthogonalised momentum update of a batch of weight matrices (Muon): the
// experts' W_gate_up [E][2I][H] and W_down [E][H][I] from the gradients that
// the backward writes (bf16 dW, or the fp32 main_grad).
//
//   mom' = mu mom + g,  u = g + mu mom' (Nesterov) or mom'
//   X0   = u / |u|_F                      (zero where u is zero)
//   X   <- a X + (b A + c A^2) X, A = X X^T          steps times
//   update = scale X,  or  w' = w (1 - lr wd) - lr scale X
// The odd quintic drives every singular value of X towards one, so X becomes
// the orthogonal factor of u.
//
// The matrix is taken with its short side first (X [M][N], M <= N; a tall one
// transposed), since A is then the smaller product.  Every product is one of
// tcgen05 kind::f16 on operands stored with the contraction contiguous:
//   A  = X X^T        rows of X with rows of X
//   B  = b A + c A A  rows of A with rows of A   (A is symmetric)
//   X' = a X + B X    rows of B with rows of X^T
// so X is kept together with its transpose.  A and B are symmetric: only the
// tiles on and above the diagonal are computed, each stored twice.
//
// Number format.  Operands are fp16: X, A and B are bounded (|X|_F = 1 at the
// start, singular values at most ~1.2 afterwards), so the eleven-bit
// significand is worth more than bf16's range, and each is stored times a
// power of two that puts its entries well inside fp16's normal range:
//   X 2^ex, 2^ex ~ sqrt(N)  (an orthogonal X has entries of size 1 / sqrt(N)),
//   A 2^12, B 2^12          (entries at most ~1.5 and ~3).
// Sums are fp32 (tensor-core accumulators); momentum and norms are fp32/fp64.
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kExpA = 12;                 // A and B are stored times 2^12

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
  __device__ __forceinline__ double total() const {
    return static_cast<double>(lo) * 2.938735877055718770e-39 + static_cast<double>(mid) +
           static_cast<double>(hi) * 1.461501637330902918e48;   // 2^-128, 2^160
  }
};

constexpr int kMoThreads = 256;
constexpr int kMoTile = 64;               // the cast works on 64 x 64 tiles

struct MomentumArgs {
  const void* grad;                       // bf16 or fp32 [batch][rows][cols]
  int grad_f32;
  const float* mom_in;                    // nullable
  float* mom_out;                         // nullable
  float mu;
  int nesterov;
  int rows, cols;                         // as the caller has them
  int64_t per;                            // rows * cols
};

__device__ __forceinline__ float load_grad(const MomentumArgs& P, int64_t i) {
  return P.grad_f32 ? static_cast<const float*>(P.grad)[i]
                    : bf16_bits_to_float(static_cast<const uint16_t*>(P.grad)[i]);
}

// Momentum of element i (new, written when asked) -> u.
template <bool WRITE>
__device__ __forceinline__ float momentum_u(const MomentumArgs& P, int64_t i) {
  const float g = load_grad(P, i);
  float m;
  if (WRITE || P.mom_out == nullptr) {
    m = P.mom_in != nullptr ? fmaf(P.mu, P.mom_in[i], g) : g;
    if (WRITE && P.mom_out != nullptr) P.mom_out[i] = m;
  } else {
    m = P.mom_out[i];
  }
  return P.mom_out != nullptr ? (P.nesterov ? fmaf(P.mu, m, g) : m) : g;
}

// New momentum and the sum of squares of u: one partial per block.
__global__ void __launch_bounds__(kMoThreads) momentum_kernel(MomentumArgs P, int chunks, double* __restrict__ part) {
  const int64_t base = static_cast<int64_t>(blockIdx.y) * P.per;
  SumSq s{0.f, 0.f, 0.f};
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoThreads + threadIdx.x; i < P.per;
       i += static_cast<int64_t>(chunks) * kMoThreads)
    s.add(momentum_u<true>(P, base + i));
  double t = s.total();
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  __shared__ double w[kMoThreads / 32];
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int i = 0; i < kMoThreads / 32; ++i) v += w[i];
    part[static_cast<int64_t>(blockIdx.y) * chunks + blockIdx.x] = v;
  }
}

// X0 and its transpose in fp16: u / |u|_F 2^ex.  One 64 x 64 tile per block.
// x: the matrix in the caller's orientation, xt: its transpose.
__global__ void __launch_bounds__(kMoThreads) cast_kernel(MomentumArgs P, int chunks, const double* __restrict__ part,
                                                         int ex, __half* __restrict__ x, int64_t ldx, int64_t sx,
                                                         __half* __restrict__ xt, int64_t ldt, int64_t st) {
  __shared__ __half tile[kMoTile][kMoTile + 2];
  __shared__ float s_f[3];
  const int b = blockIdx.z;
  if (threadIdx.x == 0) {
    double n2 = 0.0;
    for (int i = 0; i < chunks; ++i) n2 += part[static_cast<int64_t>(b) * chunks + i];
    // u / |u| 2^ex as three factors, so no intermediate leaves fp32's range
    const double norm = sqrt(n2);
    if (norm == 0.0) {
      s_f[0] = s_f[1] = s_f[2] = 0.f;
    } else if (isfinite(norm)) {
      const int e = ilogb(norm);
      const int h = (ex - e) / 2;
      s_f[0] = scalbnf(1.f, h);
      s_f[1] = scalbnf(1.f, ex - e - h);
      s_f[2] = static_cast<float>(1.0 / scalbn(norm, -e));
    } else {
      s_f[0] = s_f[1] = 1.f;
      s_f[2] = static_cast<float>(1.0 / norm);
    }
  }
  __syncthreads();
  const float f0 = s_f[0], f1 = s_f[1], f2 = s_f[2];
  const int r0 = blockIdx.y * kMoTile, c0 = blockIdx.x * kMoTile;
  for (int i = threadIdx.x; i < kMoTile * kMoTile; i += kMoThreads) {
    const int r = i / kMoTile, c = i % kMoTile;
    if (r0 + r < P.rows && c0 + c < P.cols) {
      const float u = momentum_u<false>(P, b * P.per + static_cast<int64_t>(r0 + r) * P.cols + c0 + c);
      const __half h = __float2half_rn(u * f0 * f1 * f2);
      tile[r][c] = h;
      x[b * sx + static_cast<int64_t>(r0 + r) * ldx + c0 + c] = h;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kMoTile * kMoTile; i += kMoThreads) {
    const int c = i / kMoTile, r = i % kMoTile;
    if (r0 + r < P.rows && c0 + c < P.cols) xt[b * st + static_cast<int64_t>(c0 + c) * ldt + r0 + r] = tile[r][c];
  }
}

// ------------------------------------------------------------------ products
// D = P Q^T over fp16 operands [batch][rows][K], tiles of 128 x 128 on one SM
// or 256 x 256 on a CTA pair (cta_group::2, each SM holding its 128 rows of
// both operands).  Warp 0 issues TMA, warp 1 owns TMEM and issues the MMAs,
// warps 4-11 run the epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 and
// half of the tile's columns.  Persistent over the tiles of all matrices, the
// accumulator double-buffered in TMEM.  Every wait is bounded; one that gives
// up records MXG_ERR_TIMEOUT and stops the CTA's pipeline.
constexpr int kNsThreads = 384;
constexpr int kNsK = 64;                  // contraction elements per stage: one 128-byte swizzled row
constexpr int kNsRows = 128;              // rows of each operand per SM and stage
constexpr int kNsOpBytes = kNsRows * kNsK * 2;
constexpr int kNsStageBytes = 2 * kNsOpBytes;
constexpr int kNsStages = 5;
constexpr int kNsBox = 2048;              // 32 x 32 fp16: one store box
constexpr int kNsWarpOut = 4 * kNsBox;    // per epilogue warp: two boxes of D and two of D^T
constexpr int kNsCtrl = 1024;
constexpr int kNsSmem = 1024 + kNsStages * kNsStageBytes + 8 * kNsWarpOut + kNsCtrl;
static_assert(32 * 33 * 4 <= kNsWarpOut, "the last product stages 32 x 32 fp32 values");
static_assert(kNsSmem <= 232448, "shared memory budget");

struct NsArgs {
  int sym;                                // only tiles on and above the diagonal; stored twice
  int m, n, k;                            // D [m][n], contraction k
  int batch;
  int tiles_m, tiles_n;                   // per matrix
  int64_t total;                          // tiles of all matrices
  int p_rows, q_rows;                     // operand rows per matrix
  float alpha, beta;                      // D = alpha P Q^T + beta C
  const __half* c;                        // [batch][m][ldc], nullable; ldc a multiple of 16
  int64_t ldc, sc;
  // the last product: bf16 update, or new weights, in the caller's layout
  uint16_t* update;                       // nullable
  const uint16_t* w_in;
  uint16_t* w_out;                        // nullable: w_in * w_keep - D * lr
  float w_keep, lr;
  int flip;                               // the caller's matrix is D^T
  int64_t ldu, su;
  int32_t* status;
};

struct NsTile {
  int b, ti, tj;
};

__device__ __forceinline__ NsTile ns_tile(const NsArgs& P, int64_t t) {
  NsTile r;
  const int per = static_cast<int>(P.total / P.batch);
  r.b = static_cast<int>(t / per);
  int l = static_cast<int>(t - static_cast<int64_t>(r.b) * per);
  if (P.sym) {
    r.ti = 0;
    while (l >= P.tiles_m - r.ti) {
      l -= P.tiles_m - r.ti;
      ++r.ti;
    }
    r.tj = r.ti + l;
  } else {
    r.tj = l / P.tiles_m;                 // the short side fastest: B stays in L2
    r.ti = l - r.tj * P.tiles_m;
  }
  return r;
}

// 32 columns of C for this thread's row, zero past the matrix.
__device__ __forceinline__ void ns_load_c(const NsArgs& P, int b, int row, int col, uint32_t (&w)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (row < P.m && col + 16 * h < P.n) {          // whole 32-byte pieces: ldc is a multiple of 16
      ld_global_nc_v8(P.c + b * P.sc + row * P.ldc + col + 16 * h, w + 8 * h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[8 * h + i] = 0u;
    }
  }
}

// One 32 x 32 block of D = alpha acc + beta C as fp16, to D and (mirror) D^T:
// staged in two 2 KB boxes (64-byte rows, 16-byte chunk j of row r at
// j ^ ((r / 2) % 4): the tensor maps' 64-byte swizzle) and stored by TMA, which
// also cuts the block at the matrix's edges.  A lane writes its row of D in
// four 16-byte pieces and its column of D^T in 2-byte pieces, 32 lanes side by
// side: both free of bank conflicts.
__device__ __forceinline__ void ns_store_block(const NsArgs& P, const uint32_t (&r)[32], const uint32_t (&c)[16],
                                               uint8_t* box, const CUtensorMap* tmO, const CUtensorMap* tmT, int row0,
                                               int col0, int b, bool mirror, int lane) {
  uint32_t h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 cf = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
    const __half2 v = __floats2half2_rn(fmaf(P.beta, cf.x, P.alpha * __uint_as_float(r[2 * i])),
                                        fmaf(P.beta, cf.y, P.alpha * __uint_as_float(r[2 * i + 1])));
    h[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  // the boxes written two blocks ago have left shared memory
  if (lane == 0) bulk_wait_group_read<1>();
  __syncwarp();
  const int sw = (lane >> 1) & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ sw) << 4)) =
        make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
  if (mirror) {
    uint8_t* tb = box + kNsBox;
#pragma unroll
    for (int i = 0; i < 32; ++i) {                   // row i of the transposed box, column `lane`
      const uint16_t v = static_cast<uint16_t>(i & 1 ? h[i / 2] >> 16 : h[i / 2]);
      *reinterpret_cast<uint16_t*>(tb + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + (lane & 7) * 2) = v;
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(tmO, box, col0, row0, b);
    if (mirror) tma_store_3d(tmT, box + kNsBox, row0, col0, b);
    bulk_commit_group();
  }
}

// One 32 x 32 block of the last product to the caller's bf16 matrix, whose
// rows may start at any even address: staged in fp32 (rows of 33 words) and
// written row by row of the caller's matrix, 32 lanes side by side.
__device__ __forceinline__ void ns_store_last(const NsArgs& P, const uint32_t (&r)[32], const uint32_t (&c)[16],
                                              float* buf, int row0, int col0, int b, int lane) {
  __syncwarp();                                      // the previous block has been read
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 cf = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
    buf[lane * 33 + 2 * i] = fmaf(P.beta, cf.x, P.alpha * __uint_as_float(r[2 * i]));
    buf[lane * 33 + 2 * i + 1] = fmaf(P.beta, cf.y, P.alpha * __uint_as_float(r[2 * i + 1]));
  }
  __syncwarp();
  const int y0 = P.flip ? col0 : row0, x0 = P.flip ? row0 : col0;      // of the caller's matrix
  const int ny = min(32, (P.flip ? P.n : P.m) - y0);
  const bool in = x0 + lane < (P.flip ? P.m : P.n);
  const int64_t base = b * P.su + static_cast<int64_t>(y0) * P.ldu + x0 + lane;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    if (i < ny && in) {
      const float v = P.flip ? buf[lane * 33 + i] : buf[i * 33 + lane];
      const int64_t u = base + i * P.ldu;
      if (P.update != nullptr) P.update[u] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
      if (P.w_out != nullptr)
        P.w_out[u] =
            static_cast<uint16_t>(pack_bf16x2(fmaf(-P.lr, v, bf16_bits_to_float(P.w_in[u]) * P.w_keep), 0.f));
    }
  }
}

template <bool PAIR, bool LAST>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_product_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmT,
                      const __grid_constant__ NsArgs P) {
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int BN = PAIR ? 256 : 128;    // columns of a tile (and accumulator columns)
  constexpr int TM = PAIR ? 256 : 128;    // rows of a tile, both CTAs
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = sm + kNsStages * kNsStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + 8 * kNsWarpOut);
  uint64_t* empty = full + kNsStages;
  uint64_t* tfull = empty + kNsStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drained = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_set = abort_flag + 1;
  uint32_t* landing = tmem_slot + 4;      // rank 1's release stores (pair)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNsStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      // the eight epilogue warps; in a pair also the MMA thread's expect_tx for
      // the 8 x 4 bytes that rank 1's warps store
      mbar_init(&tempty[a], PAIR ? 9 : 8);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    *never_set = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  __syncthreads();
  if (warp == 1) {
    tmem_alloc<CG>(tmem_slot, 2 * BN);
    tmem_relinquish<CG>();
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t tile0 = PAIR ? blockIdx.x / 2 : blockIdx.x;
  const int64_t tstep = PAIR ? gridDim.x / 2 : gridDim.x;
  const int nk = (P.k + kNsK - 1) / kNsK;
  auto fail = [&]() {
    report(P.status, MXG_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool aborted = false;
      const uint32_t full0 = PAIR ? map_to_rank(smem_u32(full), 0) : 0u;
      for (int64_t t = tile0; t < P.total && !aborted; t += tstep) {
        const NsTile tc = ns_tile(P, t);
        const int prow = tc.b * P.p_rows + tc.ti * TM + static_cast<int>(rank) * kNsRows;
        const int qrow = tc.b * P.q_rows + tc.tj * BN + static_cast<int>(rank) * kNsRows;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          uint8_t* sP = sm + stage * kNsStageBytes;
          uint8_t* sQ = sP + kNsOpBytes;
          if (!PAIR || rank == 0) {
            mbar_arrive_expect_tx(&full[stage], CG * kNsStageBytes);     // both CTAs' bytes
            tma_load_2d(sP, &tmP, kb * kNsK, prow, &full[stage]);
            tma_load_2d(sQ, &tmQ, kb * kNsK, qrow, &full[stage]);
          } else {
            tma_load_2d_pair(sP, &tmP, kb * kNsK, prow, full0 + stage * 8);
            tma_load_2d_pair(sQ, &tmQ, kb * kNsK, qrow, full0 + stage * 8);
          }
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (aborted) {                      // let copies already in flight land before the CTA exits
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool aborted = false;
      int64_t done = 0;
      for (int64_t t = tile0; t < P.total && !aborted; t += tstep) {
        const bool got = PAIR ? mbar_wait_bounded_cluster(&tempty[acc], acc_phase ^ 1, abort_flag, kWaitLimitNs)
                              : mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, abort_flag, kWaitLimitNs);
        if (!got) {
          fail();
          break;
        }
        tc_fence_after();
        const uint32_t d_t = tmem + acc * BN;
        for (int kb = 0; kb < nk; ++kb) {
          const bool in = PAIR ? mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, kWaitLimitNs)
                               : mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs);
          if (!in) {
            fail();
            aborted = true;
            break;
          }
          tc_fence_after();
          uint8_t* sP = sm + stage * kNsStageBytes;
          const uint64_t pd = smem_desc(smem_u32(sP), 0, 1024, kLayoutSwizzle128B);
          const uint64_t qd = smem_desc(smem_u32(sP + kNsOpBytes), 0, 1024, kLayoutSwizzle128B);
#pragma unroll
          for (int k = 0; k < kNsK / 16; ++k)
            mma_bf16<CG>(d_t, pd + 2 * k, qd + 2 * k, idesc_f16(TM, BN), (kb | k) != 0 ? 1u : 0u);
          mma_commit<CG>(&empty[stage]);
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (aborted) break;
        mma_commit<CG>(&tfull[acc]);
        if (PAIR) mbar_arrive_expect_tx(&tempty[acc], 8 * 4);
        ++done;
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      // rank 1's release stores of the last two tiles have landed here before this CTA exits
      if (PAIR && done > 1) mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, never_set, kWaitLimitNs);
      if (PAIR && done > 0) {
        const uint32_t last = acc ^ 1;
        const uint32_t last_phase = acc == 0 ? acc_phase ^ 1 : acc_phase;   // phase bit in use when it was filled
        mbar_wait_bounded(&tempty[last], last_phase, never_set, kWaitLimitNs);
      }
      mma_commit<CG>(drained);
      mbar_wait_bounded(drained, 0, never_set, kWaitLimitNs);
    }
  } else if (warp >= 4) {
    constexpr int COLS = BN / 2;
    const int q = warp & 3;
    const int hf = (warp - 4) >> 2;
    uint8_t* box = boxes + (warp - 4) * kNsWarpOut;
    uint32_t acc = 0, acc_phase = 0, flip = 0;
    for (int64_t t = tile0; t < P.total; t += tstep) {
      const NsTile tc = ns_tile(P, t);
      const int row0 = tc.ti * TM + static_cast<int>(rank) * kNsRows + q * 32;
      const int col0 = tc.tj * BN + hf * COLS;
      const bool mirror = P.sym == 0 || tc.ti != tc.tj;
      // the addend is on its way while the tile's MMAs run
      uint32_t cv[COLS / 32][16];
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) {
        if (P.c != nullptr) {
          ns_load_c(P, tc.b, row0 + lane, col0 + 32 * c, cv[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) cv[c][i] = 0u;
        }
      }
      bool got = mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs);
      got = __all_sync(0xffffffffu, got);
      if (!got) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + hf * COLS;
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tb + 32 * c, r);
        tmem_ld_wait();
        if (c == COLS / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (PAIR && rank == 1)
              st_async_complete_tx(map_to_rank(smem_u32(&landing[warp - 4]), 0), 1u,
                                   map_to_rank(smem_u32(&tempty[acc]), 0));
            else
              mbar_arrive(&tempty[acc]);
          }
        }
        if (row0 < P.m && col0 + 32 * c < P.n) {
          if constexpr (LAST) {
            ns_store_last(P, r, cv[c], reinterpret_cast<float*>(box), row0, col0 + 32 * c, tc.b, lane);
          } else {
            ns_store_block(P, r, cv[c], box + flip * 2 * kNsBox, &tmO, &tmT, row0, col0 + 32 * c, tc.b, mirror, lane);
            flip ^= 1;
          }
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (!LAST) {
      if (lane == 0) bulk_wait_group<0>();           // the stores have completed before the CTA exits
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<CG>(tmem, 2 * BN);
}

// --------------------------------------------------------------------- host
int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

template <bool PAIR, bool LAST>
cudaError_t launch_ns(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, const CUtensorMap& mt,
                      const NsArgs& a, cudaStream_t s) {
  auto kern = ns_product_kernel<PAIR, LAST>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem);
  if (err != cudaSuccess) return err;
  const int64_t units = PAIR ? sm_count() / 2 : sm_count();
  const int64_t n = a.total < units ? a.total : units;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? 2 * n : n));
  cfg.blockDim = dim3(kNsThreads);
  cfg.dynamicSmemBytes = kNsSmem;
  cfg.stream = s;
  if (PAIR) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  err = cudaLaunchKernelEx(&cfg, kern, mp, mq, mo, mt, a);
  count_launch();
  return err != cudaSuccess ? err : cudaGetLastError();
}

struct NsMat {                            // fp16 [batch][rows][cols], rows ld apart
  __half* p;
  int rows, cols;
  int64_t ld;
};

// D of one product over the batch: operands p and q, D and D^T to o and t
// (none for the last product, whose outputs are in a).
cudaError_t ns_product(NsArgs a, const NsMat& p, const NsMat& q, const NsMat* o, const NsMat* t, cudaStream_t s) {
  CUtensorMap mp, mq, mo, mt;
  a.p_rows = p.rows;
  a.q_rows = q.rows;
  a.m = p.rows;
  a.n = q.rows;
  a.k = p.cols;
  if (!tma_map_f16(&mp, p.p, p.cols, static_cast<int64_t>(a.batch) * p.rows, p.ld, kNsRows) ||
      !tma_map_f16(&mq, q.p, q.cols, static_cast<int64_t>(a.batch) * q.rows, q.ld, kNsRows))
    return cudaErrorInvalidValue;
  mo = mt = mp;
  if (o != nullptr && (!tma_map_f16_boxes(&mo, o->p, o->cols, o->rows, a.batch, o->ld) ||
                       !tma_map_f16_boxes(&mt, t->p, t->cols, t->rows, a.batch, t->ld)))
    return cudaErrorInvalidValue;
  auto tiles = [&](int w) {
    a.tiles_m = (a.m + w - 1) / w;
    a.tiles_n = (a.n + w - 1) / w;
    const int64_t per = a.sym ? static_cast<int64_t>(a.tiles_m) * (a.tiles_m + 1) / 2
                              : static_cast<int64_t>(a.tiles_m) * a.tiles_n;
    a.total = per * a.batch;
    return a.total;
  };
  if (tiles(256) >= sm_count() / 2)
    return o != nullptr ? launch_ns<true, false>(mp, mq, mo, mt, a, s) : launch_ns<true, true>(mp, mq, mo, mt, a, s);
  tiles(128);
  return o != nullptr ? launch_ns<false, false>(mp, mq, mo, mt, a, s) : launch_ns<false, true>(mp, mq, mo, mt, a, s);
}

struct NsPlan {
  int m, n, tall;                         // X is [m][n], m <= n; tall: the caller's matrix is X^T
  int64_t ldx, ldt;                       // row lengths of X [m][ldx] and X^T [n][ldt] (also of A and B)
  int chunks;                             // partial sums of squares per matrix
  int64_t part, x0, x1, t0, t1, a, b, bytes;
};

NsPlan ns_plan(int batch, int rows, int cols) {
  NsPlan p{};
  p.tall = rows > cols;
  p.m = p.tall ? cols : rows;
  p.n = p.tall ? rows : cols;
  p.ldx = api::align_up(p.n, 16);
  p.ldt = api::align_up(p.m, 16);
  const int64_t per = static_cast<int64_t>(rows) * cols;
  int64_t c = (per + kMoThreads * 16 - 1) / (kMoThreads * 16);
  const int64_t most = (152 * 8 + batch - 1) / batch;
  p.chunks = static_cast<int>(c < most ? c : most);
  api::Carver w;
  p.part = w.take(8ll * batch * p.chunks);
  const int64_t xb = 2ll * batch * p.m * p.ldx, tb = 2ll * batch * p.n * p.ldt, ab = 2ll * batch * p.m * p.ldt;
  p.x0 = w.take(xb);
  p.x1 = w.take(xb);
  p.t0 = w.take(tb);
  p.t1 = w.take(tb);
  p.a = w.take(ab);
  p.b = w.take(ab);
  p.bytes = w.off;
  return p;
}

int muon_shape(int batch, int rows, int cols) {
  if (batch <= 0 || rows <= 0 || cols <= 0) return MXG_ERR_ARG;
  const int64_t longest = rows > cols ? rows : cols;
  // grid and tensor-map coordinates are 32-bit
  if (batch > 65535 || longest > (1 << 21) || batch * longest > INT32_MAX - 256) return MXG_ERR_SHAPE;
  return MXG_OK;
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" size_t mxg_muon_workspace_bytes(int batch, int rows, int cols) {
  if (muon_shape(batch, rows, cols) != MXG_OK) return 0;
  return static_cast<size_t>(ns_plan(batch, rows, cols).bytes);
}

extern "C" int mxg_muon_update(const mxg_muon_args* a, void* stream) {
  if (!a || !a->grad || !a->workspace || !a->dev_status) return MXG_ERR_ARG;
  if (a->momentum_in && !a->momentum_out) return MXG_ERR_ARG;
  if ((a->w_in != nullptr) != (a->w_out != nullptr)) return MXG_ERR_ARG;
  if (!a->update && !a->w_out) return MXG_ERR_ARG;
  if (a->steps < 1 || a->steps > 64) return MXG_ERR_ARG;
  if (const int err = muon_shape(a->batch, a->rows, a->cols)) return err;
  if (!api::aligned32(a->grad) || !api::aligned32(a->momentum_in) || !api::aligned32(a->momentum_out) ||
      !api::aligned32(a->update) || !api::aligned32(a->w_in) || !api::aligned32(a->w_out) ||
      !api::aligned32(a->workspace))
    return MXG_ERR_ALIGN;
  const NsPlan p = ns_plan(a->batch, a->rows, a->cols);
  if (a->workspace_bytes < static_cast<uint64_t>(p.bytes)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.muon_update");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = api::at<double>(a->workspace, p.part);
  const NsMat x[2] = {{api::at<__half>(a->workspace, p.x0), p.m, p.n, p.ldx},
                      {api::at<__half>(a->workspace, p.x1), p.m, p.n, p.ldx}};
  const NsMat xt[2] = {{api::at<__half>(a->workspace, p.t0), p.n, p.m, p.ldt},
                       {api::at<__half>(a->workspace, p.t1), p.n, p.m, p.ldt}};
  const NsMat am{api::at<__half>(a->workspace, p.a), p.m, p.m, p.ldt};
  const NsMat bm{api::at<__half>(a->workspace, p.b), p.m, p.m, p.ldt};
  int ex = 0;                             // 2^ex ~ sqrt(n)
  while ((1ll << (2 * ex)) < p.n) ++ex;

  MomentumArgs mo{a->grad, a->grad_f32, a->momentum_in, a->momentum_out, a->mu, a->nesterov, a->rows, a->cols,
                  static_cast<int64_t>(a->rows) * a->cols};
  momentum_kernel<<<dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>(a->batch)), kMoThreads, 0, s>>>(
      mo, p.chunks, part);
  count_launch();
  const dim3 cgrid(static_cast<unsigned>((a->cols + kMoTile - 1) / kMoTile),
                   static_cast<unsigned>((a->rows + kMoTile - 1) / kMoTile), static_cast<unsigned>(a->batch));
  const NsMat& u = p.tall ? xt[0] : x[0];
  const NsMat& ut = p.tall ? x[0] : xt[0];
  cast_kernel<<<cgrid, kMoThreads, 0, s>>>(mo, p.chunks, part, ex, u.p, u.ld, u.rows * u.ld, ut.p, ut.ld,
                                           ut.rows * ut.ld);
  count_launch();
  if (cudaGetLastError() != cudaSuccess) return MXG_ERR_CUDA;

  for (int i = 0; i < a->steps; ++i) {
    const int cur = i & 1, nxt = cur ^ 1;
    const bool last = i + 1 == a->steps;
    // A 2^12 = (X 2^ex)(X 2^ex)^T 2^(12 - 2 ex)
    NsArgs ga{};
    ga.batch = a->batch;
    ga.status = a->dev_status;
    ga.sym = 1;
    ga.alpha = static_cast<float>(std::ldexp(1.0, kExpA - 2 * ex));
    MXG_TRY(ns_product(ga, x[cur], x[cur], &am, &am, s));
    // B 2^12 = b (A 2^12) + c 2^-12 (A 2^12)(A 2^12)
    NsArgs gb = ga;
    gb.alpha = static_cast<float>(std::ldexp(static_cast<double>(a->c), -kExpA));
    gb.beta = a->b;
    gb.c = am.p;
    gb.ldc = am.ld;
    gb.sc = am.rows * am.ld;
    MXG_TRY(ns_product(gb, am, am, &bm, &bm, s));
    // X' 2^ex = a (X 2^ex) + 2^-12 (B 2^12)(X 2^ex); the last one leaves as scale X'
    const double f = last ? a->scale * std::ldexp(1.0, -ex) : 1.0;
    NsArgs gx{};
    gx.batch = a->batch;
    gx.status = a->dev_status;
    gx.alpha = static_cast<float>(f * std::ldexp(1.0, -kExpA));
    gx.beta = static_cast<float>(f * a->a);
    gx.c = x[cur].p;
    gx.ldc = x[cur].ld;
    gx.sc = x[cur].rows * x[cur].ld;
    if (last) {
      gx.update = a->update;
      gx.w_in = a->w_in;
      gx.w_out = a->w_out;
      gx.w_keep = static_cast<float>(1.0 - static_cast<double>(a->lr) * a->weight_decay);
      gx.lr = a->lr;
      gx.flip = p.tall;
      gx.ldu = a->cols;
      gx.su = mo.per;
    }
    MXG_TRY(ns_product(gx, bm, xt[cur], last ? nullptr : &x[nxt], last ? nullptr : &xt[nxt], s));
  }
  return MXG_OK;
}
