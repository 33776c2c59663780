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
// Every matrix is stored once, in the caller's orientation.  With M the short
// side and N the long one, the three products of a step contract over
//   A  = X X^T                 N   (a tall X [N][M]: A = X^T X)
//   B  = a I + b A + c A A     M
//   X' = B X                   M   (tall: X' = X B)
// on tcgen05 kind::f16, whose operands may be read with the contraction
// contiguous (K-major) or across it (MN-major), so no transposed copy is kept.
// A and B are symmetric: only their tiles on and above the diagonal are
// computed and stored, and a block below it is read as the transpose of the
// one above (see ns_transposed).
//
// Number format.  Operands are fp16: X, A and B are bounded (|X|_F = 1 at the
// start, singular values at most ~1.2 afterwards), so the eleven-bit
// significand is worth more than bf16's range, and each is stored times a
// power of two that puts its entries well inside fp16's normal range:
//   X 2^ex, 2^ex ~ sqrt(N)  (an orthogonal X has entries of size 1 / sqrt(N)),
//   A 2^12, B 2^12          (entries at most ~1.5 and ~5).
// Folding a I into B rounds a + B_ii to eleven bits, an error of the size of
// X's own rounding, and spares the last product a second read of X.
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
constexpr int kMoVec = 8;                 // elements a thread takes at once

struct MomentumArgs {
  const void* grad;                       // bf16 or fp32 [batch][rows][cols]
  int grad_f32;
  const float* mom_in;                    // nullable
  float* mom_out;                         // nullable
  float mu;
  int nesterov;
  int64_t per;                            // elements of a matrix
};

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

// New momentum and the sum of squares of u: one partial per block.  VEC: every
// matrix starts on a 32-byte boundary of each buffer.
template <bool VEC>
__global__ void __launch_bounds__(kMoThreads) momentum_kernel(MomentumArgs P, int chunks, double* __restrict__ part) {
  const int64_t base = static_cast<int64_t>(blockIdx.y) * P.per;
  SumSq s{0.f, 0.f, 0.f};
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kMoThreads + threadIdx.x) * kMoVec; i < P.per;
       i += static_cast<int64_t>(chunks) * kMoThreads * kMoVec) {
    const int n = static_cast<int>(P.per - i < kMoVec ? P.per - i : kMoVec);
    float g[kMoVec], m[kMoVec];
    load_grad<VEC>(P, base + i, n, g);
    if (P.mom_in != nullptr) {
      load_f32<VEC>(P.mom_in, base + i, n, m);
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) m[j] = fmaf(P.mu, m[j], g[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) m[j] = g[j];
    }
    if (P.mom_out != nullptr) {
      if constexpr (VEC) {
        st_global_v8(P.mom_out + base + i, reinterpret_cast<const uint32_t*>(m));
      } else {
#pragma unroll
        for (int j = 0; j < kMoVec; ++j)
          if (j < n) P.mom_out[base + i + j] = m[j];
      }
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) s.add(P.nesterov ? fmaf(P.mu, m[j], g[j]) : m[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) s.add(g[j]);
    }
  }
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

// X0 = u / |u|_F 2^ex in fp16, rows ld apart.  A block takes whole rows; its
// first act is the matrix's norm from the partials (the same sum, in the same
// order, in every block).
template <bool VEC>
__global__ void __launch_bounds__(kMoThreads) cast_kernel(MomentumArgs P, int chunks, const double* __restrict__ part,
                                                         int ex, int rows, int cols, __half* __restrict__ x,
                                                         int64_t ld) {
  __shared__ double s_w[kMoThreads / 32];
  __shared__ float s_f[3];
  const int b = blockIdx.y;
  double n2 = 0.0;
  for (int i = threadIdx.x; i < chunks; i += kMoThreads) n2 += part[static_cast<int64_t>(b) * chunks + i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, off);
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = n2;
  __syncthreads();
  if (threadIdx.x == 0) {
    n2 = 0.0;
    for (int i = 0; i < kMoThreads / 32; ++i) n2 += s_w[i];
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
  const int groups = (cols + kMoVec - 1) / kMoVec;          // of a row
  const int64_t total = static_cast<int64_t>(rows) * groups;
  for (int64_t gi = static_cast<int64_t>(blockIdx.x) * kMoThreads + threadIdx.x; gi < total;
       gi += static_cast<int64_t>(gridDim.x) * kMoThreads) {
    const int64_t r = gi / groups;
    const int c = static_cast<int>(gi - r * groups) * kMoVec;
    const int n = min(kMoVec, cols - c);
    const int64_t i = b * P.per + r * cols + c;
    float u[kMoVec];
    if (P.mom_out == nullptr || P.nesterov) load_grad<VEC>(P, i, n, u);
    if (P.mom_out != nullptr) {
      float m[kMoVec];
      load_f32<VEC>(P.mom_out, i, n, m);
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) u[j] = P.nesterov ? fmaf(P.mu, m[j], u[j]) : m[j];
    }
    uint32_t h[kMoVec / 2];
#pragma unroll
    for (int j = 0; j < kMoVec / 2; ++j) {
      const __half2 v = __floats2half2_rn(u[2 * j] * f0 * f1 * f2, u[2 * j + 1] * f0 * f1 * f2);
      h[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
    // ld is a multiple of 16, so a group of eight starts on 16 bytes and fits the row's padding
    *reinterpret_cast<uint4*>(x + (static_cast<int64_t>(b) * rows + r) * ld + c) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

// ------------------------------------------------------------------ products
// D = P Q^T over fp16 operands, tiles of 128 x 128 on one SM or 256 x 256 on a
// CTA pair (cta_group::2, each SM holding its 128 rows of both operands).
// Warp 0 issues TMA, warp 1 owns TMEM and issues the MMAs, warps 4-11 run the
// epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 and half of the tile's
// columns.  Persistent over the tiles of all matrices, the accumulator
// double-buffered in TMEM.  Every wait is bounded; one that gives up records
// MXG_ERR_TIMEOUT and stops the CTA's pipeline.
//
// An operand's 128 rows x 64 contraction elements come as two 64 x 64 boxes of
// 128-byte swizzled rows, 8 KB each.  K-major: box h holds rows 64 h ..; the
// two follow one another as 128 rows of 128 bytes (8-row groups 1024 bytes
// apart; a K = 16 step is 32 bytes).  MN-major: box h holds the 64 contraction
// rows of operand rows 64 h .. (leading offset 8192 between them, 8-row groups
// 1024 bytes apart; a K = 16 step is 16 rows, 2048 bytes).
constexpr int kNsThreads = 384;
constexpr int kNsK = 64;                  // contraction elements per stage
constexpr int kNsRows = 128;              // rows of each operand per SM and stage
constexpr int kNsBoxBytes = 64 * 64 * 2;
constexpr int kNsOpBytes = 2 * kNsBoxBytes;
constexpr int kNsStageBytes = 2 * kNsOpBytes;
constexpr int kNsStages = 5;
constexpr int kNsOut = 32 * 64 * 2;       // 32 rows x 64 columns of D: one store box
constexpr int kNsWarpOut = 2 * kNsOut;    // two per epilogue warp
constexpr int kNsCtrl = 1024;
constexpr int kNsSmem = 1024 + kNsStages * kNsStageBytes + 8 * kNsWarpOut + kNsCtrl;
constexpr int kNsSym = 256;               // a symmetric matrix is stored in full within diagonal blocks of this size
static_assert(kNsSmem <= 232448, "shared memory budget");
static_assert(32 * 33 * 4 <= kNsWarpOut, "unaligned outputs stage 32 x 32 fp32 values");

// How an operand lies in memory.
enum NsForm { NS_K = 0,                   // [rows][k]
              NS_MN = 1,                  // [k][rows]
              NS_SYM = 2 };               // symmetric [rows][rows], blocks on and above the diagonal

enum NsOut { NS_F16 = 0,                  // D to fp16 boxes
             NS_POLY = 3,                 // the same with beta C + diag I added
             NS_LAST = 1,                 // D, or weights, to the caller's bf16 matrix by TMA
             NS_ROWS = 2 };               // the same by plain stores (rows that TMA cannot address, or both outputs)

struct NsArgs {
  int sym;                                // only tiles on and above the diagonal
  int m, n, k;                            // D [m][n], contraction k
  int batch;
  int tiles_m, tiles_n;                   // per matrix
  int n_fast;                             // column tiles vary fastest
  int64_t total;                          // tiles of all matrices
  int p_form, q_form;
  float alpha, beta, diag;                // D = alpha P Q^T + beta C + diag I
  const __half* c;                        // [batch][m][ldc], nullable; ldc a multiple of 16
  int64_t ldc;
  // the last product: bf16 [batch][m][n]
  uint16_t* update;                       // nullable
  const uint16_t* w_in;
  uint16_t* w_out;                        // nullable: w_in * w_keep - D * lr
  float w_keep, lr;
  int32_t* status;
};

struct NsTile {
  int b, ti, tj;
};

// First column tile of row tile ti of a symmetric matrix: tiles of 128 fill
// the diagonal blocks of kNsSym as well.
template <bool PAIR>
__host__ __device__ __forceinline__ int ns_first(int ti) {
  return PAIR ? ti : ti & ~1;
}

template <bool PAIR>
__device__ __forceinline__ NsTile ns_tile(const NsArgs& P, int64_t t) {
  NsTile r;
  const int per = static_cast<int>(P.total / P.batch);
  r.b = static_cast<int>(t / per);
  int l = static_cast<int>(t - static_cast<int64_t>(r.b) * per);
  if (P.sym) {
    r.ti = 0;
    while (l >= P.tiles_m - ns_first<PAIR>(r.ti)) {
      l -= P.tiles_m - ns_first<PAIR>(r.ti);
      ++r.ti;
    }
    r.tj = ns_first<PAIR>(r.ti) + l;
  } else if (P.n_fast) {
    r.ti = l / P.tiles_n;
    r.tj = l - r.ti * P.tiles_n;
  } else {
    r.tj = l / P.tiles_m;
    r.ti = l - r.tj * P.tiles_m;
  }
  return r;
}

// Whether the 64 contraction elements from k0 of operand rows row0 .. are read
// MN-major: below the diagonal a symmetric matrix holds nothing, and the block
// (rows, k) is the transpose of (k, rows).
__device__ __forceinline__ bool ns_transposed(int form, int row0, int k0) {
  return form == NS_MN || (form == NS_SYM && k0 / kNsSym < row0 / kNsSym);
}

template <bool PEER>
__device__ __forceinline__ void ns_load(uint8_t* dst, const CUtensorMap* map, bool mn, int row0, int k0, int b,
                                        uint64_t* bar, uint32_t peer_bar) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int x = mn ? row0 + 64 * h : k0, y = mn ? k0 : row0 + 64 * h;
    if (PEER) tma_load_3d_pair(dst + h * kNsBoxBytes, map, x, y, b, peer_bar);
    else tma_load_3d(dst + h * kNsBoxBytes, map, x, y, b, bar);
  }
}

__device__ __forceinline__ uint64_t ns_desc(const uint8_t* op, bool mn) {
  return smem_desc(smem_u32(op), mn ? kNsBoxBytes : 0, 1024, kLayoutSwizzle128B);
}

// 64 columns of a row of C, zero past the matrix's edge (whole 32-byte pieces:
// rows are padded to 16).  NC: nothing writes the matrix during the kernel.
template <bool NC>
__device__ __forceinline__ void ns_load_row(const void* base, int64_t off, bool in, int col, int n,
                                            uint32_t (&w)[32]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (in && col + 16 * h < n) {
      const uint16_t* src = static_cast<const uint16_t*>(base) + off + 16 * h;
      if (NC) ld_global_nc_v8(src, w + 8 * h);
      else ld_global_v8(src, w + 8 * h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[8 * h + i] = 0u;
    }
  }
}

// alpha acc, and for a polynomial in A (ADD) + beta C + diag where row == col.
template <bool ADD>
__device__ __forceinline__ float2 ns_value(const NsArgs& P, uint32_t r0, uint32_t r1, uint32_t c, int row, int col) {
  float2 v = make_float2(P.alpha * __uint_as_float(r0), P.alpha * __uint_as_float(r1));
  if constexpr (ADD) {
    const float2 cf = __half22float2(*reinterpret_cast<const __half2*>(&c));
    v.x = fmaf(P.beta, cf.x, v.x) + (row == col ? P.diag : 0.f);
    v.y = fmaf(P.beta, cf.y, v.y) + (row == col + 1 ? P.diag : 0.f);
  }
  return v;
}

// 32 rows x 64 columns of packed 16-bit results (this lane's row in h) to
// global memory: staged as 128-byte rows (16-byte piece j of row r at
// j ^ (r % 8): the tensor map's 128-byte swizzle, free of bank conflicts) and
// stored by one TMA box, which is cut at the matrix's edges.
__device__ __forceinline__ void ns_store_box(const uint32_t (&h)[32], uint8_t* box, const CUtensorMap* tm, int row0,
                                             int col0, int b, int lane) {
  if (lane == 0) bulk_wait_group_read<1>();          // the box written two boxes ago has left shared memory
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(tm, box, col0, row0, b);
    bulk_commit_group();
  }
}

// One 32 x 32 block of the last product to a bf16 matrix whose rows may start
// at any even address: staged in fp32 (rows of 33 words) and written row by
// row, 32 lanes side by side.
__device__ __forceinline__ void ns_store_rows(const NsArgs& P, const float (&v)[32], float* buf, int row0, int col0,
                                              int b, int lane) {
  __syncwarp();                                      // the previous block has been read
#pragma unroll
  for (int i = 0; i < 32; ++i) buf[lane * 33 + i] = v[i];
  __syncwarp();
  const int ny = min(32, P.m - row0);
  const bool in = col0 + lane < P.n;
  const int64_t base = (static_cast<int64_t>(b) * P.m + row0) * P.n + col0 + lane;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    if (i < ny && in) {
      const float x = buf[i * 33 + lane];
      const int64_t u = base + static_cast<int64_t>(i) * P.n;
      if (P.update != nullptr) P.update[u] = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
      if (P.w_out != nullptr)
        P.w_out[u] =
            static_cast<uint16_t>(pack_bf16x2(fmaf(-P.lr, x, bf16_bits_to_float(P.w_in[u]) * P.w_keep), 0.f));
    }
  }
}

template <bool PAIR, int OUT>
__global__ void __launch_bounds__(kNsThreads, 1)
    ns_product_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmO, const __grid_constant__ NsArgs P) {
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
    if (OUT != NS_ROWS) tma_prefetch_desc(&tmO);
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
        const NsTile tc = ns_tile<PAIR>(P, t);
        const int prow = tc.ti * TM + static_cast<int>(rank) * kNsRows;
        const int qrow = tc.tj * BN + static_cast<int>(rank) * kNsRows;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          uint8_t* sP = sm + stage * kNsStageBytes;
          uint8_t* sQ = sP + kNsOpBytes;
          const int k0 = kb * kNsK;
          const bool pmn = ns_transposed(P.p_form, prow, k0), qmn = ns_transposed(P.q_form, qrow, k0);
          if (!PAIR || rank == 0) {
            mbar_arrive_expect_tx(&full[stage], CG * kNsStageBytes);     // both CTAs' bytes
            ns_load<false>(sP, &tmP, pmn, prow, k0, tc.b, &full[stage], 0u);
            ns_load<false>(sQ, &tmQ, qmn, qrow, k0, tc.b, &full[stage], 0u);
          } else {
            ns_load<true>(sP, &tmP, pmn, prow, k0, tc.b, nullptr, full0 + stage * 8);
            ns_load<true>(sQ, &tmQ, qmn, qrow, k0, tc.b, nullptr, full0 + stage * 8);
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
        const NsTile tc = ns_tile<PAIR>(P, t);
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
          // a tile's rows lie in one block of kNsSym, so the pair's CTAs agree on the form
          const bool pmn = ns_transposed(P.p_form, tc.ti * TM, kb * kNsK);
          const bool qmn = ns_transposed(P.q_form, tc.tj * BN, kb * kNsK);
          const uint8_t* sP = sm + stage * kNsStageBytes;
          const uint64_t pd = ns_desc(sP, pmn), qd = ns_desc(sP + kNsOpBytes, qmn);
          const uint32_t pstep = pmn ? 2048 >> 4 : 32 >> 4, qstep = qmn ? 2048 >> 4 : 32 >> 4;
          const uint32_t id = idesc_f16(TM, BN) | (pmn ? kIdescAMn : 0u) | (qmn ? kIdescBMn : 0u);
#pragma unroll
          for (uint32_t k = 0; k < kNsK / 16; ++k)
            mma_bf16<CG>(d_t, pd + k * pstep, qd + k * qstep, id, (kb | k) != 0 ? 1u : 0u);
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
    constexpr int BOXES = COLS / 64;
    constexpr bool ADD = OUT == NS_POLY;
    const int q = warp & 3;
    const int hf = (warp - 4) >> 2;
    uint8_t* box = boxes + (warp - 4) * kNsWarpOut;
    uint32_t acc = 0, acc_phase = 0, flip = 0;
    for (int64_t t = tile0; t < P.total; t += tstep) {
      const NsTile tc = ns_tile<PAIR>(P, t);
      const int row0 = tc.ti * TM + static_cast<int>(rank) * kNsRows + q * 32;
      const int col0 = tc.tj * BN + hf * COLS;
      const bool in = row0 + lane < P.m;
      // the addend is on its way while the tile's MMAs run
      uint32_t cv[ADD ? BOXES : 1][32];
      if constexpr (ADD) {
#pragma unroll
        for (int c = 0; c < BOXES; ++c)
          ns_load_row<true>(P.c, (static_cast<int64_t>(tc.b) * P.m + row0 + lane) * P.ldc + col0 + 64 * c, in,
                            col0 + 64 * c, P.n, cv[c]);
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
      for (int c = 0; c < BOXES; ++c) {
        const int col = col0 + 64 * c;
        const bool any = row0 < P.m && col < P.n;
        uint32_t h[32], w[32];
        if (OUT == NS_LAST && P.w_out != nullptr)
          ns_load_row<false>(P.w_in, (static_cast<int64_t>(tc.b) * P.m + row0 + lane) * P.n + col, in, col, P.n, w);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tb + 64 * c + 32 * half, r);
          tmem_ld_wait();
          if (c == BOXES - 1 && half == 1) {
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
          if constexpr (OUT == NS_ROWS) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = ns_value<false>(P, r[2 * i], r[2 * i + 1], 0u, 0, 0);
              v[2 * i] = x.x;
              v[2 * i + 1] = x.y;
            }
            if (any && col + 32 * half < P.n)
              ns_store_rows(P, v, reinterpret_cast<float*>(box), row0, col + 32 * half, tc.b, lane);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 x = ns_value<ADD>(P, r[2 * i], r[2 * i + 1], cv[ADD ? c : 0][16 * half + i], row0 + lane,
                                       col + 32 * half + 2 * i);
              if constexpr (OUT == NS_F16 || ADD) {
                const __half2 v = __floats2half2_rn(x.x, x.y);
                h[16 * half + i] = *reinterpret_cast<const uint32_t*>(&v);
              } else {
                if (P.w_out != nullptr) {
                  const uint32_t wv = w[16 * half + i];
                  x.x = fmaf(-P.lr, x.x, __uint_as_float(wv << 16) * P.w_keep);
                  x.y = fmaf(-P.lr, x.y, __uint_as_float(wv & 0xffff0000u) * P.w_keep);
                }
                h[16 * half + i] = pack_bf16x2(x.x, x.y);
              }
            }
          }
        }
        if (OUT != NS_ROWS && any) {
          ns_store_box(h, box + flip * kNsOut, &tmO, row0, col, tc.b, lane);
          flip ^= 1;
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (OUT != NS_ROWS) {
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

template <bool PAIR, int OUT>
cudaError_t launch_ns(const CUtensorMap& mp, const CUtensorMap& mq, const CUtensorMap& mo, NsArgs a, cudaStream_t s) {
  constexpr int W = PAIR ? 256 : 128;
  a.tiles_m = (a.m + W - 1) / W;
  a.tiles_n = (a.n + W - 1) / W;
  int64_t per = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
  if (a.sym) {
    per = 0;
    for (int i = 0; i < a.tiles_m; ++i) per += a.tiles_m - ns_first<PAIR>(i);
  }
  a.total = per * a.batch;
  auto kern = ns_product_kernel<PAIR, OUT>;
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
  err = cudaLaunchKernelEx(&cfg, kern, mp, mq, mo, a);
  count_launch();
  return err != cudaSuccess ? err : cudaGetLastError();
}

struct NsMat {                            // 16-bit [batch][rows][cols], rows ld apart
  void* p;
  int rows, cols;
  int64_t ld;
};

// D of one product over the batch: operands p and q in their forms, D to o
// (fp16, or the caller's bf16 matrix as a says).
cudaError_t ns_product(NsArgs a, const NsMat& p, const NsMat& q, const NsMat& o, int out, cudaStream_t s) {
  CUtensorMap mp, mq, mo;
  a.m = o.rows;
  a.n = o.cols;
  a.k = a.p_form == NS_K ? p.cols : p.rows;
  if (!tma_map_b16_3d(&mp, p.p, p.cols, p.rows, a.batch, p.ld, 64) ||
      !tma_map_b16_3d(&mq, q.p, q.cols, q.rows, a.batch, q.ld, 64))
    return cudaErrorInvalidValue;
  mo = mp;
  if (out != NS_ROWS && !tma_map_b16_3d(&mo, o.p, o.cols, o.rows, a.batch, o.ld, 32)) return cudaErrorInvalidValue;
  const int64_t tm = (a.m + 255) / 256, tn = (a.n + 255) / 256;
  const bool pair = (a.sym ? tm * (tm + 1) / 2 : tm * tn) * a.batch >= sm_count() / 2;
  if (out == NS_POLY)
    return pair ? launch_ns<true, NS_POLY>(mp, mq, mo, a, s) : launch_ns<false, NS_POLY>(mp, mq, mo, a, s);
  if (out == NS_F16) return pair ? launch_ns<true, NS_F16>(mp, mq, mo, a, s) : launch_ns<false, NS_F16>(mp, mq, mo, a, s);
  if (out == NS_LAST)
    return pair ? launch_ns<true, NS_LAST>(mp, mq, mo, a, s) : launch_ns<false, NS_LAST>(mp, mq, mo, a, s);
  return pair ? launch_ns<true, NS_ROWS>(mp, mq, mo, a, s) : launch_ns<false, NS_ROWS>(mp, mq, mo, a, s);
}

struct NsPlan {
  int m, n, tall;                         // short and long side; tall: the matrix is [n][m]
  int64_t ldx, lda;                       // row lengths of X and of A and B, padded to 16
  int chunks;                             // partial sums of squares per matrix
  int64_t part, x0, x1, a, b, bytes;
};

NsPlan ns_plan(int batch, int rows, int cols) {
  NsPlan p{};
  p.tall = rows > cols;
  p.m = p.tall ? cols : rows;
  p.n = p.tall ? rows : cols;
  p.ldx = api::align_up(cols, 16);
  p.lda = api::align_up(p.m, 16);
  const int64_t per = static_cast<int64_t>(rows) * cols;
  const int64_t c = (per + kMoThreads * kMoVec - 1) / (kMoThreads * kMoVec);
  const int64_t most = (152 * 8 + batch - 1) / batch;
  p.chunks = static_cast<int>(c < most ? c : most);
  api::Carver w;
  p.part = w.take(8ll * batch * p.chunks);
  const int64_t xb = 2ll * batch * rows * p.ldx, ab = 2ll * batch * p.m * p.lda;
  p.x0 = w.take(xb);
  p.x1 = w.take(xb);
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
  const NsMat x[2] = {{api::at<void>(a->workspace, p.x0), a->rows, a->cols, p.ldx},
                      {api::at<void>(a->workspace, p.x1), a->rows, a->cols, p.ldx}};
  const NsMat am{api::at<void>(a->workspace, p.a), p.m, p.m, p.lda};
  const NsMat bm{api::at<void>(a->workspace, p.b), p.m, p.m, p.lda};
  int ex = 0;                             // 2^ex ~ sqrt(n)
  while ((1ll << (2 * ex)) < p.n) ++ex;

  const int64_t per = static_cast<int64_t>(a->rows) * a->cols;
  const MomentumArgs mo{a->grad, a->grad_f32, a->momentum_in, a->momentum_out, a->mu, a->nesterov, per};
  const unsigned nb = static_cast<unsigned>(a->batch);
  // 32-byte loads where every matrix (and, for the cast, every row) starts on 32 bytes of each buffer
  if (per % 16 == 0) momentum_kernel<true><<<dim3(static_cast<unsigned>(p.chunks), nb), kMoThreads, 0, s>>>(mo, p.chunks, part);
  else momentum_kernel<false><<<dim3(static_cast<unsigned>(p.chunks), nb), kMoThreads, 0, s>>>(mo, p.chunks, part);
  count_launch();
  const dim3 cgrid(static_cast<unsigned>(p.chunks), nb);
  __half* x0 = static_cast<__half*>(x[0].p);
  if (a->cols % 16 == 0) cast_kernel<true><<<cgrid, kMoThreads, 0, s>>>(mo, p.chunks, part, ex, a->rows, a->cols, x0, p.ldx);
  else cast_kernel<false><<<cgrid, kMoThreads, 0, s>>>(mo, p.chunks, part, ex, a->rows, a->cols, x0, p.ldx);
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
    ga.p_form = ga.q_form = p.tall ? NS_MN : NS_K;
    ga.alpha = static_cast<float>(std::ldexp(1.0, kExpA - 2 * ex));
    MXG_TRY(ns_product(ga, x[cur], x[cur], am, NS_F16, s));
    // B 2^12 = a 2^12 I + b (A 2^12) + c 2^-12 (A 2^12)(A 2^12)
    NsArgs gb = ga;
    gb.p_form = gb.q_form = NS_SYM;
    gb.alpha = static_cast<float>(std::ldexp(static_cast<double>(a->c), -kExpA));
    gb.beta = a->b;
    gb.diag = static_cast<float>(std::ldexp(static_cast<double>(a->a), kExpA));
    gb.c = static_cast<const __half*>(am.p);
    gb.ldc = am.ld;
    MXG_TRY(ns_product(gb, am, am, bm, NS_POLY, s));
    // X' 2^ex = 2^-12 (B 2^12)(X 2^ex), X B when tall; the last one leaves as scale X'.
    // The short side's tiles vary fastest, so B stays in L2 and X streams.
    NsArgs gx{};
    gx.batch = a->batch;
    gx.status = a->dev_status;
    gx.n_fast = p.tall;
    gx.p_form = p.tall ? NS_K : NS_SYM;
    gx.q_form = p.tall ? NS_SYM : NS_MN;
    gx.alpha = static_cast<float>(last ? a->scale * std::ldexp(1.0, -kExpA - ex) : std::ldexp(1.0, -kExpA));
    NsMat o = x[nxt];
    int out = NS_F16;
    if (last) {
      gx.update = a->update;
      gx.w_in = a->w_in;
      gx.w_out = a->w_out;
      gx.w_keep = static_cast<float>(1.0 - static_cast<double>(a->lr) * a->weight_decay);
      gx.lr = a->lr;
      o = NsMat{a->w_out ? a->w_out : a->update, a->rows, a->cols, a->cols};
      // whole 32-byte pieces of the caller's rows, one output
      out = a->cols % 16 == 0 && !(a->w_out && a->update) ? NS_LAST : NS_ROWS;
    }
    MXG_TRY(ns_product(gx, p.tall ? x[cur] : bm, p.tall ? bm : x[cur], o, out, s));
  }
  return MXG_OK;
}
