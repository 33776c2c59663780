// The orthogonalised momentum update of small matrices, on the chip from the
// gradient to the update (see muon.cu for the mathematics and the number
// format): short side M at most 128, long side N at most 8192.
//
// A cluster of 1, 2, 4, 8 or 16 CTAs takes a matrix; each keeps its share of the
// long side (up to 512 columns) of X in shared memory for the whole run, as
// rows of the short side: boxes of 128 rows x 64 columns, 128-byte swizzle.
// The same bytes serve as an operand of both products over X:
//   A = X X^T   K-major (contraction along the columns), both operands alike
//   X' = B X    MN-major (contraction along the rows)
// so a step is: partial A on the tensor cores; the partials added up in rank
// order through distributed shared memory (each CTA adds up its share of the
// rows and hands them to all); B = a I + b A + c A A in every CTA; X' in place.
// Two cluster barriers are all that a step waits for outside its own SM, where
// the tiled kernel takes a launch-wide trip through memory after each product.
//
// SPLIT (M <= 64): rows 0-63 of a box hold the high and rows 64-127 the low
// fp16 parts; one product yields all pairs of parts, and
// A = (high, high) + (high, low) + (low, high).
//
// Otherwise A and X have one part, and B one or two (see muon_b_low).
//
// Latency bounds it: a step is a chain of three products of 1-2 k cycles and
// the passes between them.  4 x 128 x 256, five steps: 41 us, of 78 k cycles 12 k
// for the momentum, 4 k for the norm and 10 k for X0 (57 us tiled); 20 x 64 x 512
// 41 us (84), 5 x 128 x 4096 90 us (115), 2 x 48 x 8192 on sixteen CTAs 74 (124).
#include <atomic>
#include <climits>

#include "kernels.h"
#include "muon.cuh"

namespace mxg {
namespace {

constexpr int kRsWarps = 8;                       // warps that compute; one more issues the MMAs
constexpr int kRsThreads = 32 * (kRsWarps + 1);
constexpr int kRsSlice = 512;                     // columns of the long side per CTA, at most
constexpr int kRsCluster = 16;                    // more than eight: by opt-in
static_assert(kRsSlice * kRsCluster == kResidentMost, "largest long side");
constexpr int kRsBox = 128 * 128;                 // 128 rows x 64 fp16
constexpr int kRsX = kRsSlice / 64 * kRsBox;
constexpr int kRsAb = 2 * kRsBox;                 // A, later B, as an operand (SPLIT: high, low)
constexpr int kRsPart = 128 * 128 * 4;            // fp32 sums (SPLIT: three blocks of 64 x 64); output staging
constexpr int kRsSmem = 1024 + kRsX + kRsAb + kRsPart + 1024;
static_assert(kRsSmem <= 232448, "shared memory budget");
static_assert(kRsWarps * 32 * 33 * 4 <= kRsPart, "output staging");

// 16-byte piece j of row r of a box or of the sums: rows 0-7 start in distinct bank groups.
__device__ __forceinline__ int swz(int j, int r) { return (j ^ (r & 7)) << 4; }

// Sum of the cluster's fp32 blocks [SIDE][SIDE] (16-byte pieces swizzled), left
// in every CTA: CTA k adds up its share of the rows in rank order and stores
// them everywhere.  Only that CTA reads those rows of the others, so they can
// be overwritten at once.  All threads of all CTAs.
template <int SIDE, int MOST>
__device__ __forceinline__ void cluster_sum(uint8_t* part, int C, uint32_t rank, int tid) {
  cluster_sync();
  if (tid < 32 * kRsWarps) {
    constexpr int PIECES = SIDE / 4;
    const uint32_t base = smem_u32(part);
    const int r0 = SIDE / C * static_cast<int>(rank);
    for (int i = tid; i < SIDE / C * PIECES; i += 32 * kRsWarps) {
      const int row = r0 + i / PIECES;
      const uint32_t at = base + row * SIDE * 4 + swz(i % PIECES, row);
      float4 s;
#pragma unroll
      for (int k0 = 0; k0 < MOST; k0 += 8) {        // eight requested together
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k0 + k < C) v[k] = ld_shared_cluster_v4(map_to_rank(at, k0 + k));
        if (k0 == 0) s = v[0];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k0 + k > 0 && k0 + k < C) {
            s.x += v[k].x;
            s.y += v[k].y;
            s.z += v[k].z;
            s.w += v[k].w;
          }
      }
#pragma unroll
      for (int k = 0; k < MOST; ++k)
        if (k < C) st_shared_cluster_v4(map_to_rank(at, k), s);
    }
  }
  cluster_sync();
}

// This lane's 64 accumulator columns from taddr on, times alpha.
__device__ __forceinline__ void read64(float alpha, uint32_t taddr, float (&v)[64]) {
  uint32_t r[2][32];
  tmem_ld_32x32b_x32(taddr, r[0]);
  tmem_ld_32x32b_x32(taddr + 32, r[1]);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = alpha * __uint_as_float(r[i >> 5][i & 31]);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 rows (m0 ..) x 64 columns (n0 ..) of the result, this lane's row in v, to
// the caller's matrix: rows of a wide matrix go through a 32 x 32 tile so that
// 32 lanes write side by side; a tall matrix has this lane's values a row
// apart and the lanes side by side already.
__device__ __forceinline__ void write_out(const ResidentArgs& P, const float (&v)[64], float* buf, int b, int m0, int n0,
                                          int lane) {
  const int64_t mat = static_cast<int64_t>(b) * P.rows * P.cols;
  auto put = [&](int64_t at, float x) {
    if (P.update != nullptr) P.update[at] = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
    if (P.w_out != nullptr)
      P.w_out[at] = static_cast<uint16_t>(pack_bf16x2(fmaf(-P.lr, x, bf16_bits_to_float(P.w_in[at]) * P.w_keep), 0.f));
  };
  if (P.tall) {
    if (m0 + lane < P.m)
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (n0 + i < P.n) put(mat + static_cast<int64_t>(n0 + i) * P.m + m0 + lane, v[i]);
    return;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) buf[lane * 33 + i] = v[32 * half + i];
    __syncwarp();
    const int c = n0 + 32 * half + lane;
    if (c < P.n)
#pragma unroll 8
      for (int i = 0; i < 32; ++i)
        if (m0 + i < P.m) put(mat + static_cast<int64_t>(m0 + i) * P.n + c, buf[i * 33 + lane]);
  }
}

// A CTA's share of a matrix in items of 8 values along the long side of one
// row of the short side: contiguous in a wide matrix (consecutive threads take
// consecutive items of a row), a row apart in a tall one (consecutive threads
// take consecutive rows of the short side).
struct Items {
  int tall, m, n0, ncols, groups, cols;
  int64_t mat;
};
struct Item {
  int r, g, n;                                    // row, group of 8, values in it (0: none)
  int64_t at;
};
// The items of a thread, 256 apart: their place is stepped, not divided out.
struct ItemWalk {
  int fast, fi, si, fstep, sstep;
  __device__ __forceinline__ ItemWalk(const Items& I, int tid) {
    fast = I.tall ? I.m : max(I.groups, 1);
    fi = tid % fast;
    si = tid / fast;
    fstep = 32 * kRsWarps % fast;
    sstep = 32 * kRsWarps / fast;
  }
  __device__ __forceinline__ Item next(const Items& I) {
    Item x;
    x.r = I.tall ? fi : si;
    x.g = I.tall ? si : fi;
    x.n = x.r < I.m && x.g < I.groups ? min(8, I.ncols - 8 * x.g) : 0;
    x.at = I.mat + (I.tall ? static_cast<int64_t>(I.n0 + 8 * x.g) * I.m + x.r
                           : static_cast<int64_t>(x.r) * I.cols + I.n0 + 8 * x.g);
    fi += fstep;
    si += sstep;
    if (fi >= fast) {
      fi -= fast;
      ++si;
    }
    return x;
  }
};

// Gradient and momentum of an item, zeros where there is none.
template <bool VEC>
__device__ __forceinline__ void fetch_item(const MomentumArgs& P, const Items& I, const Item& x, const float* mom,
                                           float (&g)[8], float (&m)[8]) {
  if constexpr (VEC) {                            // whole items: cols is a multiple of 16
    if (x.n > 0) {
      load_grad<true>(P, x.at, 8, g);
      if (mom != nullptr) load_f32<true>(mom, x.at, 8, m);
    }
  } else {
    const int64_t pitch = I.tall ? I.m : 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = m[j] = 0.f;
      if (j < x.n) {
        const int64_t i = x.at + j * pitch;
        g[j] = P.grad_f32 ? static_cast<const float*>(P.grad)[i]
                          : bf16_bits_to_float(static_cast<const uint16_t*>(P.grad)[i]);
        if (mom != nullptr) m[j] = mom[i];
      }
    }
  }
}

constexpr int kRsAhead = 2;                       // items of a thread requested together

template <bool VEC>
__device__ __forceinline__ void momentum_pass(const MomentumArgs& P, const Items& I, int tid, SumSq& sq) {
  ItemWalk walk(I, tid);
  const int items = I.groups * I.m;
#pragma unroll 1
  for (int it = tid; it < items; it += kRsAhead * 32 * kRsWarps) {
    Item x[kRsAhead];
    float g[kRsAhead][8], m[kRsAhead][8];
#pragma unroll
    for (int k = 0; k < kRsAhead; ++k) {
      x[k] = walk.next(I);
      fetch_item<VEC>(P, I, x[k], P.mom_in, g[k], m[k]);
    }
#pragma unroll
    for (int k = 0; k < kRsAhead; ++k) {
      if (x[k].n == 0) continue;
      if (P.mom_out != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[k][j] = P.mom_in != nullptr ? fmaf(P.mu, m[k][j], g[k][j]) : g[k][j];
          g[k][j] = P.nesterov ? fmaf(P.mu, m[k][j], g[k][j]) : m[k][j];
        }
        if constexpr (VEC) {
          st_global_v8(P.mom_out + x[k].at, reinterpret_cast<const uint32_t*>(m[k]));
        } else {
          const int64_t pitch = I.tall ? I.m : 1;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < x[k].n) P.mom_out[x[k].at + j * pitch] = m[k][j];
        }
      }
      sq.add8(g[k]);
    }
  }
}

// X0 = u / |u| 2^ex (its factors in f) into the boxes, the momentum read back.
template <bool SPLIT, bool VEC>
__device__ __forceinline__ void x0_pass(const MomentumArgs& P, const Items& I, int tid, const float (&f)[3],
                                        uint8_t* xs) {
  ItemWalk walk(I, tid);
  const int items = I.groups * I.m;
#pragma unroll 1
  for (int it = tid; it < items; it += kRsAhead * 32 * kRsWarps) {
    Item x[kRsAhead];
    float g[kRsAhead][8], m[kRsAhead][8];
#pragma unroll
    for (int k = 0; k < kRsAhead; ++k) {
      x[k] = walk.next(I);
      fetch_item<VEC>(P, I, x[k], P.mom_out, g[k], m[k]);
    }
#pragma unroll
    for (int k = 0; k < kRsAhead; ++k) {
      if (x[k].n == 0) continue;
      uint32_t h[4], l[4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (P.mom_out != nullptr) g[k][j] = P.nesterov ? fmaf(P.mu, m[k][j], g[k][j]) : m[k][j];
        g[k][j] = g[k][j] * f[0] * f[1] * f[2];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = split_half2(g[k][2 * j], g[k][2 * j + 1], l[j]);
      uint8_t* dst = xs + (x[k].g >> 3) * kRsBox + x[k].r * 128 + swz(x[k].g & 7, x[k].r);
      *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
      if constexpr (SPLIT) *reinterpret_cast<uint4*>(dst + 64 * 128) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
}

// MOST: CTAs of a cluster (8 or 16: the sums of sixteen need registers that cost the others 2 %).
template <bool SPLIT, int MOST>
__global__ void __launch_bounds__(kRsThreads, 1) muon_resident_kernel(const __grid_constant__ ResidentArgs P, int C) {
  extern __shared__ uint8_t raw[];
  uint8_t* xs = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ab = xs + kRsX;
  uint8_t* part = ab + kRsAb;
  uint64_t* bar = reinterpret_cast<uint64_t*>(part + kRsPart);
  double* s_norm = reinterpret_cast<double*>(bar + 1);                // this CTA's sum of squares (read by the cluster)
  double* s_warp = s_norm + 1;
  float* s_f = reinterpret_cast<float*>(s_warp + kRsWarps);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_f + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = C > 1 ? cluster_ctarank() : 0u;
  const int b = blockIdx.x / C;
  const int n0 = static_cast<int>(rank) * P.slice;                    // first column of the long side
  const int ncols = max(0, min(P.slice, P.n - n0));
  const int boxes = P.slice / 64;

  for (int i = tid; i < (boxes * kRsBox + kRsAb) / 16; i += kRsThreads)
    reinterpret_cast<uint4*>(i < boxes * (kRsBox / 16) ? xs : ab - boxes * kRsBox)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kRsWarps) {
    tmem_alloc<1>(tmem_slot, 512);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // ---- momentum, norm, X0
  const Items I{P.tall, P.m, n0, ncols, (ncols + 7) / 8, P.cols, static_cast<int64_t>(b) * P.mo.per};
  const bool vec = !P.tall && P.cols % 16 == 0;
  if (warp < kRsWarps) {
    SumSq sq{0.f, 0.f, 0.f};
    if (vec) momentum_pass<true>(P.mo, I, tid, sq);
    else momentum_pass<false>(P.mo, I, tid, sq);
    double t = sq.total();
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (lane == 0) s_warp[warp] = t;
  }
  __syncthreads();
  if (tid == 0) {
    double t = 0.0;
    for (int w = 0; w < kRsWarps; ++w) t += s_warp[w];
    *s_norm = t;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (tid == 0) {                                                     // one thread: fp64 is slow here
    double n2 = 0.0;
    if (C > 1)
      for (int k = 0; k < C; ++k) n2 += ld_shared_cluster_f64(map_to_rank(smem_u32(s_norm), k));
    else
      n2 = *s_norm;
    float f[3];
    norm_factors(n2, P.ex, f);
    for (int i = 0; i < 3; ++i) s_f[i] = f[i];
  }
  __syncthreads();
  if (warp < kRsWarps) {
    const float f[3] = {s_f[0], s_f[1], s_f[2]};
    if (vec) x0_pass<SPLIT, true>(P.mo, I, tid, f, xs);
    else x0_pass<SPLIT, false>(P.mo, I, tid, f, xs);
  }
  fence_proxy_async_smem();
  __syncthreads();

  // ---- steps.  warp w < 8: TMEM lanes (rows) 32 (w % 4) .., first or second half of the columns
  const int q = warp & 3, hf = warp >> 2;
  const int row = q * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
  const uint64_t xd = smem_desc(smem_u32(xs), 0, 1024, kLayoutSwizzle128B);            // K-major
  const uint64_t xm = smem_desc(smem_u32(xs), kRsBox, 1024, kLayoutSwizzle128B);       // MN-major
  const bool b_low = !SPLIT && muon_b_low(P.m, P.n);
  const uint64_t ad = smem_desc(smem_u32(ab), 0, 1024, kLayoutSwizzle128B);
  const int ksteps = (P.m + 15) / 16;
  uint32_t phase = 0;
  auto wait_mma = [&]() {
    if (!mbar_wait_bounded(bar, phase, abort_flag, kWaitLimitNs) && lane == 0) {       // the barriers below are kept
      report(P.status, MXG_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    phase ^= 1;
    tc_fence_after();
  };
  for (int step = 0; step < P.steps; ++step) {
    const bool last = step + 1 == P.steps;
    if (warp == kRsWarps) {
      if (lane == 0) {
        tc_fence_after();
        for (int i = 0; i < boxes; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t d = xd + ((i * kRsBox + k * 32) >> 4);
            mma_bf16<1>(tmem, d, d, idesc_f16(128, 128), (i | k) != 0 ? 1u : 0u);
          }
        mma_commit<1>(bar);
      }
      __syncwarp();
    } else {
      wait_mma();
      float v[64];
      read64(P.alpha[0], lanes + hf * 64, v);
      // non-SPLIT: [128][128] sums; SPLIT: blocks (high, high), (high, low), (low, high) of [64][64]
      if (SPLIT ? q < 2 || hf == 0 : C > 1) {
        uint8_t* dst = SPLIT ? part + (q < 2 ? hf : 2) * 16384 + (row & 63) * 256 : part + row * 512;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          *reinterpret_cast<float4*>(dst + swz(SPLIT ? j : hf * 16 + j, row)) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      }
      if constexpr (!SPLIT) {
        if (C == 1) {
          // A as an operand at once
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(ab + hf * kRsBox + row * 128 + swz(j, row)) =
                make_uint4(half2_bits(v[8 * j], v[8 * j + 1]), half2_bits(v[8 * j + 2], v[8 * j + 3]),
                           half2_bits(v[8 * j + 4], v[8 * j + 5]), half2_bits(v[8 * j + 6], v[8 * j + 7]));
        }
      }
    }
    // SPLIT: thread t adds the three blocks for 16 columns of row t / 4
    const int sr = tid >> 2, sp = 4 * (tid & 3);
    if constexpr (SPLIT) {
      __syncthreads();
      if (warp < kRsWarps)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float4* p = reinterpret_cast<float4*>(part + sr * 256 + swz(sp + j, sr));
          const float4 x = p[0], y = p[1024], z = p[2048];
          p[0] = make_float4(x.x + (y.x + z.x), x.y + (y.y + z.y), x.z + (y.z + z.z), x.w + (y.w + z.w));
        }
    }
    if (C > 1) cluster_sum<SPLIT ? 64 : 128, MOST>(part, C, rank, tid);
    if (warp < kRsWarps) {
      if constexpr (SPLIT) {
        // (C = 1: the thread's own sums; else the cluster's, behind its barrier)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 x = *reinterpret_cast<const float4*>(part + sr * 256 + swz(sp + 2 * j, sr));
          const float4 y = *reinterpret_cast<const float4*>(part + sr * 256 + swz(sp + 2 * j + 1, sr));
          uint32_t h[4], l[4];
          h[0] = split_half2(x.x, x.y, l[0]);
          h[1] = split_half2(x.z, x.w, l[1]);
          h[2] = split_half2(y.x, y.y, l[2]);
          h[3] = split_half2(y.z, y.w, l[3]);
          uint8_t* dst = ab + sr * 128 + swz(sp / 2 + j, sr);
          *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + kRsBox) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      } else if (C > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 x = *reinterpret_cast<const float4*>(part + row * 512 + swz(hf * 16 + 2 * j, row));
          const float4 y = *reinterpret_cast<const float4*>(part + row * 512 + swz(hf * 16 + 2 * j + 1, row));
          *reinterpret_cast<uint4*>(ab + hf * kRsBox + row * 128 + swz(j, row)) =
              make_uint4(half2_bits(x.x, x.y), half2_bits(x.z, x.w), half2_bits(y.x, y.y), half2_bits(y.z, y.w));
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();

    // ---- B = a I + b A + c A A, in A's place
    if (warp == kRsWarps) {
      if (lane == 0) {
        tc_fence_after();
        for (int p = 0; p < (SPLIT ? 3 : 1); ++p) {          // (high, low), (low, high), (high, high)
          const uint64_t pa = ad + (SPLIT && p == 1 ? kRsBox >> 4 : 0), qa = ad + (SPLIT && p == 0 ? kRsBox >> 4 : 0);
#pragma unroll
          for (int k = 0; k < (SPLIT ? 4 : 8); ++k) {
            const uint32_t off = ((k >> 2) * kRsBox + (k & 3) * 32) >> 4;
            if (k < ksteps)
              mma_bf16<1>(tmem + 128, pa + off, qa + off, idesc_f16(128, SPLIT ? 64 : 128), (p | k) != 0 ? 1u : 0u);
          }
        }
        mma_commit<1>(bar);
      }
      __syncwarp();
    } else {
      wait_mma();
      if constexpr (SPLIT) {
        if (q < 2) {                                         // row < 64, columns 32 hf ..
          uint32_t r[32];
          tmem_ld_32x32b_x32(lanes + 128 + 32 * hf, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j) {                      // eight columns
            const float4 x = *reinterpret_cast<const float4*>(part + row * 256 + swz(8 * hf + 2 * j, row));
            const float4 y = *reinterpret_cast<const float4*>(part + row * 256 + swz(8 * hf + 2 * j + 1, row));
            const float a[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = fmaf(P.beta, a[i], P.alpha[1] * __uint_as_float(r[8 * j + i])) +
                     (row < P.m && row == 32 * hf + 8 * j + i ? P.diag : 0.f);
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = split_half2(v[2 * i], v[2 * i + 1], l[i]);
            uint8_t* dst = ab + row * 128 + swz(4 * hf + j, row);
            *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + kRsBox) = make_uint4(l[0], l[1], l[2], l[3]);
          }
        }
      } else {
        float v[64];
        read64(P.alpha[1], lanes + 128 + hf * 64, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4* p = reinterpret_cast<uint4*>(ab + hf * kRsBox + row * 128 + swz(j, row));
          const uint4 a4 = *p;                               // the A that was multiplied: eleven bits, as the product saw it
          const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w};
          uint32_t o[4], l[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 af = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
            const int c = hf * 64 + 8 * j + 2 * i;
            o[i] = split_half2(fmaf(P.beta, af.x, v[8 * j + 2 * i]) + (row < P.m && row == c ? P.diag : 0.f),
                               fmaf(P.beta, af.y, v[8 * j + 2 * i + 1]) + (row < P.m && row == c + 1 ? P.diag : 0.f), l[i]);
          }
          *p = make_uint4(o[0], o[1], o[2], o[3]);
          // B's low part, where the sums were
          if (b_low)
            *reinterpret_cast<uint4*>(part + hf * kRsBox + row * 128 + swz(j, row)) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();

    // ---- X' = B X
    if (warp == kRsWarps) {
      if (lane == 0) {
        tc_fence_after();
        for (int c = 0; c < P.slice; c += 256) {
          const uint32_t id = idesc_f16(128, min(256, P.slice - c)) | kIdescBMn;
          const uint64_t qb = xm + (c / 64 * kRsBox >> 4);
          const int p0 = SPLIT || b_low ? 0 : 1;
          for (int p = p0; p < (SPLIT ? 3 : 2); ++p) {      // one part of X: B's low part, then its high part
            const uint64_t pa = SPLIT ? ad + (p == 1 ? kRsBox >> 4 : 0) : p == 0 ? ad + (kRsAb >> 4) : ad;
            const uint64_t qa = qb + (SPLIT && p == 0 ? 64 * 128 >> 4 : 0);            // low parts: rows 64 ..
#pragma unroll
            for (int k = 0; k < (SPLIT ? 4 : 8); ++k)
              if (k < ksteps)
                mma_bf16<1>(tmem + c, pa + (((k >> 2) * kRsBox + (k & 3) * 32) >> 4), qa + k * (2048 >> 4), id,
                            p != p0 || k != 0 ? 1u : 0u);
          }
        }
        mma_commit<1>(bar);
      }
      __syncwarp();
    } else {
      wait_mma();
      if (!SPLIT || q < 2)
        for (int i = hf; i < boxes; i += 2) {
          float v[64];
          read64(last ? P.alpha_last : P.alpha[2], lanes + 64 * i, v);
          if (last) {
            if (q * 32 < P.m && 64 * i < ncols)
              write_out(P, v, reinterpret_cast<float*>(part) + warp * 32 * 33, b, q * 32, n0 + 64 * i, lane);
            continue;
          }
          uint8_t* dst = xs + i * kRsBox + row * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (SPLIT) h[e] = split_half2(v[8 * j + 2 * e], v[8 * j + 2 * e + 1], l[e]);
              else h[e] = half2_bits(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
            }
            *reinterpret_cast<uint4*>(dst + swz(j, row)) = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (SPLIT) *reinterpret_cast<uint4*>(dst + 64 * 128 + swz(j, row)) = make_uint4(l[0], l[1], l[2], l[3]);
          }
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
  }
  tc_fence_after();
  if (C > 1) cluster_sync();
  if (warp == kRsWarps) tmem_dealloc<1>(tmem, 512);
}

template <bool SPLIT, int MOST>
cudaError_t launch(const ResidentArgs& a, int C, cudaStream_t s) {
  auto kern = muon_resident_kernel<SPLIT, MOST>;
  cudaError_t err = allow_smem(kern, kRsSmem);
  if (err == cudaSuccess && MOST > 8) err = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch * C));
  cfg.blockDim = dim3(kRsThreads);
  cfg.dynamicSmemBytes = kRsSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, kern, a, C);
  count_launch();
  return err != cudaSuccess ? err : cudaGetLastError();
}

// Clusters of C CTAs that the device holds at once (asked once; a cluster lies
// within one part of the chip, so 152 SMs hold 76 of two, but 36 of four and 15
// of eight).
int clusters_at_once(int C) {
  static std::atomic<int> known[64][5];   // one more than the answer
  int log = 0;
  while (1 << log < C) ++log;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return device_sms() / C;
  if (dev < 64 && (n = known[dev][log].load()) > 0) return n - 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(C));
  cfg.blockDim = dim3(kRsThreads);
  cfg.dynamicSmemBytes = kRsSmem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = C > 8 ? muon_resident_kernel<true, kRsCluster> : muon_resident_kernel<true, 8>;
  if (allow_smem(kern, kRsSmem) != cudaSuccess ||
      (C > 8 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return C > 8 ? 0 : device_sms() / C;
  }
  if (dev < 64) known[dev][log].store(n + 1);
  return n;
}

}  // namespace

// Measured (five steps, us): more CTAs per matrix than its size needs pay off
// while the device holds all clusters at once, 1 x 64 x 512 64 (one CTA) 50 (two)
// 38 (eight), 2 x 128 x 1024 80 (two) 54 (eight), 19 x 64 x 1024 52 (four) 79
// (eight, in turns), except up to 256 columns of more than 64 rows: 4 x 128 x 256
// 41 (one) 46 (four), where the 128 x 128 sums cost more than they spare.  Around
// that edge, one / two / four / eight CTAs (the same for 1 and 4 matrices):
//   72 x 256 35 46 45 49    96 x 256 39 47 45 50    128 x 256 41 48 47 50
//   72 x 257 45 54 52 52    96 x 257 48 58 52 52    128 x 257 54 60 56 52
//   72 x 400 50 54 48 49    96 x 400 52 56 49 49    128 x 400 58 60 51 50
//   72 x 512 54 54 49 50    96 x 512 58 56 49 50    128 x 512 64 60 52 50
// so eight cost up to 13 % just past 256 columns of fewer than 128 rows.  Those
// sums also make clusters that need several turns slower than the tiled kernel:
// 16 x 100 x 3000 183 against 132, 64 x 128 x 4096 499 against 405 (in one turn
// 30 x 128 x 2000 92 against 133); 64 x 64 x 2048 is 150 against 232.  Sixteen
// CTAs, of which the device holds seven clusters, only where eight are too few
// (6 x 128 x 6000 91 against 129) and in one turn.
int resident_cluster(int batch, int m, int n, bool split) {
  if (m > 128 || n > kResidentMost) return 0;
  int C = 1;
  while (C * kRsSlice < n) C *= 2;
  if (C > 8 ? batch > clusters_at_once(C) : !split && C > 1 && batch > clusters_at_once(C)) return 0;
  if (split || n > 256)
    while (C < 8 && C * 64 < n && batch <= clusters_at_once(2 * C)) C *= 2;
  return C;
}

cudaError_t launch_muon_resident(ResidentArgs a, int C, bool split, cudaStream_t s) {
  a.tall = a.rows > a.cols;
  a.m = a.tall ? a.cols : a.rows;
  a.n = a.tall ? a.rows : a.cols;
  a.slice = ((a.n + C - 1) / C + 63) / 64 * 64;
  if (C > 8) return split ? launch<true, kRsCluster>(a, C, s) : launch<false, kRsCluster>(a, C, s);
  return split ? launch<true, 8>(a, C, s) : launch<false, 8>(a, C, s);
}

}  // namespace mxg
