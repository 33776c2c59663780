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
// one above (see ns_mn_stages).
//
// Number format.  Operands are fp16: X, A and B are bounded (|X|_F = 1 at the
// start, singular values at most ~1.2 afterwards), so the eleven-bit
// significand is worth more than bf16's range, and each is stored times a
// power of two that puts its entries well inside fp16's normal range:
//   X 2^ex, 2^ex ~ sqrt(N)  (an orthogonal X has entries of size 1 / sqrt(N)),
//   A 2^12, B 2^12          (entries at most ~1.5 and ~5).
// Folding a I into B rounds a + B_ii to eleven bits, an error of the size of
// X's own rounding, and spares the last product a second read of X.
// One part serves gradients whose singular values are of one size (2.0-2.5e-3 of
// the update, 1.66e-3 of it bf16's rounding).  Directions that are nearly empty
// fill with X0's rounding, 1.7e-4 of its norm, and are multiplied by up to a^5 =
// 485: 0.15 of a rank-1 update, 0.04 at rank 8, 4e-3 for singular values 1 / i.
// Two parts of X in the first three steps would take 6 products more than the 15
// (of m x m x n) of a long matrix; up to 64 rows, where a tile has room for both
// parts, all operands have two and only the result's rounding is left.
// Sums are fp32 (tensor-core accumulators); momentum and norms are fp32/fp64.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "api_common.h"
#include "kernels.h"
#include "muon.cuh"
#include "ptx.cuh"

namespace mxg {
namespace {

// The products' counters lie a cache line apart: waiting CTAs read them without
// pause, and side by side the matrices slowed each other down (60 x 200 x 200,
// 128-wide tiles: 148 us, 103 apart; 20 x 300 x 300 121 and 96).
constexpr int kNsLine = 32;

// New momentum and the sum of squares of u: one partial per block; the
// products' counters are cleared.  Groups of eight elements are counted from the
// start of the whole batch, so that they lie on 32 bytes of every buffer
// whatever the size of a matrix; what is left of a matrix at its two ends goes
// to its first block, one element a thread.  HBM bounds it: 64 x 2048 x 1024 with
// bf16 gradients 210 us, 6.4 TB/s.
__global__ void __launch_bounds__(kMoThreads) momentum_kernel(MomentumArgs P, int chunks, double* __restrict__ part,
                                                             int32_t* __restrict__ done, int n_done) {
  if (blockIdx.x == 0)
    for (int i = blockIdx.y * kMoThreads + threadIdx.x; i < n_done; i += gridDim.y * kMoThreads) done[i] = 0;
  const int64_t start = static_cast<int64_t>(blockIdx.y) * P.per, end = start + P.per;
  const int64_t lo = (start + kMoVec - 1) / kMoVec * kMoVec;                   // the whole groups are [lo, hi)
  const int64_t hi = end / kMoVec * kMoVec > lo ? end / kMoVec * kMoVec : lo;
  SumSq s{0.f, 0.f, 0.f};
  for (int64_t i = lo + (static_cast<int64_t>(blockIdx.x) * kMoThreads + threadIdx.x) * kMoVec; i < hi;
       i += static_cast<int64_t>(chunks) * kMoThreads * kMoVec) {
    float u[kMoVec];
    step_momentum<true>(P, i, kMoVec, u);
    s.add8(u);
  }
  if (blockIdx.x == 0 && threadIdx.x < 2 * kMoVec) {
    const int64_t i = threadIdx.x < kMoVec ? start + threadIdx.x : hi + threadIdx.x - kMoVec;
    if (threadIdx.x < kMoVec ? i < lo && i < end : i < end) {
      float u[kMoVec];
      step_momentum<false>(P, i, 1, u);
#pragma unroll
      for (int j = 1; j < kMoVec; ++j) u[j] = 0.f;
      s.add8(u);
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

// X0 = u / |u|_F 2^ex in fp16, rows ld apart.  A block's first act is the
// matrix's norm from the partials (the same sum, in the same order, in every
// block).  VEC: rows of whole groups of eight elements, which lie on 32 bytes of
// every buffer.  Otherwise 32 lanes take 32 elements side by side, eight in
// flight, and step through rows and columns (groups along the rows were 2-4 %
// of the whole update slower, 40 x 511 x 770 340 us against 325).  It reads the
// gradient and the new momentum again: 64 x 2048 x 1024 156 us, 6.9 TB/s.  (u cannot be written in fp16
// before its norm is known, and in fp32 it costs more bytes.)
template <bool VEC>
__global__ void __launch_bounds__(kMoThreads) cast_kernel(MomentumArgs P, int chunks, const double* __restrict__ part,
                                                         int ex, int rows, int cols, __half* __restrict__ x,
                                                         int64_t ld, int64_t lo_off) {
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
    float f[3];
    norm_factors(n2, ex, f);
    for (int i = 0; i < 3; ++i) s_f[i] = f[i];
  }
  __syncthreads();
  const float f0 = s_f[0], f1 = s_f[1], f2 = s_f[2];
  if constexpr (!VEC) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kMoThreads;
    const int64_t dr = stride / cols;
    const int dc = static_cast<int>(stride - dr * cols);
    int64_t e = static_cast<int64_t>(blockIdx.x) * kMoThreads + threadIdx.x;
    int64_t r = e / cols;
    int c = static_cast<int>(e - r * cols);
    const int64_t per = P.per;
    __half* dst = x + static_cast<int64_t>(b) * rows * ld;
    while (e < per) {
      float u[kMoVec];
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) u[j] = e + j * stride < per ? momentum_u1(P, b * per + e + j * stride) : 0.f;
#pragma unroll
      for (int j = 0; j < kMoVec; ++j) {
        if (e < per) {
          const float v = u[j] * f0 * f1 * f2;
          const __half h = __float2half_rn(v);
          dst[r * ld + c] = h;
          if (lo_off != 0) dst[r * ld + c + lo_off] = __float2half_rn(v - __half2float(h));
        }
        e += stride;
        r += dr;
        c += dc;
        if (c >= cols) {
          c -= cols;
          ++r;
        }
      }
    }
    return;
  }
  const int groups = cols / kMoVec;                         // of a row
  const int64_t total = static_cast<int64_t>(rows) * groups;
  for (int64_t gi = static_cast<int64_t>(blockIdx.x) * kMoThreads + threadIdx.x; gi < total;
       gi += static_cast<int64_t>(gridDim.x) * kMoThreads) {
    const int64_t r = gi / groups;
    const int c = static_cast<int>(gi - r * groups) * kMoVec;
    float u[kMoVec];
    momentum_u8(P, b * P.per + r * cols + c, u);
    uint32_t h[kMoVec / 2], l[kMoVec / 2];
#pragma unroll
    for (int j = 0; j < kMoVec / 2; ++j) h[j] = split_half2(u[2 * j] * f0 * f1 * f2, u[2 * j + 1] * f0 * f1 * f2, l[j]);
    // ld is a multiple of 16, so a group of eight starts on 16 bytes and fits the row's padding
    __half* dst = x + (static_cast<int64_t>(b) * rows + r) * ld + c;
    *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
    if (lo_off != 0) *reinterpret_cast<uint4*>(dst + lo_off) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// ------------------------------------------------------------------ products
// D = P Q^T over fp16 operands, tiles of 128 x 64 or 128 x 128 on one SM or 256
// x 256 on a CTA pair (cta_group::2, each SM holding its 128 rows of both
// operands).
// Warps 0 and 2 issue TMA, warp 1 owns TMEM and issues the MMAs, warps 4-11 run
// the epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 and half of the tile's
// columns.  The accumulator is double-buffered in TMEM.
//
// What bounds them: long contractions the tensor cores and the power cap (1 x
// 28672 x 4096, X X^T 1.66-1.81 PFLOP/s, all five steps 1.55), a pair's tiles of
// K = 1024 the refill of stages that MMAs hold while they read them (40-48 bytes a
// cycle and SM, 64 at the full rate: the MMAs alone need 8.2 k cycles a tile, with
// their loads 11-13 k; 64 x 2048 x 1024 1.9 ms for five steps, 1.35 PFLOP/s), small and middling matrices the hand-over from product
// to product: 1.0 k cycles to see the count, 1.3 k for the first loads, 0.7 k
// from the last MMA to the epilogue, 1.2 k there, 1.8 k for the release (3 x 1001
// x 333: 97 us, 15 products).  TMA boxes instead of plain stores for the small
// tiles are 1-8 % slower there, a sixth stage or a third loading warp no faster.
//
// One launch runs all products of all steps: the tiles of the whole run form
// one list that the CTAs (or pairs) deal out in turn, so a product's last
// tiles overlap the next one's first, and a small matrix pays no launch per
// product.  A tile needs the earlier products of its own matrix: every epilogue
// warp adds one to the matrix's counter once its part is in memory, and the
// loads wait for the count of the products before.  What a tile waits for is
// earlier in the list and the launch is cooperative (all CTAs resident), so
// the waits end.  Every wait is bounded all the same; one that gives up
// records MXG_ERR_TIMEOUT and stops the CTA's pipeline.
//
// An operand's 128 rows x 64 contraction elements come as two 64 x 64 boxes of
// 128-byte swizzled rows, 8 KB each.  K-major: box h holds rows 64 h ..; the
// two follow one another as 128 rows of 128 bytes (8-row groups 1024 bytes
// apart; a K = 16 step is 32 bytes).  MN-major: box h holds the 64 contraction
// rows of operand rows 64 h .. (leading offset 8192 between them, 8-row groups
// 1024 bytes apart; a K = 16 step is 16 rows, 2048 bytes).
//
// X X^T has the fewest tiles and the longest contraction.  Where SMs would be
// idle, or the contraction is too long for one accumulator (kNsLongest), several
// CTAs share it: each leaves its fp32 sums in global memory, and the one that is
// last to do so adds them up in order.
//
// FUSED (a short side of at most 128): A is one tile, so both operands of
// X X^T are the same 128 rows.  They are loaded once, and a stage holds 128
// contraction elements instead of 64 of each operand.  SPLIT (at most 64):
// the 128 rows are the high and the low parts, so one product yields all
// pairs of parts, and A = (high, high) + (high, low) + (low, high).
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
// FUSED, in the store boxes' place: A as an operand (128 x 128; SPLIT: 64 columns
// of its high part, then of its low part, then the two 64 x 64 fp32 blocks that
// are added to the third)
constexpr int kNsALow = kNsOpBytes;
constexpr int kNsSwap = 2 * kNsOpBytes;
static_assert(kNsSwap + 2 * 64 * 64 * 4 <= 8 * kNsWarpOut, "A and the blocks added to it");
static_assert(32 * 33 * 4 <= kNsWarpOut, "unaligned outputs stage 32 x 32 fp32 values");

// How an operand lies in memory.
enum NsForm { NS_K = 0,                   // [rows][k]
              NS_MN = 1,                  // [k][rows]
              NS_SYM = 2 };               // symmetric [rows][rows], blocks on and above the diagonal

// The three products of a step, in order.
enum NsOp { NS_GRAM = 0, NS_POLY = 1, NS_APPLY = 2 };

struct NsArgs {
  CUtensorMap x[2], a, b;                 // loads: 64 x 64 boxes
  CUtensorMap xs[2], as, bs, out;         // stores: 64 columns x 32 rows
  int rows, cols, m;                      // X [rows][cols], m the short side
  int tall;                               // rows > cols
  int batch, steps;
  int sym_tiles;                          // tiles of A (and of B) of one matrix; FUSED: CTAs that share A's contraction
  int splits;                             // not FUSED: CTAs (pairs) that share the contraction of a tile of A
  float* a_parts;                         // FUSED, sym_tiles > 1: their sums [batch][sym_tiles][side][side];
                                          // splits > 1: [batch][sym_tiles][pair's CTA][splits][128 x BN]
  int app_m, app_n;                       // row and column tiles of X
  float alpha[3], alpha_last;             // each product's factor on the accumulators
  float beta, diag;                       // POLY: + beta A + diag I
  uint16_t *xp[2], *ap, *bp;              // X, A, B; rows ldx and lda apart (multiples of 16), low parts low_x, low_a on
  int64_t ldx, lda, low_x, low_a;
  uint16_t* update;                       // bf16 [batch][rows][cols], nullable
  const uint16_t* w_in;
  uint16_t* w_out;                        // nullable: w_in * w_keep - lr * value
  float w_keep, lr;
  int b_low;                              // FUSED, not SPLIT: B has a low part
  int32_t* done;                          // [batch]: epilogue warps that have stored their part of a tile
  int32_t* shares;                        // [batch] (splits: [batch][sym_tiles][pair's CTA]): CTAs that have left their sum
  int32_t* status;
};

struct NsTile {
  int step, op, b, ti, tj;
  int share;                              // NS_GRAM: which part of the contraction
  int tile;                               // NS_GRAM, splits: which tile of A, of all matrices
  int need;                               // done[b] once every earlier product of the matrix is stored
};

// First column tile of row tile ti of a symmetric matrix: small tiles fill the
// diagonal blocks of kNsSym as well.
template <int TM, int BN>
__host__ __device__ __forceinline__ int ns_first(int ti) {
  return ti * TM / kNsSym * (kNsSym / BN);
}

// Tile t of the whole run: step by step, product by product, matrix by matrix.
// FUSED: A and B are one tile, computed together under NS_GRAM by sym_tiles
// CTAs, of which one finishes it.
template <int TM, int BN, bool FUSED>
__device__ __forceinline__ NsTile ns_tile(const NsArgs& P, int64_t t) {
  constexpr int kArrive = TM / 16;        // epilogue warps of a tile (BN = 64: half as many, that count twice)
  constexpr int kSyms = FUSED ? 1 : 2;    // products before the last
  NsTile r;
  const int app = P.app_m * P.app_n;
  const int64_t sym_all = static_cast<int64_t>(P.sym_tiles) * P.batch;
  const int splits = FUSED ? 1 : P.splits;
  const int64_t extra = (splits - 1) * sym_all;                               // tiles of A that others share
  const int64_t per_step = extra + kSyms * sym_all + static_cast<int64_t>(app) * P.batch;
  r.step = static_cast<int>(t / per_step);
  int64_t l = t - r.step * per_step - extra;
  const int before = l < sym_all ? 0 : l < kSyms * sym_all ? 1 : kSyms;       // products of the step
  r.op = before == kSyms ? NS_APPLY : before;
  r.share = r.tile = 0;
  if (splits > 1 && before == 0) {
    l += extra;
    r.tile = static_cast<int>(l / splits);
    r.share = static_cast<int>(l - static_cast<int64_t>(r.tile) * splits);
    l = r.tile;
  }
  l -= before * sym_all;
  const int syms = FUSED ? 1 : P.sym_tiles;                                   // tiles that are stored
  r.need = kArrive * (r.step * (kSyms * syms + app) + before * syms);
  if (r.op != NS_APPLY) {
    r.b = static_cast<int>(l / P.sym_tiles);
    int i = static_cast<int>(l - static_cast<int64_t>(r.b) * P.sym_tiles);
    const int tiles = (P.m + BN - 1) / BN;
    r.ti = 0;
    if (FUSED) {
      r.share = i;
      i = 0;
    }
    while (i >= tiles - ns_first<TM, BN>(r.ti)) {
      i -= tiles - ns_first<TM, BN>(r.ti);
      ++r.ti;
    }
    r.tj = ns_first<TM, BN>(r.ti) + i;
  } else {
    // the short side's tiles vary fastest: B stays in L2, X streams
    r.b = static_cast<int>(l / app);
    const int i = static_cast<int>(l - static_cast<int64_t>(r.b) * app);
    const int f = P.tall ? P.app_n : P.app_m;
    r.ti = P.tall ? i / f : i % f;
    r.tj = P.tall ? i % f : i / f;
  }
  return r;
}

struct NsOperands {
  const CUtensorMap *p, *q;
  int p_form, q_form;
  int nk;                                 // stages of the contraction, of one pair of parts
};

__device__ __forceinline__ NsOperands ns_operands(const NsArgs& P, const NsTile& tc) {
  const CUtensorMap* x = &P.x[tc.step & 1];
  const int short_k = (P.m + kNsK - 1) / kNsK;
  if (tc.op == NS_GRAM) {
    const int f = P.tall ? NS_MN : NS_K;
    return {x, x, f, f, ((P.tall ? P.rows : P.cols) + kNsK - 1) / kNsK};
  }
  if (tc.op == NS_POLY) return {&P.a, &P.a, NS_SYM, NS_SYM, short_k};
  if (P.tall) return {x, &P.b, NS_K, NS_SYM, short_k};
  return {&P.b, x, NS_SYM, NS_MN, short_k};
}

// First stage of a share of A: of sym_tiles (FUSED, stages of 128 contraction elements) or of splits.
template <bool FUSED>
__device__ __forceinline__ int ns_share_begin(const NsArgs& P, const NsOperands& o, int share) {
  return FUSED ? (o.nk + 1) / 2 * share / P.sym_tiles : o.nk * share / P.splits;
}

// Waits until the products before tile tc of its matrix are in memory.
__device__ __forceinline__ bool ns_wait_done(const NsArgs& P, const NsTile& tc, volatile int* abort) {
  const int32_t* c = P.done + tc.b * kNsLine;
  if (ld_acquire_gpu(c) >= tc.need) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    for (int i = 0; i < 32; ++i)          // the clock is read now and then: it takes longer than the count
      if (ld_acquire_gpu(c) >= tc.need) return true;
    if (*abort || globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

// How many stages of 64 contraction elements of operand rows row0 .. are read
// MN-major, from the first on: below the diagonal a symmetric matrix holds
// nothing, and the block (rows, k) is the transpose of (k, rows).
__device__ __forceinline__ int ns_mn_stages(int form, int row0) {
  return form == NS_MN ? INT_MAX : form == NS_SYM ? row0 / kNsSym * (kNsSym / kNsK) : 0;
}

template <bool PEER, int BOXES>
__device__ __forceinline__ void ns_load(uint8_t* dst, const CUtensorMap* map, bool mn, int row0, int k0, int b,
                                        uint64_t* bar, uint32_t peer_bar) {
#pragma unroll
  for (int h = 0; h < BOXES; ++h) {
    const int x = mn ? row0 + 64 * h : k0, y = mn ? k0 : row0 + 64 * h;
    if (PEER) tma_load_3d_pair(dst + h * kNsBoxBytes, map, x, y, b, peer_bar);
    else tma_load_3d(dst + h * kNsBoxBytes, map, x, y, b, bar);
  }
}

// 64 columns of a row, zero past the matrix's edge (whole 32-byte pieces: rows
// are padded to 16), through L2: other SMs wrote A during this kernel.
__device__ __forceinline__ void ns_load_row(const void* base, int64_t off, bool in, int col, int n,
                                            uint32_t (&w)[32]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (in && col + 16 * h < n) {
      ld_global_cg_v8(static_cast<const uint16_t*>(base) + off + 16 * h, w + 8 * h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[8 * h + i] = 0u;
    }
  }
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

// The same (or 32 columns) by plain stores, 32 bytes at a time (rows are padded to 16).
template <int HALVES = 2>
__device__ __forceinline__ void ns_store_direct(const uint32_t (&h)[32], uint16_t* dst, bool in, int col, int n) {
#pragma unroll
  for (int j = 0; j < 2 * HALVES; ++j)
    if (in && col + 16 * j < n) st_global_v8(dst + 16 * j, h + 8 * j);
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
  const int ny = min(32, P.rows - row0);
  const bool in = col0 + lane < P.cols;
  const int64_t base = (static_cast<int64_t>(b) * P.rows + row0) * P.cols + col0 + lane;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    if (i < ny && in) {
      const float x = buf[i * 33 + lane];
      const int64_t u = base + static_cast<int64_t>(i) * P.cols;
      if (P.update != nullptr) P.update[u] = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
      if (P.w_out != nullptr)
        P.w_out[u] =
            static_cast<uint16_t>(pack_bf16x2(fmaf(-P.lr, x, bf16_bits_to_float(P.w_in[u]) * P.w_keep), 0.f));
    }
  }
}

// What an epilogue warp does with its 32 rows x 64 columns of a tile.
enum NsKind { NS_STORE,                   // alpha acc to fp16
              NS_POLYNOMIAL,              // alpha acc + beta A + diag I to fp16
              NS_UPDATE,                  // alpha acc to bf16
              NS_WEIGHTS,                 // w_in * w_keep - lr alpha acc to bf16
              NS_BY_ROWS };               // update and / or weights by plain stores

// Where 64 columns of a tile go: by TMA through shared-memory boxes, or (DIRECT)
// by plain stores to rows `ld` apart of a matrix [rows][cols], low parts `low`
// elements further on.
struct NsDst {
  const CUtensorMap* map;
  uint16_t* p;
  int rows, cols;
  int64_t ld, low;
};

// Requests the addend, lets ready() wait for the accumulator, reads the 64
// columns from TMEM at taddr, lets release() run once they are in registers,
// and stores them (row0, col: of D; any: the block is not wholly outside it).
// KEPT: the polynomial's A is already in w (and wl), zero outside the matrix.
template <int KIND, bool SPLIT, bool DIRECT, bool KEPT, typename W, typename F>
__device__ __forceinline__ bool ns_epilogue(const NsArgs& P, float alpha, uint32_t taddr, uint8_t* boxes,
                                            uint32_t& flip, const NsDst& dst, int row0, int col, int b, bool any,
                                            int lane, uint32_t (&w)[32], uint32_t (&wl)[SPLIT ? 32 : 1], W ready,
                                            F release) {
  if constexpr (KIND == NS_POLYNOMIAL && !KEPT) {
    const bool in = row0 + lane < P.m;
    const int64_t off = (static_cast<int64_t>(b) * P.m + row0 + lane) * P.lda + col;
    ns_load_row(P.ap, off, in, col, P.m, w);
    if constexpr (SPLIT) ns_load_row(P.ap + P.low_a, off, in, col, P.m, wl);
  }
  if constexpr (KIND == NS_WEIGHTS)
    ns_load_row(P.w_in, (static_cast<int64_t>(b) * P.rows + row0 + lane) * P.cols + col, row0 + lane < P.rows, col,
                P.cols, w);
  if (!ready()) return false;
  // KEPT and one part of A: B may have a low part all the same
  constexpr bool B_LOW = KIND == NS_POLYNOMIAL && KEPT && !SPLIT;
  uint32_t h[32], l[SPLIT || B_LOW ? 32 : 1];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + 32 * half, r);
    tmem_ld_wait();
    if (half == 1) release();
    if constexpr (KIND == NS_BY_ROWS) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = alpha * __uint_as_float(r[i]);
      if (any && col + 32 * half < P.cols)
        ns_store_rows(P, v, reinterpret_cast<float*>(boxes), row0, col + 32 * half, b, lane);
    } else {
      const int d = row0 + lane - col - 32 * half;             // row - column of the first value
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 16 * half + i;
        float x = alpha * __uint_as_float(r[2 * i]), y = alpha * __uint_as_float(r[2 * i + 1]);
        if constexpr (KIND == NS_POLYNOMIAL) {
          float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          if constexpr (SPLIT) {
            const float2 al = __half22float2(*reinterpret_cast<const __half2*>(&wl[j]));
            a.x += al.x;
            a.y += al.y;
          }
          x = fmaf(P.beta, a.x, x) + (d == 2 * i ? P.diag : 0.f);
          y = fmaf(P.beta, a.y, y) + (d == 2 * i + 1 ? P.diag : 0.f);
        }
        if constexpr (KIND == NS_WEIGHTS) {
          x = fmaf(-P.lr, x, __uint_as_float(w[j] << 16) * P.w_keep);
          y = fmaf(-P.lr, y, __uint_as_float(w[j] & 0xffff0000u) * P.w_keep);
        }
        if constexpr (KIND == NS_UPDATE || KIND == NS_WEIGHTS) {
          h[j] = pack_bf16x2(x, y);
        } else if constexpr (SPLIT || B_LOW) {
          h[j] = split_half2(x, y, l[j]);
        } else {
          const __half2 v = __floats2half2_rn(x, y);
          h[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
    }
  }
  constexpr bool LOW = SPLIT && (KIND == NS_STORE || KIND == NS_POLYNOMIAL);
  if constexpr (KIND != NS_BY_ROWS) {
    if constexpr (DIRECT) {
      const bool in = row0 + lane < dst.rows;
      uint16_t* p = dst.p + (static_cast<int64_t>(b) * dst.rows + row0 + lane) * dst.ld + col;
      ns_store_direct(h, p, in, col, dst.cols);
      if constexpr (LOW) ns_store_direct(l, p + dst.low, in, col, dst.cols);
      if constexpr (B_LOW)
        if (P.b_low) ns_store_direct(l, p + dst.low, in, col, dst.cols);
    } else if (any) {
      ns_store_box(h, boxes + flip * kNsOut, dst.map, row0, col, b, lane);
      flip ^= 1;
      if constexpr (LOW) {
        ns_store_box(l, boxes + flip * kNsOut, dst.map, row0, col, b + P.batch, lane);
        flip ^= 1;
      }
    }
  }
  return true;
}

// FUSED: this lane's row of 32 rows x 64 columns of the accumulator, scaled.
__device__ __forceinline__ void ns_read64(float alpha, uint32_t taddr, float (&v)[64]) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr + 32 * half, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[32 * half + i] = alpha * __uint_as_float(r[i]);
  }
}

// FUSED: 64 values of a row of A (columns col ..) to registers (h, low parts l)
// and to shared memory as an operand: boxes of 64 columns, 128-byte swizzle.
// Whatever lies outside the matrix becomes zero, since it is contracted over.
template <bool SPLIT>
__device__ __forceinline__ void ns_keep_a(const NsArgs& P, const float (&v)[64], uint8_t* abuf, int row, int col,
                                          uint32_t (&h)[32], uint32_t (&l)[SPLIT ? 32 : 1]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int c = col + 2 * i;
    const float x = row < P.m && c < P.m ? v[2 * i] : 0.f;
    const float y = row < P.m && c + 1 < P.m ? v[2 * i + 1] : 0.f;
    if constexpr (SPLIT) {
      h[i] = split_half2(x, y, l[i]);
    } else {
      const __half2 p = __floats2half2_rn(x, y);
      h[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  uint8_t* dst = abuf + (col >> 6) * kNsOpBytes + row * 128;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint8_t* p = dst + ((j ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(p) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
    if constexpr (SPLIT)
      *reinterpret_cast<uint4*>(p + kNsALow) = make_uint4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
  }
  fence_proxy_async_smem();
}

// Joins the eight epilogue warps, bounded like every wait; false: some warp gave up.
__device__ __forceinline__ bool ns_join(uint64_t* bar, uint32_t& phase, volatile int* abort, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  const bool ok = mbar_wait_bounded(bar, phase, abort, kWaitLimitNs);
  phase ^= 1;
  return __all_sync(0xffffffffu, ok);
}

// ROWS: the last product leaves by plain stores (rows that TMA cannot address,
// or both outputs at once).  SPLIT: operands in two fp16 parts.
// FUSED: a short side of at most 128 makes A and B a single tile: B is computed
// from the A in shared memory, without a trip to global memory between them.
// BN: columns of a tile (and of an accumulator); 256 on a CTA pair.  64: four of
// the epilogue warps store a tile (eight with half the columns each, and so
// twice the releases, measured 4 to 8 us slower over five steps).
template <int BN, bool ROWS, bool SPLIT, bool FUSED>
__global__ void __launch_bounds__(kNsThreads, 1) ns_kernel(const __grid_constant__ NsArgs P) {
  constexpr bool PAIR = BN == 256;
  constexpr int CG = PAIR ? 2 : 1;
  constexpr int TM = PAIR ? 256 : 128;    // rows of a tile, both CTAs
  constexpr int COLS = BN == 64 ? 64 : BN / 2;                    // columns of an epilogue warp
  constexpr int kStage = kNsOpBytes + (BN == 64 ? kNsBoxBytes : kNsOpBytes);      // bytes that a CTA loads
  static_assert((BN == 64 || BN == 128 || BN == 256) && (!FUSED || BN == 128), "tiles");
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = sm + kNsStages * kNsStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + 8 * kNsWarpOut);
  uint64_t* empty = full + kNsStages;
  uint64_t* tfull = empty + kNsStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drained = tempty + 2;
  uint64_t* a_ready = drained + 1;
  uint64_t* join = a_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(join + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_set = abort_flag + 1;
  volatile int* finishes = abort_flag + 2;          // FUSED: this CTA has the whole A
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
    mbar_init(a_ready, 8);
    mbar_init(join, 8);
    *abort_flag = 0;
    *never_set = 0;
    *finishes = 1;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&P.x[0]);
    tma_prefetch_desc(&P.a);
    tma_prefetch_desc(&P.b);
    tma_prefetch_desc(&P.as);
    tma_prefetch_desc(&P.bs);
    tma_prefetch_desc(&P.xs[1]);
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
  const int64_t total = static_cast<int64_t>(P.steps) * P.batch *
                        ((FUSED ? 1 : 1 + P.splits) * P.sym_tiles + P.app_m * P.app_n);
  // in parts: first (high, low), (low, high), then (high, high)
  constexpr int parts = SPLIT ? 3 : 1;
  const bool b_parts = FUSED && !SPLIT && P.b_low;      // X' = (B's low part) X + (its high part) X
  auto fail = [&]() {
    report(P.status, MXG_ERR_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == 0 || warp == 2) {
    // warp 0 loads P, warp 2 Q: one thread takes ~150 cycles per box, and the
    // boxes of a small product are its critical path
    if (lane == 0) {
      const bool second = warp == 2;
      uint32_t stage = 0, phase = 0;
      bool aborted = false;
      const uint32_t full0 = PAIR ? map_to_rank(smem_u32(full), 0) : 0u;
      for (int64_t t = tile0; t < total && !aborted; t += tstep) {
        const NsTile tc = ns_tile<TM, BN, FUSED>(P, t);
        const NsOperands o = ns_operands(P, tc);
        const int row = (second ? tc.tj * BN : tc.ti * TM) + static_cast<int>(rank) * kNsRows;
        const int mn_stages = ns_mn_stages(second ? o.q_form : o.p_form, row);
        const CUtensorMap* map = second ? o.q : o.p;
        const bool halved = SPLIT && tc.op == NS_APPLY;      // B: at most 64 rows
        const bool shared = FUSED && tc.op == NS_GRAM;
        const bool part_of = shared || (!FUSED && tc.op == NS_GRAM && P.splits > 1);
        const int first = part_of ? ns_share_begin<FUSED>(P, o, tc.share) : 0;
        const int stages = part_of ? ns_share_begin<FUSED>(P, o, tc.share + 1) : parts * (b_parts && tc.op == NS_APPLY ? 2 : 1) * o.nk;
        if (!ns_wait_done(P, tc, abort_flag)) {
          fail();
          aborted = true;
          break;
        }
        fence_proxy_async_global();       // the counts were acquired; the loads are the async proxy's
        for (int kp = first, kb = shared ? 0 : first, part = 0; kp < stages; ++kp) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          uint8_t* dst = sm + stage * kNsStageBytes + (second ? kNsOpBytes : 0);
          if (!second && (!PAIR || rank == 0))
            mbar_arrive_expect_tx(&full[stage], CG * (halved ? kStage - kNsBoxBytes : kStage));   // all bytes of both CTAs
          if (shared) {
            // rows 0 .. 127, or the high and low parts of rows 0 .. 63, of the stage's first or second 64 elements
            const int k0 = (2 * kp + second) * kNsK;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = SPLIT ? 0 : 64 * h;
              tma_load_3d(dst + h * kNsBoxBytes, map, mn_stages ? r : k0, mn_stages ? k0 : r, tc.b + (SPLIT && h ? P.batch : 0),
                          &full[stage]);
            }
          } else {
            const bool low = SPLIT ? part == (second ? 0 : 1) : b_parts && part == 0 && second == (P.tall != 0);
            const int z = tc.b + (low ? P.batch : 0);
            if ((BN == 64 && second) || (halved && second == (P.tall != 0))) ns_load<false, 1>(dst, map, kb < mn_stages, row, kb * kNsK, z, &full[stage], 0u);
            else if (!PAIR || rank == 0) ns_load<false, 2>(dst, map, kb < mn_stages, row, kb * kNsK, z, &full[stage], 0u);
            else ns_load<true, 2>(dst, map, kb < mn_stages, row, kb * kNsK, z, nullptr, full0 + stage * 8);
          }
          if (++stage == kNsStages) {
            stage = 0;
            phase ^= 1;
          }
          if (++kb == o.nk) {
            kb = 0;
            ++part;
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
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0, a_phase = 0;
      bool aborted = false;
      int64_t done = 0;
      const uint64_t desc0 = smem_desc(smem_u32(sm), kNsBoxBytes, 1024, kLayoutSwizzle128B);
      for (int64_t t = tile0; t < total && !aborted; t += tstep) {
        const NsTile tc = ns_tile<TM, BN, FUSED>(P, t);
        const bool got = PAIR ? mbar_wait_bounded_cluster(&tempty[acc], acc_phase ^ 1, abort_flag, kWaitLimitNs)
                              : mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, abort_flag, kWaitLimitNs);
        if (!got) {
          fail();
          break;
        }
        tc_fence_after();
        const uint32_t d_t = tmem + acc * BN;
        const NsOperands o = ns_operands(P, tc);
        // a tile's rows lie in one block of kNsSym, so the pair's CTAs agree on the form
        const int pmn = ns_mn_stages(o.p_form, tc.ti * TM), qmn = ns_mn_stages(o.q_form, tc.tj * BN);
        const bool shared = FUSED && tc.op == NS_GRAM;
        const bool part_of = shared || (!FUSED && tc.op == NS_GRAM && P.splits > 1);
        const int first = part_of ? ns_share_begin<FUSED>(P, o, tc.share) : 0;
        const int stages = part_of ? ns_share_begin<FUSED>(P, o, tc.share + 1) : parts * (b_parts && tc.op == NS_APPLY ? 2 : 1) * o.nk;
        for (int kp = first, kb = shared ? 0 : first; kp < stages; ++kp) {
          const bool in = PAIR ? mbar_wait_bounded_cluster(&full[stage], phase, abort_flag, kWaitLimitNs)
                               : mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs);
          if (!in) {
            fail();
            aborted = true;
            break;
          }
          tc_fence_after();
          // one thread issues everything: few instructions between the waits (the leading offset only matters
          // MN-major)
          const uint64_t pd = desc0 + stage * (kNsStageBytes >> 4);
          const uint64_t qd = shared ? pd : pd + (kNsOpBytes >> 4);
          const uint32_t pstep = kb < pmn ? 2048 >> 4 : 32 >> 4, qstep = kb < qmn ? 2048 >> 4 : 32 >> 4;
          const uint32_t id = idesc_f16(TM, SPLIT && tc.op == NS_APPLY && P.tall ? 64 : BN) | (kb < pmn ? kIdescAMn : 0u) | (kb < qmn ? kIdescBMn : 0u);
#pragma unroll
          for (uint32_t k = 0; k < kNsK / 16; ++k)
            mma_bf16<CG>(d_t, pd + k * pstep, qd + k * qstep, id, kp != first || k != 0 ? 1u : 0u);
          if (shared) {                   // the stage's second 64 contraction elements
            const uint64_t sd = pd + (kNsOpBytes >> 4);
#pragma unroll
            for (uint32_t k = 0; k < kNsK / 16; ++k) mma_bf16<CG>(d_t, sd + k * pstep, sd + k * pstep, id, 1u);
          }
          mma_commit<CG>(&empty[stage]);
          if (++kb == o.nk) kb = 0;
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
        if (FUSED && tc.op == NS_GRAM) {
          // A A^T from the A that the epilogue has put into shared memory, into the other accumulator
          if (!mbar_wait_bounded(a_ready, a_phase, abort_flag, kWaitLimitNs)) {
            fail();
            break;
          }
          a_phase ^= 1;
          if (*finishes == 0) continue;   // another CTA finishes this A
          if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1, abort_flag, kWaitLimitNs)) {
            fail();
            break;
          }
          tc_fence_after();
          const uint64_t ad = smem_desc(smem_u32(boxes), 0, 1024, kLayoutSwizzle128B);
          const uint32_t d2 = tmem + acc * BN;
          if constexpr (SPLIT) {          // 64 x 64: (high, low), (low, high), (high, high)
            for (int part = 0; part < 3; ++part) {
              const uint64_t pa = ad + (part == 1 ? kNsALow >> 4 : 0), qa = ad + (part == 0 ? kNsALow >> 4 : 0);
#pragma unroll
              for (uint32_t k = 0; k < 4; ++k)
                mma_bf16<CG>(d2, pa + 2 * k, qa + 2 * k, idesc_f16(TM, 64), (part | k) != 0 ? 1u : 0u);
            }
          } else {
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
              const uint32_t off = ((k >> 2) * kNsOpBytes + (k & 3) * 32) >> 4;
              mma_bf16<CG>(d2, ad + off, ad + off, idesc_f16(TM, BN), k != 0 ? 1u : 0u);
            }
          }
          mma_commit<CG>(&tfull[acc]);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
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
    constexpr int BOXES = COLS / 64;
    const int q = warp & 3;
    const int hf = (warp - 4) >> 2;
    uint8_t* box = boxes + (warp - 4) * kNsWarpOut;
    uint32_t acc = 0, acc_phase = 0, flip = 0, join_phase = 0;
    auto free_accumulator = [&]() {       // it has been read and may be overwritten
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR && rank == 1)
          st_async_complete_tx(map_to_rank(smem_u32(&landing[warp - 4]), 0), 1u, map_to_rank(smem_u32(&tempty[acc]), 0));
        else
          mbar_arrive(&tempty[acc]);
      }
    };
    for (int64_t t = tile0; t < total; t += tstep) {
      const NsTile tc = ns_tile<TM, BN, FUSED>(P, t);
      const bool last = tc.op == NS_APPLY && tc.step + 1 == P.steps;
      const int row0 = tc.ti * TM + static_cast<int>(rank) * kNsRows + q * 32;
      const int col0 = tc.tj * BN + (SPLIT && P.tall && tc.op == NS_APPLY ? 0 : hf * COLS);
      const int dm = tc.op == NS_APPLY ? P.rows : P.m, dn = tc.op == NS_APPLY ? P.cols : P.m;   // of D
      // A is read by plain loads here, so this warp, too, waits for it
      bool got = true;
      if (tc.op == NS_POLY && (BN != 64 || hf == 0)) {
        if (lane == 0) got = ns_wait_done(P, tc, abort_flag);
        got = __all_sync(0xffffffffu, got);
      }
      uint32_t w[32], wl[SPLIT ? 32 : 1];
      bool mine = true;                   // this CTA finishes the tile
      if (FUSED && tc.op == NS_GRAM) {
        got = __all_sync(0xffffffffu, mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs));
        tc_fence_after();
        if (got) {
          float v[64];
          ns_read64(P.alpha[NS_GRAM], tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + hf * COLS, v);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
          const int row = q * 32 + lane, ca = SPLIT ? 0 : hf * COLS;
          const bool holds = !SPLIT || (q < 2 && hf == 0);      // this warp's values are A's
          if constexpr (SPLIT) {
            // (high, low) and (low, high) to the warps that hold (high, high); 16-byte piece j of row r at
            // j ^ (r % 16), free of bank conflicts
            float4* swap = reinterpret_cast<float4*>(boxes + kNsSwap) + (q < 2 ? 0 : 64 * 16) + (row & 63) * 16;
            const int sw = row & 15;
            if ((q < 2) == (hf == 1))
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (4 * j < P.m) swap[j ^ sw] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            got = ns_join(join, join_phase, abort_flag, lane);
            if (got && holds)
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (4 * j < P.m) {
                  const float4 x = swap[j ^ sw], y = swap[64 * 16 + (j ^ sw)];
                  v[4 * j] += x.x + y.x;
                  v[4 * j + 1] += x.y + y.y;
                  v[4 * j + 2] += x.z + y.z;
                  v[4 * j + 3] += x.w + y.w;
                }
          }
          if (P.sym_tiles > 1 && got) {
            // A share of the sum; the CTA that leaves the last one adds them up in order.  128 x 128: column by
            // column, 32 rows side by side; SPLIT: row by row, only the few columns inside the matrix (measured,
            // five steps: 2 x 8000 x 100 by columns 125 us, by rows 139; 15 x 1894 x 15 126 and 106).
            constexpr int SIDE = SPLIT ? 64 : 128;
            float* base = P.a_parts + static_cast<int64_t>(tc.b) * P.sym_tiles * SIDE * SIDE +
                          (SPLIT ? row * SIDE : ca * SIDE + row);
            const int live = holds && row < P.m ? P.m : 0;             // SPLIT: columns
            float* dst = base + tc.share * SIDE * SIDE;
            if constexpr (SPLIT) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (8 * j < live) st_global_v8(dst + 8 * j, reinterpret_cast<const uint32_t*>(v) + 8 * j);
            } else {
#pragma unroll
              for (int i = 0; i < 64; ++i) dst[i * SIDE] = v[i];
            }
            __threadfence();
            got = ns_join(join, join_phase, abort_flag, lane);
            if (got && warp == 4 && lane == 0)
              *finishes = (atomicAdd(P.shares + tc.b * kNsLine, 1) + 1) % P.sym_tiles == 0;
            got = got && ns_join(join, join_phase, abort_flag, lane);
            mine = got && *finishes != 0;
            if (mine && holds) {
              __threadfence();
#pragma unroll
              for (int i = 0; i < 64; ++i) v[i] = 0.f;
#pragma unroll
              for (int c0 = 0; c0 < 64; c0 += 32) {    // 32 columns of two shares requested together
                if (SPLIT && c0 >= live) continue;
                for (int k = 0; k < P.sym_tiles; k += 2) {
                  const float* src = base + k * SIDE * SIDE + c0 * (SPLIT ? 1 : SIDE);
                  const float* nxt = k + 1 < P.sym_tiles ? src + SIDE * SIDE : src;
                  uint32_t x[32], y[32];
                  if constexpr (SPLIT) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                      const int c = c0 + j < live ? j : 0;             // columns past the matrix repeat the first ones
                      ld_global_cg_v8(src + c, x + j);
                      ld_global_cg_v8(nxt + c, y + j);
                    }
                  } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                      x[i] = __float_as_uint(__ldcg(src + i * SIDE));
                      y[i] = __float_as_uint(__ldcg(nxt + i * SIDE));
                    }
                  }
#pragma unroll
                  for (int i = 0; i < 32; ++i) {
                    v[c0 + i] += __uint_as_float(x[i]);
                    if (k + 1 < P.sym_tiles) v[c0 + i] += __uint_as_float(y[i]);
                  }
                }
              }
            }
          }
          if (mine && got && holds) ns_keep_a<SPLIT>(P, v, boxes, row, ca, w, wl);
          __syncwarp();
          if (lane == 0) mbar_arrive(a_ready);
        }
      }
      const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN + hf * (BN / 2);
      if (!FUSED && tc.op == NS_GRAM && P.splits > 1) {
        // A share of the sum of a tile: half the columns of this lane's row, in pieces of 16 bytes with the lanes
        // side by side.  The CTA that leaves the last share of its 128 rows adds them up in order and stores them.
        constexpr int kChunks = BN / 64;                               // of 32 columns
        constexpr int kPiece = 128 * 4, kShare = 128 * BN;             // floats
        got = __all_sync(0xffffffffu, mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs));
        tc_fence_after();
        if (got) {
          const int64_t sum = static_cast<int64_t>(tc.tile) * CG + rank;
          float* base = P.a_parts + sum * P.splits * kShare + hf * (BN / 8) * kPiece + (q * 32 + lane) * 4;
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tb + 32 * c, r);
            tmem_ld_wait();
            float* dst = base + tc.share * kShare + c * 8 * kPiece;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(dst + j * kPiece) = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
          }
          free_accumulator();
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
          __threadfence();
          got = ns_join(join, join_phase, abort_flag, lane);
          if (got && warp == 4 && lane == 0)
            *finishes = (atomicAdd(P.shares + sum * kNsLine, 1) + 1) % P.splits == 0;
          got = got && ns_join(join, join_phase, abort_flag, lane);
          if (got && *finishes != 0) {
            __threadfence();
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              float v[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.f;
              const float* src = base + c * 8 * kPiece;
              for (int k = 0; k < P.splits; k += 2) {                  // two shares requested together
                float4 x[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    x[u][j] = __ldcg(reinterpret_cast<const float4*>(src + min(k + u, P.splits - 1) * kShare + j * kPiece));
#pragma unroll
                for (int u = 0; u < 2; ++u)
                  if (k + u < P.splits)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                      v[4 * j] += x[u][j].x;
                      v[4 * j + 1] += x[u][j].y;
                      v[4 * j + 2] += x[u][j].z;
                      v[4 * j + 3] += x[u][j].w;
                    }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const __half2 h = __floats2half2_rn(P.alpha[NS_GRAM] * v[2 * i], P.alpha[NS_GRAM] * v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
              const int col = tc.tj * BN + hf * (BN / 2) + 32 * c;
              ns_store_direct<1>(w, P.ap + (static_cast<int64_t>(tc.b) * P.m + row0 + lane) * P.lda + col,
                                 row0 + lane < P.m, col, P.m);
            }
            __syncwarp();
            if (lane == 0) red_release_gpu_add(P.done + tc.b * kNsLine, 1);
          }
        }
        if (!got) {
          if (lane == 0) fail();
          break;
        }
        continue;
      }
      // SPLIT: half of the tile of X' lies outside the matrix.  Rows past 63 leave two of four quadrants idle; in a tall
      // matrix the columns past 63 do, and the two groups of four warps take turns at the tiles instead.
      const bool halved = SPLIT && tc.op == NS_APPLY;
      const bool turns = halved && P.tall;
      if ((BN == 64 && hf == 1) || (halved && (P.tall ? acc != static_cast<uint32_t>(hf) : q >= 2))) {
        // other warps store this tile
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs))) {
          if (lane == 0) fail();
          break;
        }
        if (lane == 0) mbar_arrive(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
        continue;
      }
      const uint32_t tq = turns ? tb - hf * COLS : tb;
#pragma unroll 1
      for (int c = 0; c < BOXES && got && mine; ++c) {
        const int col = col0 + 64 * c;
        const bool any = row0 < dm && col < dn;
        auto ready = [&]() {              // before the first columns: the accumulator is complete
          if (c != 0) return true;
          const bool in = __all_sync(0xffffffffu, mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, kWaitLimitNs));
          tc_fence_after();
          return in;
        };
        auto release = [&]() {            // after the last columns
          if (c == BOXES - 1) free_accumulator();
        };
        const uint32_t ta = tq + 64 * c;
        const NsDst da{&P.as, P.ap, P.m, P.m, P.lda, P.low_a}, db{&P.bs, P.bp, P.m, P.m, P.lda, P.low_a},
            dx{&P.xs[(tc.step & 1) ^ 1], P.xp[(tc.step & 1) ^ 1], P.rows, P.cols, P.ldx, P.low_x},
            out{&P.out, P.w_out != nullptr ? P.w_out : P.update, P.rows, P.cols, P.cols, 0};
        if (!FUSED && tc.op == NS_GRAM)
          got = ns_epilogue<NS_STORE, SPLIT, !PAIR, false>(P, P.alpha[NS_GRAM], ta, box, flip, da, row0, col, tc.b, any,
                                                           lane, w, wl, ready, release);
        else if (FUSED ? tc.op == NS_GRAM : tc.op == NS_POLY)
          got = ns_epilogue<NS_POLYNOMIAL, SPLIT, !PAIR, FUSED>(P, P.alpha[NS_POLY], ta, box, flip, db, row0, col, tc.b,
                                                                any, lane, w, wl, ready, release);
        else if (!last)
          got = ns_epilogue<NS_STORE, SPLIT, !PAIR, false>(P, P.alpha[NS_APPLY], ta, box, flip, dx, row0, col, tc.b,
                                                           any, lane, w, wl, ready, release);
        else if (ROWS)
          got = ns_epilogue<NS_BY_ROWS, SPLIT, !PAIR, false>(P, P.alpha_last, ta, box, flip, out, row0, col, tc.b, any,
                                                             lane, w, wl, ready, release);
        else if (P.w_out != nullptr)
          got = ns_epilogue<NS_WEIGHTS, SPLIT, !PAIR, false>(P, P.alpha_last, ta, box, flip, out, row0, col, tc.b, any,
                                                             lane, w, wl, ready, release);
        else
          got = ns_epilogue<NS_UPDATE, SPLIT, !PAIR, false>(P, P.alpha_last, ta, box, flip, out, row0, col, tc.b, any,
                                                            lane, w, wl, ready, release);
      }
      if (!got) {
        if (lane == 0) fail();
        break;
      }
      if (!mine) continue;                // another CTA finishes this A
      if (!last) {
        __syncwarp();                     // plain stores: the warp's, before the release below
        if (lane == 0) {
          if (PAIR) {                     // TMA stores: in memory,
            bulk_wait_group<0>();
            fence_proxy_async_global();
          }
          red_release_gpu_add(P.done + tc.b * kNsLine, BN == 64 || halved ? 2 : 1);
        }
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (lane == 0) bulk_wait_group<0>();  // the stores have completed before the CTA exits
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<CG>(tmem, 2 * BN);
}

// --------------------------------------------------------------------- host
// CTAs (or pairs) of a kernel that the device holds at once.
template <int BN, bool ROWS, bool SPLIT, bool FUSED>
int ns_resident() {
  constexpr bool PAIR = BN == 256;
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && known[dev].load() > 0) return known[dev].load();
  auto kern = ns_kernel<BN, ROWS, SPLIT, FUSED>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsSmem) != cudaSuccess) return 0;
  int n = 0;
  if (PAIR) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kNsThreads);
    cfg.dynamicSmemBytes = kNsSmem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
  } else {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kNsThreads, kNsSmem) != cudaSuccess) return 0;
    n *= device_sms();
  }
  if (dev < 64) known[dev].store(n);
  return n;
}

template <int BN, bool ROWS, bool SPLIT, bool FUSED>
cudaError_t launch_ns(NsArgs& a, cudaStream_t s) {
  constexpr bool PAIR = BN == 256;
  constexpr int TM = PAIR ? 256 : 128;
  a.app_m = (a.rows + TM - 1) / TM;
  a.app_n = (a.cols + BN - 1) / BN;
  // the largest product's tiles: X's, unless A's contraction is shared out
  const int64_t most = static_cast<int64_t>(a.batch) * std::max(a.app_m * a.app_n, a.sym_tiles * a.splits);
  const int64_t units = ns_resident<BN, ROWS, SPLIT, FUSED>();
  if (units <= 0) return cudaErrorCooperativeLaunchTooLarge;
  const int64_t n = most < units ? most : units;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? 2 * n : n));
  cfg.blockDim = dim3(kNsThreads);
  cfg.dynamicSmemBytes = kNsSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, ns_kernel<BN, ROWS, SPLIT, FUSED>, a);
  count_launch();
  return err != cudaSuccess ? err : cudaGetLastError();
}

struct NsPlan {
  int m, n, tall;                         // short and long side; tall: the matrix is [n][m]
  int split;
  int cluster;                            // CTAs per matrix that stays on the chip, 0: tiled
  int bn;                                 // columns of a tile
  int sym_tiles;                          // tiles of A; of a single-tile A the CTAs that share its contraction
  int splits;                             // CTAs that share the contraction of a tile of A
  int n_done;                             // counters
  int64_t ldx, lda;                       // row lengths of X and of A and B, padded to 16
  int chunks;                             // partial sums of squares per matrix
  int64_t part, done, x0, x1, a, b, a_parts, bytes;
};

// A short side up to this is computed in two fp16 parts (high and low, three
// products instead of one).  Simulated in 64 bits, gradients of a few strong
// directions over noise, the error of the bf16 update against an exact run
// (its own rounding alone is 1.66e-3): one part 3.1e-3 at 8 x 8, 2.4e-3 at
// 16 x 2000, 2.2e-3 from 64 x 64 to 256 x 256; two parts 1.67e-3.
constexpr int kNsSplitMost = 64;          // not above 128: only single tiles of A split

// The longest contraction of X X^T that one accumulator takes.  The tensor cores
// cut their running sums, by about 1.5e-8 of the result per instruction (16
// elements), and the diagonal of X X^T is a sum of squares: all of it is cut the
// same way, and the quintic's steps magnify the bias of A by up to 30 in X.
// Measured in one accumulator, 4 x n, the result's gain 1 + g: g = 1.8e-3 at n =
// 65536, 2.4e-3 at 131072, 1.0e-2 at 524288, 3.7e-2 at 2097152; longer sides are
// therefore added up in fp32 from shares, whether SMs are idle or not.  Where A is
// one tile a share costs little: 4 x n then has g at most 5e-4 at any n (152 x 4 x
// 131072 15.0 -> 15.3 ms, 152 x 4 x 2097152 233 -> 285).  With more tiles there are
// more, smaller singular values, whose first steps hardly see A (130 x 131072 in
// one accumulator 1.1e-3, in two 4e-4 at the same time).
constexpr int kNsLongestOne = 16384;      // A one tile
constexpr int kNsLongest = 65536;

// CTAs that share the contraction n of a single-tile A while SMs are idle: a
// stage of 128 elements takes about 550 cycles; leaving and joining the sums
// about 3500 and, per CTA, what it takes to read 64 x 64 (split) or 128 x 128
// fp32 values.
int ns_shares(int batch, int m, int n, int split) {
  if (m > 128) return 1;
  const int stages = (n + 2 * kNsK - 1) / (2 * kNsK);
  const int least = (n + kNsLongestOne - 1) / kNsLongestOne;
  const int most = std::max(least, std::min(std::min(device_sms() / batch, stages), 16));
  int best = 1, best_cost = least > 1 ? INT_MAX : stages * 550;
  for (int s = std::max(least, 2); s <= most; ++s) {
    const int cost = (stages + s - 1) / s * 550 + 3500 + s * (split ? 400 : 1300);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

// Tiles of a symmetric m x m matrix that are computed.
template <int TM, int BN>
int ns_sym_tiles(int m) {
  const int tm = (m + TM - 1) / TM, tn = (m + BN - 1) / BN;
  int n = 0;
  for (int i = 0; i < tm; ++i) n += tn - ns_first<TM, BN>(i);
  return n;
}

// Cycles of a step with tiles of TM x BN, fitted to timings of some forty shapes
// with each kind of tile: a product takes 3000 until its first stage is there
// (the count of the one before, the first loads), then per tile of the busiest
// SM its stages (550 cycles, a pair's 600) and its epilogue (up to the release
// of the next product).  SMs without a tile of A can share its contraction
// instead: each of `splits` CTAs leaves its sums, and the last one reads them
// all.  Five steps with 64 / 128 / 256 columns, microseconds, the rule's choice
// within 7 % of the best one everywhere:
//   8 x 256 x 256    68  77  93      1 x 8192 x 700   276 235 273
//   1 x 1300 x 1300 196 173 189      60 x 200 x 200   136 104 113
//   100 x 256 x 256 203 140 127      1 x 8192 x 2000 1242 716 544
// and not shared / shared: 1 x 200 x 3000 (64) 128 / 95, 1 x 6000 x 140 (64)
// 193 / 102, 1 x 3000 x 1000 (128) 251 / 217, 2 x 1000 x 8000 (256) 430 / 368.
template <int TM, int BN>
double ns_step_cost(int batch, int rows, int cols, int* splits) {
  constexpr bool PAIR = BN == 256;
  const double units = PAIR ? device_sms() / 2 : device_sms();
  const double stage = PAIR ? 600 : 550, epilogue = PAIR ? 7000 : BN == 128 ? 3200 : 2000;
  const int m = std::min(rows, cols), n = std::max(rows, cols);
  const int long_k = (n + kNsK - 1) / kNsK, short_k = (m + kNsK - 1) / kNsK;
  const double a = static_cast<double>(batch) * ns_sym_tiles<TM, BN>(m);
  const double x = static_cast<double>(batch) * ((rows + TM - 1) / TM) * ((cols + BN - 1) / BN);
  auto product = [&](double tiles, int stages) { return 3000 + std::max(1.0, tiles / units) * (stages * stage + epilogue); };
  const double others = product(a, short_k) + product(x, short_k);
  const int least = (n + kNsLongest - 1) / kNsLongest;
  double gram = least > 1 ? HUGE_VAL : product(a, long_k);
  *splits = 1;
  const int most = std::max(least, static_cast<int>(std::min({units / a, static_cast<double>(long_k), 16.0})));
  for (int s = std::max(least, 2); s <= most; ++s) {
    const double c = product(a * s, (long_k + s - 1) / s) + (PAIR ? 6000 + 2000 * s : BN == 128 ? 4500 + 1300 * s : 3700 + 750 * s);
    if (c < gram) {
      gram = c;
      *splits = s;
    }
  }
  return gram + others;
}

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
  p.split = p.m <= kNsSplitMost;
  p.cluster = resident_cluster(batch, p.m, p.n, p.split);
  if (p.cluster != 0) {                   // nothing of it leaves the chip
    p.bytes = api::kAlign;
    return p;
  }
  p.part = w.take(8ll * batch * p.chunks);
  p.splits = 1;
  if (p.m <= 128) {
    p.bn = 128;
    p.sym_tiles = ns_shares(batch, p.m, p.n, p.split);
  } else {
    // 64, 128 (one SM) or 256 columns (a pair; half the operand bytes per product of the others)
    int splits[3];
    const double c64 = ns_step_cost<128, 64>(batch, rows, cols, &splits[0]);
    const double c128 = ns_step_cost<128, 128>(batch, rows, cols, &splits[1]);
    const double c256 = ns_step_cost<256, 256>(batch, rows, cols, &splits[2]);
    const int best = c64 <= c128 && c64 <= c256 ? 0 : c128 <= c256 ? 1 : 2;
    p.bn = 64 << best;
    p.splits = splits[best];
    p.sym_tiles = best == 0   ? ns_sym_tiles<128, 64>(p.m)
                  : best == 1 ? ns_sym_tiles<128, 128>(p.m)
                              : ns_sym_tiles<256, 256>(p.m);
  }
  const int ctas = p.bn == 256 ? 2 : 1;   // of a tile
  p.n_done = batch * (p.splits > 1 ? 1 + ctas * p.sym_tiles : 2) * kNsLine;
  p.done = w.take(4ll * p.n_done);        // and the shares' counters
  const int64_t one = p.split ? 4 : 2;    // bytes of an element
  const int64_t xb = one * batch * rows * p.ldx, ab = one * batch * p.m * p.lda;
  p.x0 = w.take(xb);
  p.x1 = w.take(xb);
  p.a = w.take(ab);
  p.b = w.take(p.m <= 128 && !p.split && muon_b_low(p.m, p.n) ? 2 * ab : ab);
  // the shares of the sums of A
  p.a_parts = w.take(p.splits > 1 ? 4ll * 128 * p.bn * ctas * batch * p.sym_tiles * p.splits
                     : p.m <= 128 && p.sym_tiles > 1 ? (p.split ? 4ll * 64 * 64 : 4ll * 128 * 128) * batch * p.sym_tiles
                                                     : 0);
  p.bytes = w.off;
  return p;
}

int muon_shape(int batch, int rows, int cols) {
  if (batch <= 0 || rows <= 0 || cols <= 0) return MXG_ERR_ARG;
  const int64_t longest = rows > cols ? rows : cols;
  // grid and tensor-map coordinates are 32-bit, and so are the counts of finished parts of a matrix (sixteen
  // warps on each of at most three tiles per 128 x 128 elements, 64 steps)
  const int64_t tiles = static_cast<int64_t>((rows + 127) / 128) * ((cols + 127) / 128);
  if (batch > 65535 || longest > (1 << 21) || batch * longest > INT32_MAX - 256 || tiles > INT32_MAX / (16 * 3 * 64))
    return MXG_ERR_SHAPE;
  return MXG_OK;
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" size_t mxg_muon_workspace_bytes(int batch, int rows, int cols) {
  if (muon_shape(batch, rows, cols) != MXG_OK) return 0;
  return static_cast<size_t>(ns_plan(batch, rows, cols).bytes);
}

extern "C" int mxg_muon_form(int batch, int rows, int cols, int32_t* form) {
  if (!form) return MXG_ERR_ARG;
  if (const int err = muon_shape(batch, rows, cols)) return err;
  const NsPlan p = ns_plan(batch, rows, cols);
  form[0] = p.cluster;
  form[1] = p.bn;
  form[2] = p.cluster != 0 ? 0 : p.m <= 128 ? p.sym_tiles : p.splits;
  form[3] = p.split ? 2 : 1;
  return MXG_OK;
}

extern "C" int mxg_muon_update(const mxg_muon_args* a, void* stream) {
  if (!a || !a->grad || !a->workspace || !a->dev_status) return MXG_ERR_ARG;
  if (a->momentum_in && !a->momentum_out) return MXG_ERR_ARG;
  if ((a->w_in != nullptr) != (a->w_out != nullptr)) return MXG_ERR_ARG;
  if (!a->update && !a->w_out) return MXG_ERR_ARG;
  if (a->steps < 1 || a->steps > 64) return MXG_ERR_ARG;
  if (!(std::fabs(a->a) < kMostA)) return MXG_ERR_ARG;
  if (const int err = muon_shape(a->batch, a->rows, a->cols)) return err;
  if (!api::aligned32(a->grad) || !api::aligned32(a->momentum_in) || !api::aligned32(a->momentum_out) ||
      !api::aligned32(a->update) || !api::aligned32(a->w_in) || !api::aligned32(a->w_out) ||
      !api::aligned32(a->workspace))
    return MXG_ERR_ALIGN;
  const NsPlan p = ns_plan(a->batch, a->rows, a->cols);
  if (a->workspace_bytes < static_cast<uint64_t>(p.bytes)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.muon_update");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int ex = 0;                             // 2^ex ~ sqrt(n)
  while ((1ll << (2 * ex)) < p.n) ++ex;
  // A 2^12 = (X 2^ex)(X 2^ex)^T 2^(12 - 2 ex);  B 2^12 = a 2^12 I + b (A 2^12) + c 2^-12 (A 2^12)(A 2^12);
  // X' 2^ex = 2^-12 (B 2^12)(X 2^ex), the last one scale X'
  const float alpha[3] = {static_cast<float>(std::ldexp(1.0, kExpA - 2 * ex)),
                          static_cast<float>(std::ldexp(static_cast<double>(a->c), -kExpA)),
                          static_cast<float>(std::ldexp(1.0, -kExpA))};
  const float alpha_last = static_cast<float>(std::ldexp(static_cast<double>(a->scale), -kExpA - ex));
  const float diag = static_cast<float>(std::ldexp(static_cast<double>(a->a), kExpA));
  const float w_keep = static_cast<float>(1.0 - static_cast<double>(a->lr) * a->weight_decay);
  const int64_t per = static_cast<int64_t>(a->rows) * a->cols;
  const MomentumArgs mo{a->grad, a->grad_f32, a->momentum_in, a->momentum_out, a->mu, a->nesterov, per};
  if (p.cluster != 0) {
    ResidentArgs r{};
    r.mo = mo;
    r.batch = a->batch;
    r.rows = a->rows;
    r.cols = a->cols;
    r.steps = a->steps;
    r.ex = ex;
    for (int i = 0; i < 3; ++i) r.alpha[i] = alpha[i];
    r.alpha_last = alpha_last;
    r.beta = a->b;
    r.diag = diag;
    r.update = a->update;
    r.w_in = a->w_in;
    r.w_out = a->w_out;
    r.w_keep = w_keep;
    r.lr = a->lr;
    r.status = a->dev_status;
    return api::cuda_status(launch_muon_resident(r, p.cluster, p.split, s));
  }
  double* part = api::at<double>(a->workspace, p.part);
  int32_t* done = api::at<int32_t>(a->workspace, p.done);
  __half* x[2] = {api::at<__half>(a->workspace, p.x0), api::at<__half>(a->workspace, p.x1)};
  __half* am = api::at<__half>(a->workspace, p.a);
  __half* bm = api::at<__half>(a->workspace, p.b);
  const unsigned nb = static_cast<unsigned>(a->batch);
  const dim3 mgrid(static_cast<unsigned>(p.chunks), nb);
  momentum_kernel<<<mgrid, kMoThreads, 0, s>>>(mo, p.chunks, part, done, p.n_done);
  count_launch();
  const int64_t lo_off = p.split ? static_cast<int64_t>(a->batch) * a->rows * p.ldx : 0;
  if (a->cols % kMoVec == 0)
    cast_kernel<true><<<mgrid, kMoThreads, 0, s>>>(mo, p.chunks, part, ex, a->rows, a->cols, x[0], p.ldx, lo_off);
  else cast_kernel<false><<<mgrid, kMoThreads, 0, s>>>(mo, p.chunks, part, ex, a->rows, a->cols, x[0], p.ldx, lo_off);
  count_launch();
  if (cudaGetLastError() != cudaSuccess) return MXG_ERR_CUDA;

  NsArgs n{};
  n.rows = a->rows;
  n.cols = a->cols;
  n.m = p.m;
  n.tall = p.tall;
  n.batch = a->batch;
  n.steps = a->steps;
  for (int i = 0; i < 3; ++i) n.alpha[i] = alpha[i];
  n.alpha_last = alpha_last;
  n.beta = a->b;
  n.diag = diag;
  n.xp[0] = reinterpret_cast<uint16_t*>(x[0]);
  n.xp[1] = reinterpret_cast<uint16_t*>(x[1]);
  n.ap = reinterpret_cast<uint16_t*>(am);
  n.bp = reinterpret_cast<uint16_t*>(bm);
  n.ldx = p.ldx;
  n.lda = p.lda;
  n.low_x = static_cast<int64_t>(a->batch) * a->rows * p.ldx;
  n.low_a = static_cast<int64_t>(a->batch) * p.m * p.lda;
  n.update = a->update;
  n.w_in = a->w_in;
  n.w_out = a->w_out;
  n.w_keep = w_keep;
  n.lr = a->lr;
  n.done = done;
  n.shares = done + a->batch * kNsLine;
  n.sym_tiles = p.sym_tiles;
  n.splits = p.splits;
  n.b_low = p.m <= 128 && !p.split && muon_b_low(p.m, p.n);
  n.a_parts = api::at<float>(a->workspace, p.a_parts);
  n.status = a->dev_status;
  const int64_t mats = static_cast<int64_t>(a->batch) * (p.split ? 2 : 1);
  const int64_t b_mats = n.b_low ? 2ll * a->batch : mats;
  bool ok = true;
  for (int i = 0; i < 2; ++i) {
    ok = ok && tma_map_b16_3d(&n.x[i], x[i], a->cols, a->rows, mats, p.ldx, 64);
    ok = ok && tma_map_b16_3d(&n.xs[i], x[i], a->cols, a->rows, mats, p.ldx, 32);
  }
  ok = ok && tma_map_b16_3d(&n.a, am, p.m, p.m, mats, p.lda, 64) && tma_map_b16_3d(&n.as, am, p.m, p.m, mats, p.lda, 32);
  ok = ok && tma_map_b16_3d(&n.b, bm, p.m, p.m, b_mats, p.lda, 64) && tma_map_b16_3d(&n.bs, bm, p.m, p.m, b_mats, p.lda, 32);
  // whole 32-byte pieces of the caller's rows, one output
  const bool by_rows = a->cols % 16 != 0 || (a->w_out && a->update);
  if (!by_rows)
    ok = ok && tma_map_b16_3d(&n.out, a->w_out ? a->w_out : a->update, a->cols, a->rows, a->batch, a->cols, 32);
  if (!ok) return MXG_ERR_CUDA;
  cudaError_t err;
  if (p.bn == 256)
    err = by_rows ? launch_ns<256, true, false, false>(n, s) : launch_ns<256, false, false, false>(n, s);
  else if (p.bn == 64)
    err = by_rows ? launch_ns<64, true, false, false>(n, s) : launch_ns<64, false, false, false>(n, s);
  else if (p.m > 128)
    err = by_rows ? launch_ns<128, true, false, false>(n, s) : launch_ns<128, false, false, false>(n, s);
  else if (p.split)
    err = by_rows ? launch_ns<128, true, true, true>(n, s) : launch_ns<128, false, true, true>(n, s);
  else
    err = by_rows ? launch_ns<128, true, false, true>(n, s) : launch_ns<128, false, false, true>(n, s);
  return api::cuda_status(err);
}
