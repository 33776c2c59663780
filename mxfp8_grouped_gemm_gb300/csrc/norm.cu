// Residual addition with the root-mean-square norm that makes the layer's
// input, in bf16 and (optionally) row-wise MXFP8, and its backward pass.
//
//   r = x + residual,  rstd = 1 / sqrt(mean(r^2) + eps),  y = r rstd w
// and, with xh = r rstd, g = dy w,
//   dr = rstd (g - xh mean(g xh)) + dresidual,   dw = sum over rows of dy xh.
//
// A row is read once and stays in registers between its sum and its output:
// thread t of the row's threads holds the 16-byte chunks t, t + threads, ...
// (8 values each, so four neighbouring lanes hold one MX block).  Rows of up to
// 1024 values are handled by 8 to 32 lanes of a warp, several rows a CTA; wider
// ones by a CTA of their own.  Both passes are bound by HBM.  Measured, bf16
// streams, launches included: forward 16384 x 4096 with codes 92 us (6.6 TB/s),
// 262144 x 128 46 us (6.6), 4096 x 16384 111 us (5.5: two CTAs of 512 threads an
// SM, whose loads and stores take turns; shared by a cluster of four 127); backward 16384 x 4096 83 us (6.5 TB/s),
// 65536 x 1024 86 (6.2), 8192 x 4096 in fp32 98 (5.5), 4096 x 16384 121 (4.4; by
// clusters of four CTAs, whose barrier a row waits for, 118).
#include <cmath>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kSms = 152;
constexpr int kMaxH = 16384;
constexpr int kRowThreads = 128;        // CTA of the rows that lanes of a warp share
constexpr int kMaxThreads = 512;        // CTA of one wide row

enum { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) { *reinterpret_cast<uint4*>(p) = pack8(v); }

template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sum over the row's threads: LPR lanes of a warp, or (LPR 0) the whole CTA.
// The CTA's form needs one barrier: successive rows use s_part in turn.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float (*s_part)[32], int parity) {
  if constexpr (LPR != 0) {
    return lanes_sum<LPR>(v);
  } else {
    v = lanes_sum<32>(v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) s_part[parity][warp] = v;
    __syncthreads();
    return lanes_sum<32>(lane < static_cast<int>(blockDim.x >> 5) ? s_part[parity][lane] : 0.f);
  }
}

struct NormFwdParams {
  int T, H;
  const uint16_t* x;
  const void* residual;
  void* residual_out;
  const void* weight;
  int w32;
  float eps, inv_h;
  uint16_t* y;
  uint8_t* q;
  uint8_t* s;
  int layout;
  float* rstd;
};

__device__ __forceinline__ void load_weight(const void* w, int w32, int col, float (&v)[8]) {
  if (w32) load8(static_cast<const float*>(w) + col, v);
  else load8(static_cast<const uint16_t*>(w) + col, v);
}

// Ten CTAs an SM where a lane holds 32 values (48 registers, and 32 to 108 bytes of
// spills; with 64 registers and eight CTAs, which spill nothing, 65536 x 1024 took
// 97.6 us instead of 94.3, 5003 x 1000 in fp32 14.4 instead of 13.3).
template <int LPR, int NCH, int RES>
__global__ void __launch_bounds__(LPR != 0 ? kRowThreads : kMaxThreads, LPR != 0 && NCH == 4 ? 10 : 0) norm_fwd_kernel(const NormFwdParams P) {
  __shared__ float s_part[2][32];
  const int threads = LPR != 0 ? LPR : static_cast<int>(blockDim.x);
  const int th = LPR != 0 ? static_cast<int>(threadIdx.x) % LPR : static_cast<int>(threadIdx.x);
  const int64_t row = LPR != 0 ? static_cast<int64_t>(blockIdx.x) * (kRowThreads / LPR) + threadIdx.x / LPR
                               : static_cast<int64_t>(blockIdx.x);
  const bool live = row < P.T;
  const int n8 = P.H >> 3;
  const int64_t base = row * P.H;
  float r[NCH][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = th + i * threads;
    const bool in = live && c < n8;
#pragma unroll
    for (int j = 0; j < 8; ++j) r[i][j] = 0.f;
    if (in) {
      load8(P.x + base + 8 * c, r[i]);
      if constexpr (RES != RES_NONE) {
        float a[8];
        if constexpr (RES == RES_F32) load8(static_cast<const float*>(P.residual) + base + 8 * c, a);
        else load8(static_cast<const uint16_t*>(P.residual) + base + 8 * c, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] += a[j];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(r[i][j], r[i][j], sum);
  sum = row_sum<LPR>(sum, s_part, 0);
  const float rstd = 1.f / sqrtf(fmaf(sum, P.inv_h, P.eps));
  if (live && th == 0 && P.rstd != nullptr) P.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = th + i * threads;
    const bool in = live && c < n8;
    if (in) {
      if constexpr (RES != RES_NONE) {
        if (P.residual_out != nullptr) {
          if constexpr (RES == RES_F32) store8(static_cast<float*>(P.residual_out) + base + 8 * c, r[i]);
          else store8(static_cast<uint16_t*>(P.residual_out) + base + 8 * c, r[i]);
        }
      }
      float w[8];
      load_weight(P.weight, P.w32, 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * rstd * w[j];
    }
    const uint4 y = pack8(r[i]);
    if (in && P.y != nullptr) *reinterpret_cast<uint4*>(P.y + base + 8 * c) = y;
    if (P.q != nullptr) {
      // the codes of the bf16 values, so that they are mxg_mxfp8_quantize's on y; pairs stay pairs between the
      // lanes, so that a NaN gives way to the block's numbers as it does there
      uint32_t pair = absmax_bf16x2(absmax_bf16x2(y.x, y.y), absmax_bf16x2(y.z, y.w));
      pair = absmax_bf16x2(pair, __shfl_xor_sync(0xffffffffu, pair, 1));
      pair = absmax_bf16x2(pair, __shfl_xor_sync(0xffffffffu, pair, 2));
      const uint32_t sb = mx_scale_byte(pair_bits(pair));
      const float inv = mx_inv_scale(sb);
      float v[8];
      unpack8(y, v);
      const uint32_t lo = cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      const uint32_t hi = cvt_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
      if (in) {
        *reinterpret_cast<uint2*>(P.q + base + 8 * c) = make_uint2(lo, hi);
        if ((c & 3) == 0) P.s[sf_offset(P.layout, row, c >> 2, P.T, P.H >> 5)] = static_cast<uint8_t>(sb);
      }
    }
  }
}

struct NormBwdParams {
  int T, H;
  const uint16_t* dy;
  const void* r;
  const void* weight;
  int w32;
  const float* rstd;
  float inv_h;
  const void* dresidual;
  uint16_t* dx;
  float* dresidual_out;
  float* part;            // [gridDim.x][H]; the result itself where the grid is one CTA
};

// L1: of values whose other half of a 32-byte sector is copied next.
template <bool L1>
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  if constexpr (L1) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows of a CTA (or of its lane groups) in shared memory: as many as fit with the
// CTAs an SM runs (bwd_ctas); one of 16384 fp32 values.
constexpr int row_slots(int lpr, int nch, bool f32) {
  const bool widest = lpr == 0 && nch == 4;
  return f32 ? (widest ? 1 : 2) : widest ? 2 : nch == 1 || nch == 3 ? 3 : 4;
}

// A CTA takes rows blockIdx, + grid, ... and keeps the sums of its columns of
// dweight in registers.  Every thread copies its own chunks of the next rows into
// shared memory and reads them back itself, so that
// kSlots rows are on their way without a register or a barrier for them: a slot
// is filled again as soon as its row is in registers (kHold) or, where a thread
// has too much of a row for that, once it has been read a second time.
template <int LPR, int NCH, bool F32>
__global__ void __launch_bounds__(LPR != 0 ? kRowThreads : kMaxThreads) norm_bwd_kernel(const NormBwdParams P) {
  constexpr int kGroups = LPR != 0 ? kRowThreads / LPR : 1;     // rows at a time
  constexpr int kSlots = row_slots(LPR, NCH, F32);
  constexpr bool kHold = LPR != 0 || NCH < 4;
  constexpr int kR = F32 ? 2 : 1;                               // 16-byte pieces of a chunk of r
  constexpr int kPieces = NCH * (1 + 2 * kR);                   // of a thread's part of a row: dy, r, dresidual
  extern __shared__ __align__(16) uint8_t s_rows[];             // [kSlots][kPieces][threads] x 16 bytes
  __shared__ float s_part[2][32];
  launch_dependents();
  const int threads = LPR != 0 ? LPR : static_cast<int>(blockDim.x);
  const int th = LPR != 0 ? static_cast<int>(threadIdx.x) % LPR : static_cast<int>(threadIdx.x);
  const int group = LPR != 0 ? static_cast<int>(threadIdx.x) / LPR : 0;
  const int n8 = P.H >> 3;
  const uint32_t piece = blockDim.x * 16, stage_bytes = kPieces * piece;
  const uint32_t slot0 = smem_u32(s_rows) + threadIdx.x * 16;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  const int rb = F32 ? 32 : 16;                                 // bytes of a chunk of r

  const auto request = [&](int64_t row, uint32_t slot) {
    if (row < P.T) {
      const int64_t base = row * n8;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = th + i * threads;
        if (c < n8) {
          copy16<false>(slot + i * piece, P.dy + (base + c) * 8);
          const uint8_t* r = static_cast<const uint8_t*>(P.r) + (base + c) * rb;
#pragma unroll
          for (int m = 0; m < kR; ++m) copy16<F32>(slot + (NCH + kR * i + m) * piece, r + 16 * m);
          if (P.dresidual != nullptr) {
            const uint8_t* d = static_cast<const uint8_t*>(P.dresidual) + (base + c) * rb;
#pragma unroll
            for (int m = 0; m < kR; ++m) copy16<F32>(slot + (NCH + kR * (NCH + i) + m) * piece, d + 16 * m);
          }
        }
      }
    }
    copies_end();
  };
  const auto read = [&](uint32_t slot, int i, bool wide, float (&v)[8]) {      // piece(s) i of a slot
    const uint8_t* p = s_rows + (slot - smem_u32(s_rows));
    if (wide) {
      const float4 a = *reinterpret_cast<const float4*>(p + i * piece);
      const float4 b = *reinterpret_cast<const float4*>(p + (i + 1) * piece);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      unpack8(*reinterpret_cast<const uint4*>(p + i * piece), v);
    }
  };

#pragma unroll
  for (int a = 0; a < kSlots; ++a) request(row0 + a * step, slot0 + a * stage_bytes);
  float acc[NCH][8], w[kHold ? NCH : 1][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = th + i * threads;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = w[kHold ? i : 0][j] = 0.f;
    if (kHold && c < n8) load_weight(P.weight, P.w32, 8 * c, w[i]);
  }
  float rstd_next = row0 < P.T ? P.rstd[row0] : 0.f;
  int parity = 0, stage = 0;
  for (int64_t row = row0; row - group < P.T; row += step, parity ^= 1) {
    const bool live = row < P.T;
    const float rstd = live ? rstd_next : 0.f;
    if (row + step < P.T) rstd_next = P.rstd[row + step];
    copies_wait<kSlots - 1>();
    const uint32_t slot = slot0 + stage * stage_bytes;
    stage = stage == kSlots - 1 ? 0 : stage + 1;
    // chunk i of the row: dy weight and r rstd
    const auto load = [&](int i, float (&g)[8], float (&xh)[8]) {
      const int c = th + i * threads;
#pragma unroll
      for (int j = 0; j < 8; ++j) xh[j] = g[j] = 0.f;
      if (live && c < n8) {
        read(slot, i, false, g);
        read(slot, NCH + kR * i, F32, xh);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) xh[j] *= rstd;
    };
    const auto finish = [&](int i, const float (&g)[8], const float (&xh)[8], const uint4 (&held)[kR], float mean) {
      const int c = th + i * threads;
      if (live && c < n8) {
        const int64_t at = (row * n8 + c) * 8;
        float d[8];
        if constexpr (F32) {
          const uint4 a = held[0], b = held[1];
          const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = __uint_as_float(v[j]);
        } else {
          unpack8(held[0], d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-xh[j], mean, g[j]), d[j]);
        store8(P.dx + at, d);
        if constexpr (F32) {
          if (P.dresidual_out != nullptr) store8(P.dresidual_out + at, d);
        }
      }
    };
    const auto hold = [&](int i, uint4 (&held)[kR]) {             // dresidual, as it came
#pragma unroll
      for (int m = 0; m < kR; ++m) {
        held[m] = make_uint4(0, 0, 0, 0);
        if (P.dresidual != nullptr && live && th + i * threads < n8)
          held[m] = *reinterpret_cast<const uint4*>(s_rows + (slot - smem_u32(s_rows)) +
                                                    (NCH + kR * (NCH + i) + m) * piece);
      }
    };
    float dot = 0.f;
    if constexpr (kHold) {
      float xh[NCH][8], g[NCH][8];
      uint4 held[NCH][kR];
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        load(i, g[i], xh[i]);
        hold(i, held[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[i][j] = fmaf(g[i][j], xh[i][j], acc[i][j]);
          g[i][j] *= w[i][j];
          dot = fmaf(g[i][j], xh[i][j], dot);
        }
      }
      const float mean = row_sum<LPR>(dot, s_part, parity) * P.inv_h;
      __syncwarp();                                             // the slot has been read
      request(row + kSlots * step, slot);
#pragma unroll
      for (int i = 0; i < NCH; ++i) finish(i, g[i], xh[i], held[i], mean);
    } else {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        float xh[8], g[8];
        load(i, g, xh);
        const int c = th + i * threads;
        if (c < n8) load_weight(P.weight, P.w32, 8 * c, w[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[i][j] = fmaf(g[j], xh[j], acc[i][j]);
          dot = fmaf(g[j] * w[0][j], xh[j], dot);
        }
      }
      const float mean = row_sum<LPR>(dot, s_part, parity) * P.inv_h;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        float xh[8], g[8];
        uint4 held[kR];
        load(i, g, xh);
        hold(i, held);
        const int c = th + i * threads;
        if (c < n8) load_weight(P.weight, P.w32, 8 * c, w[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= w[0][j];
        finish(i, g, xh, held, mean);
      }
      __syncwarp();
      request(row + kSlots * step, slot);
    }
  }
  copies_wait<0>();
  // the row groups' sums in order
  if constexpr (kGroups > 1) {
    float* s_acc = reinterpret_cast<float*>(s_rows);
    __syncthreads();
    if (group != 0) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s_acc[(((group - 1) * NCH + i) * 8 + j) * LPR + th] = acc[i][j];
    }
    __syncthreads();
    if (group != 0) return;
    for (int k = 0; k < kGroups - 1; ++k)
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] += s_acc[((k * NCH + i) * 8 + j) * LPR + th];
  }
  float* out = P.part + static_cast<int64_t>(blockIdx.x) * P.H;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = th + i * threads;
    if (c < n8) store8(out + 8 * c, acc[i]);
  }
}

// dweight: the CTAs' partial sums, 32 threads to a column, in order.
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* __restrict__ part, int nblk, int H,
                                                            float* __restrict__ dw) {
  __shared__ float s_sum[32][33];
  dependency_wait();
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int b = k; b < nblk; b += 32) v += part[static_cast<int64_t>(b) * H + col];
  }
  s_sum[k][lane] = v;
  __syncthreads();
  v = lanes_sum<32>(s_sum[lane][k]);
  if (lane == 0 && blockIdx.x * 32 + k < H) dw[blockIdx.x * 32 + k] = v;
}

// Calls f(lanes per row or 0, chunks per thread) with the form of a width, as
// compile-time numbers (THREE: wide rows may have three chunks a thread).
template <bool THREE, typename F>
void with_width(int H, int wide_chunks, F f) {
  const int n8 = H / 8;
  using std::integral_constant;
  if (n8 <= 8) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (n8 <= 16) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (n8 <= 32) f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (n8 <= 64) f(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  else if (n8 <= 128) f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
  else if (wide_chunks == 2) f(integral_constant<int, 0>{}, integral_constant<int, 2>{});
  else if (THREE && wide_chunks == 3) f(integral_constant<int, 0>{}, integral_constant<int, THREE ? 3 : 2>{});
  else f(integral_constant<int, 0>{}, integral_constant<int, 4>{});
}

int wide_threads(int H, int chunks) { return (H / 8 + chunks * 32 - 1) / (chunks * 32) * 32; }

int rows_at_once(int H) { return H <= 64 ? 16 : H <= 128 ? 8 : H <= 1024 ? 4 : 1; }

// Chunks per thread of a wide row: two, so that a CTA has the threads to ask for a
// row at once (forward 16384 x 4096 94.5 us with four, 91.9 with two, 20000 x 2048
// 59.2 and 55.8), up to the 512 threads of a CTA (4096 x 16384 with 1024 threads
// 128 us instead of 111).
int wide_chunks(int H) { return H <= 8192 ? 2 : 4; }
// The backward of a bf16 stream keeps three chunks in registers up to 12288 (7000
// x 8200 170 us with four that are read twice, 12288 values 103).
int bwd_chunks(int H, bool f32) { return !f32 && H > 8192 && H <= 12288 ? 3 : wide_chunks(H); }
int bwd_threads(int H, bool f32) { return H <= 1024 ? kRowThreads : wide_threads(H, bwd_chunks(H, f32)); }

// CTAs of the backward: what fits on the SMs at once (their partial sums of
// dweight are read again), at most one for each set of rows.  Of the fp32 forms up
// to 256 values (80 registers) six of the eight fit, and the others start as these
// end: no slower than a grid of six (262144 x 128 91.7 us, 92.3 with six).  Up to
// kAlone sets that one SM reads in about a microsecond are left to one CTA, which
// needs no second launch.
constexpr int kAlone = 8, kAloneElements = 32768;
int bwd_ctas(int H) { return H <= 256 ? 8 : H <= 512 ? 4 : H <= 1024 ? 2 : H <= 2048 ? 4 : H <= 4096 ? 2 : 1; }
int bwd_blocks(int T, int H) {
  const int64_t need = (static_cast<int64_t>(T) + rows_at_once(H) - 1) / rows_at_once(H);
  if (need <= kAlone && static_cast<int64_t>(T) * H <= kAloneElements) return 1;
  const int64_t most = static_cast<int64_t>(kSms) * bwd_ctas(H);
  return static_cast<int>(need < most ? need : most);
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" int mxg_rms_norm_fwd(const mxg_rms_norm_fwd_args* A, void* stream) {
  if (!A || !A->x || !A->weight || (!A->y && !A->q)) return MXG_ERR_ARG;
  if ((A->q == nullptr) != (A->s == nullptr) || (A->residual_out && !A->residual)) return MXG_ERR_ARG;
  if (A->T <= 0 || A->H <= 0 || !(A->eps >= 0.f) || !std::isfinite(A->eps)) return MXG_ERR_ARG;
  if (A->q && A->layout != MXG_LAYOUT_CANONICAL && A->layout != MXG_LAYOUT_MMA) return MXG_ERR_ARG;
  if (A->H % 8 != 0 || A->H > kMaxH) return MXG_ERR_SHAPE;
  if (A->q && (A->H % 128 != 0 || (A->layout == MXG_LAYOUT_MMA && A->T % 128 != 0))) return MXG_ERR_SHAPE;
  if (!api::aligned32(A->x) || !api::aligned32(A->residual) || !api::aligned32(A->residual_out) ||
      !api::aligned32(A->weight) || !api::aligned32(A->y) || !api::aligned32(A->q) || !api::aligned32(A->s) ||
      !api::aligned32(A->rstd))
    return MXG_ERR_ALIGN;
  api::NvtxRange nvtx("mxg.rms_norm_fwd");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NormFwdParams p{A->T, A->H, A->x, A->residual, A->residual_out, A->weight, A->weight_f32 != 0, A->eps,
                  static_cast<float>(1.0 / A->H), A->y, A->q, A->s, A->layout, A->rstd};
  const int rows = rows_at_once(A->H);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(A->T) + rows - 1) / rows);
  with_width<false>(A->H, wide_chunks(A->H), [&](auto lpr, auto nch) {
    const int block = lpr.value != 0 ? kRowThreads : wide_threads(A->H, nch.value);
    if (!A->residual) norm_fwd_kernel<lpr.value, nch.value, RES_NONE><<<grid, block, 0, st>>>(p);
    else if (A->residual_f32) norm_fwd_kernel<lpr.value, nch.value, RES_F32><<<grid, block, 0, st>>>(p);
    else norm_fwd_kernel<lpr.value, nch.value, RES_BF16><<<grid, block, 0, st>>>(p);
  });
  count_launch();
  return api::cuda_status(cudaGetLastError());
}

extern "C" size_t mxg_rms_norm_bwd_workspace_bytes(int T, int H) {
  if (T <= 0 || H <= 0 || H % 8 != 0 || H > kMaxH) return 0;
  return static_cast<size_t>(4ll * bwd_blocks(T, H) * H);
}

extern "C" int mxg_rms_norm_bwd(const mxg_rms_norm_bwd_args* A, void* stream) {
  if (!A || !A->dy || !A->r || !A->weight || !A->rstd || !A->dx || !A->dweight || !A->workspace) return MXG_ERR_ARG;
  if (A->T <= 0 || A->H <= 0) return MXG_ERR_ARG;
  if (A->dresidual_out && !A->r_f32) return MXG_ERR_ARG;
  if (A->H % 8 != 0 || A->H > kMaxH) return MXG_ERR_SHAPE;
  if (!api::aligned32(A->dy) || !api::aligned32(A->r) || !api::aligned32(A->weight) || !api::aligned32(A->rstd) ||
      !api::aligned32(A->dresidual) || !api::aligned32(A->dx) || !api::aligned32(A->dresidual_out) ||
      !api::aligned32(A->dweight) || !api::aligned32(A->workspace))
    return MXG_ERR_ALIGN;
  if (A->workspace_bytes < mxg_rms_norm_bwd_workspace_bytes(A->T, A->H)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.rms_norm_bwd");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int nblk = bwd_blocks(A->T, A->H);
  NormBwdParams p{A->T, A->H, A->dy, A->r, A->weight, A->weight_f32 != 0, A->rstd, static_cast<float>(1.0 / A->H),
                  A->dresidual, A->dx, A->dresidual_out,
                  nblk == 1 ? A->dweight : static_cast<float*>(A->workspace)};
  const int block = bwd_threads(A->H, A->r_f32 != 0);
  cudaError_t err = cudaSuccess;
  with_width<true>(A->H, bwd_chunks(A->H, A->r_f32 != 0), [&](auto lpr, auto nch) {
    const auto launch = [&](auto* kern, bool f32) {
      const int smem = row_slots(lpr.value, nch.value, f32) * nch.value * (f32 ? 5 : 3) * block * 16;
      err = allow_smem(kern, 226 * 1024);
      if (err == cudaSuccess) kern<<<nblk, block, smem, st>>>(p);
    };
    if constexpr (nch.value != 3) {               // three chunks: bf16 alone (bwd_chunks)
      if (A->r_f32) return launch(norm_bwd_kernel<lpr.value, nch.value, true>, true);
    }
    launch(norm_bwd_kernel<lpr.value, nch.value, false>, false);
  });
  MXG_TRY(err);
  count_launch();
  MXG_TRY(cudaGetLastError());
  if (nblk == 1) return MXG_OK;
  MXG_TRY(launch_after(norm_dweight_kernel, dim3((A->H + 31) / 32), dim3(1024), 0, st, p.part, nblk, A->H, A->dweight));
  return MXG_OK;
}
