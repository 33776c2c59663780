// Norm over all gradients of a model, and clipping by it.
//
//   norm = sqrt(sum of g^2 over all tensors),  out = g min(1, max_norm / norm)
//
// The tensors are cut into chunks of VEC 16-byte pieces a thread, numbered
// through; the tensor table is a kernel argument (a graph keeps its own copy, and
// nothing is copied to the device).  A CTA takes chunks blockIdx, blockIdx + grid,
// ... and writes the sum of their squares as one fp64 number; the numbers are
// added up in order, by every CTA of the second pass for itself.  Both passes are
// bound by HBM: a set that is larger than L2 is read twice.  The second pass goes
// backwards, so that what the first read last comes from L2, and its own traffic
// is marked to leave L2 first.
//
// Measured: 805 M elements (3.2 GB) into other memory 1452 us, 6.66 TB/s over the
// three passes of the data; with chunks of elements instead of pieces and plain
// caching 1601.  1.6 MB in four tensors 5.4 us, two launches.
//
// A thread's squares of a chunk are added in fp32.  Where that sum is not finite
// or so small that squares may have vanished, they are added again in fp64:
// gradients of 1e30 and of 1e-30 have norms.
#include <cmath>
#include <type_traits>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxBlocks = 152 * 4;
constexpr int kTable = 512;                       // tensors per launch
constexpr int kLong = 8, kShort = 2;              // 16-byte pieces of a chunk per thread

struct Tensor {
  const void* in;
  void* out;
  int64_t numel;
  uint32_t first;                                 // number of its first chunk
  uint32_t f32;
};
template <int N>
struct Table {
  Tensor t[N];
  uint32_t n, chunks;
};

// Elements of a chunk.
constexpr int64_t chunk_elements(int vec, bool f32) { return static_cast<int64_t>(kThreads) * vec * (f32 ? 4 : 8); }

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& tab, uint32_t chunk) {
  int lo = 0, hi = static_cast<int>(tab.n) - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.t[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <bool F32>
__device__ __forceinline__ float get(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i] : bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}

// A 16-byte piece as its 4 or 8 numbers.
template <bool F32>
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (F32) {
      v[j] = __uint_as_float(w[j]);
    } else {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// A chunk's elements: all VEC pieces of each thread at once (whole), or, at the
// end of a tensor and where memory does not start on 16 bytes, pieces and single
// elements in turn.
template <int VEC, bool F32, typename W, typename P, typename S>
__device__ __forceinline__ void for_chunk(bool wide, int64_t base, int64_t left, W whole, P piece, S single) {
  constexpr int kE = F32 ? 4 : 8;
  if (wide && left >= chunk_elements(VEC, F32)) {
    whole();
  } else {
    const int n = static_cast<int>(min(left, chunk_elements(VEC, F32))), pieces = wide ? n / kE : 0;
    for (int i = threadIdx.x; i < pieces; i += kThreads) piece(base + static_cast<int64_t>(i) * kE);
    for (int i = pieces * kE + threadIdx.x; i < n; i += kThreads) single(base + i);
  }
}

// Block-wide sum in fp64, on the threads of warp 0.
__device__ __forceinline__ double block_sum(double v, double* s_sum) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kThreads / 32 ? s_sum[threadIdx.x] : 0.0;
#pragma unroll
    for (int off = kThreads / 64; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  return v;
}

// The thread's squares of one chunk.
template <int VEC, bool F32>
__device__ __forceinline__ double chunk_squares(const void* in, int64_t base, int64_t left) {
  constexpr int kE = F32 ? 4 : 8;
  const bool wide = (reinterpret_cast<uintptr_t>(in) & 15u) == 0;
  const auto at = [&](int64_t i) { return static_cast<const uint8_t*>(in) + i * (F32 ? 4 : 2); };
  float sum = 0.f;
  uint32_t any = 0;
  const auto add = [&](const uint4& q) {
    float v[8], s = 0.f;
    unpack<F32>(q, v);
#pragma unroll
    for (int j = 0; j < kE; ++j) s = fmaf(v[j], v[j], s);
    sum += s;
    any |= F32 ? (q.x | q.y | q.z | q.w) & 0x7fffffffu : (q.x | q.y | q.z | q.w) & 0x7fff7fffu;
  };
  for_chunk<VEC, F32>(
      wide, base, left,
      [&] {
        uint4 q[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          q[i] = *reinterpret_cast<const uint4*>(at(base + static_cast<int64_t>(threadIdx.x + i * kThreads) * kE));
#pragma unroll
        for (int i = 0; i < VEC; ++i) add(q[i]);
      },
      [&](int64_t i) { add(*reinterpret_cast<const uint4*>(at(i))); },
      [&](int64_t i) {
        const float v = get<F32>(in, i);
        sum = fmaf(v, v, sum);
        any |= __float_as_uint(v) & 0x7fffffffu;
      });
  // squares below 2^-126 lose digits, at most 64 x 2^-149 of a sum that is over 2^-100
  if (any == 0 || (sum > 0x1p-100f && sum < INFINITY)) return static_cast<double>(sum);
  double exact = 0.0;
  const auto one = [&](int64_t i) {
    const double v = get<F32>(in, i);
    exact = fma(v, v, exact);
  };
  const auto eight = [&](int64_t i) {
    for (int j = 0; j < kE; ++j) one(i + j);
  };
  for_chunk<VEC, F32>(
      wide, base, left,
      [&] {
        for (int i = 0; i < VEC; ++i) eight(base + static_cast<int64_t>(threadIdx.x + i * kThreads) * kE);
      },
      eight, one);
  return exact;
}

template <int N, int VEC>
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ Table<N> tab, double* part) {
  __shared__ double s_sum[kThreads / 32];
  launch_dependents();
  double total = 0.0;
  for (uint32_t c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const Tensor& t = tab.t[tensor_of(tab, c)];
    const int64_t base = static_cast<int64_t>(c - t.first) * chunk_elements(VEC, t.f32 != 0), left = t.numel - base;
    total += t.f32 != 0 ? chunk_squares<VEC, true>(t.in, base, left) : chunk_squares<VEC, false>(t.in, base, left);
  }
  total = block_sum(total, s_sum);
  if (threadIdx.x == 0) part[blockIdx.x] = total;
}

// The sum of squares from the partial sums, in a fixed order, on the threads of
// warp 0.
__device__ __forceinline__ double squares_of(const double* part, int n, double* s_sum) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v += part[i];
  return block_sum(v, s_sum);
}

// The norm, and max_norm / norm where that is below 1.  fp64 only where fp32 has
// not the range: the sum's rounding to fp32 is halved by the root.
__device__ __forceinline__ float norm_of(double squares) {
  return squares > 0x1p-100 && squares < 0x1p100 ? sqrtf(static_cast<float>(squares))
                                                 : static_cast<float>(sqrt(squares));
}
// As two factors: out = (g x) y.  x is a power of two, 1 but for quotients that
// fp32 holds with fewer bits or not at all (a norm of 1e38 clipped to 1e-3): there
// g x is exact for every g whose output is not zero, and y a normal number, or
// the output next to the smallest.
__device__ __forceinline__ float2 split(float q) { return make_float2(1.f, q); }
__device__ __forceinline__ float2 split(double q) {
  if (q < 0x1p-200) return make_float2(0x1p-126f, static_cast<float>(q * 0x1p126));
  if (q < 0x1p-100) return make_float2(0x1p-76f, static_cast<float>(q * 0x1p76));
  return split(static_cast<float>(q));
}
__device__ __forceinline__ float2 factor_of(double squares, float max_norm) {
  if (squares > 0x1p-100 && squares < 0x1p100 && max_norm > 0x1p-50f) {
    const float norm = sqrtf(static_cast<float>(squares));
    return split(norm <= max_norm ? 1.f : max_norm / norm);
  }
  const double norm = sqrt(squares);
  return split(norm <= max_norm ? 1.0 : max_norm / norm);
}
// The same of a norm in fp32.
__device__ __forceinline__ float2 factor_of(float norm, float max_norm) {
  if (norm < 0x1p50f && max_norm > 0x1p-50f) return split(norm <= max_norm ? 1.f : max_norm / norm);
  return split(norm <= max_norm ? 1.0 : static_cast<double>(max_norm) / norm);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int n, float* norm) {
  __shared__ double s_sum[kThreads / 32];
  dependency_wait();
  const double v = squares_of(part, n, s_sum);
  if (threadIdx.x == 0) *norm = norm_of(v);
}

template <int VEC, bool F32>
__device__ __forceinline__ void chunk_scale(const void* in, void* out, float2 f, int64_t base, int64_t left) {
  constexpr int kE = F32 ? 4 : 8;
  const bool wide = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const auto from = [&](int64_t i) {
    return reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(in) + i * (F32 ? 4 : 2));
  };
  const auto store = [&](int64_t i, const uint4& q) {
    float v[8];
    unpack<F32>(q, v);
#pragma unroll
    for (int j = 0; j < kE; ++j) v[j] = v[j] * f.x * f.y;
    uint4 r;
    if constexpr (F32) r = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else r = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + i * (F32 ? 4 : 2)), r);
  };
  for_chunk<VEC, F32>(
      wide, base, left,
      [&] {
        uint4 q[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[i] = __ldcs(from(base + static_cast<int64_t>(threadIdx.x + i * kThreads) * kE));
#pragma unroll
        for (int i = 0; i < VEC; ++i) store(base + static_cast<int64_t>(threadIdx.x + i * kThreads) * kE, q[i]);
      },
      [&](int64_t i) { store(i, __ldcs(from(i))); },
      [&](int64_t i) {
        const float v = get<F32>(in, i) * f.x * f.y;
        if constexpr (F32) static_cast<float*>(out)[i] = v;
        else static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
      });
}

// out = g min(1, max_norm / norm).  The norm comes from the partial sums (part), or from the caller
// (norm_in).
template <int N, int VEC>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<N> tab, const double* part, int nparts,
                                                         const float* norm_in, float max_norm, float* norm_out) {
  __shared__ double s_sum[kThreads / 32];
  __shared__ float2 s_factor;
  dependency_wait();
  // NaN makes everything NaN, infinity everything zero (and NaN what is infinite)
  float2 f;
  if (part != nullptr) {
    const double squares = squares_of(part, nparts, s_sum);
    if (threadIdx.x == 0) {
      s_factor = factor_of(squares, max_norm);
      if (blockIdx.x == 0 && norm_out != nullptr) *norm_out = norm_of(squares);
    }
    __syncthreads();
    f = s_factor;
  } else {
    f = factor_of(*norm_in, max_norm);
  }
  for (uint32_t k = blockIdx.x; k < tab.chunks; k += gridDim.x) {
    const uint32_t c = tab.chunks - 1 - k;
    const Tensor& t = tab.t[tensor_of(tab, c)];
    if (f.y == 1.f && t.in == t.out) continue;
    const int64_t base = static_cast<int64_t>(c - t.first) * chunk_elements(VEC, t.f32 != 0), left = t.numel - base;
    if (t.f32 != 0) chunk_scale<VEC, true>(t.in, t.out, f, base, left);
    else chunk_scale<VEC, false>(t.in, t.out, f, base, left);
  }
}

int64_t chunks_of(const mxg_tensor& t, int vec) {
  const int64_t e = chunk_elements(vec, t.f32 != 0);
  return (t.numel + e - 1) / e;
}

int check_tensors(const mxg_tensor* t, int n, bool out) {
  if (!t || n <= 0) return MXG_ERR_ARG;
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (t[i].numel < 0 || (t[i].f32 != 0 && t[i].f32 != 1)) return MXG_ERR_ARG;
    if (t[i].numel == 0) continue;
    if (!t[i].in || (out && !t[i].out)) return MXG_ERR_ARG;
    const uintptr_t size = t[i].f32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(t[i].in) % size != 0) return MXG_ERR_ALIGN;
    if (out && reinterpret_cast<uintptr_t>(t[i].out) % size != 0) return MXG_ERR_ALIGN;
    if (t[i].numel > (1ll << 45)) return MXG_ERR_SHAPE;
    chunks += chunks_of(t[i], kShort);
    if (chunks > INT32_MAX) return MXG_ERR_SHAPE;
  }
  return MXG_OK;
}

int blocks_of(uint32_t chunks) { return chunks < kMaxBlocks ? static_cast<int>(chunks) : kMaxBlocks; }

// Calls f(table of up to N tensors, pieces of a chunk) for every launch the
// tensors need; a small set travels in a small argument, and in short chunks
// where long ones would be fewer than SMs.  Tensors without elements take no entry.
template <typename F>
cudaError_t for_tables(const mxg_tensor* t, int n, F f) {
  int at = 0;
  int64_t all = 0;
  for (int i = 0; i < n; ++i) all += chunks_of(t[i], kLong);
  const int vec = all < 152 ? kShort : kLong;
  while (true) {
    while (at < n && t[at].numel == 0) ++at;
    if (at >= n) return cudaSuccess;
    const auto fill = [&](auto& tab) {
      tab.n = tab.chunks = 0;
      constexpr uint32_t most = sizeof(tab.t) / sizeof(tab.t[0]);
      for (; at < n && tab.n < most; ++at) {
        if (t[at].numel == 0) continue;
        tab.t[tab.n++] = Tensor{t[at].in, t[at].out, t[at].numel, tab.chunks, static_cast<uint32_t>(t[at].f32)};
        tab.chunks += static_cast<uint32_t>(chunks_of(t[at], vec));
      }
    };
    cudaError_t err;
    if (n - at <= 16) {
      Table<16> tab;
      fill(tab);
      err = vec == kLong ? f(tab, std::integral_constant<int, kLong>{}) : f(tab, std::integral_constant<int, kShort>{});
    } else {
      static thread_local Table<kTable> tab;
      fill(tab);
      err = vec == kLong ? f(tab, std::integral_constant<int, kLong>{}) : f(tab, std::integral_constant<int, kShort>{});
    }
    if (err != cudaSuccess) return err;
  }
}

int table_count(int n) { return (n - 1) / kTable + 1; }                // n > 0

// The partial sums of all tensors; their number to *nparts.
cudaError_t launch_square_sums(const mxg_tensor* t, int n, double* part, int* nparts, cudaStream_t s) {
  *nparts = 0;
  return for_tables(t, n, [&](const auto& tab, auto vec) {
    constexpr int N = sizeof(tab.t) / sizeof(tab.t[0]);
    const int blocks = blocks_of(tab.chunks);
    square_sum_kernel<N, vec.value><<<blocks, kThreads, 0, s>>>(tab, part + *nparts);
    count_launch();
    *nparts += blocks;
    return cudaGetLastError();
  });
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" size_t mxg_grad_norm_workspace_bytes(int n) {
  return n <= 0 ? 0 : static_cast<size_t>(table_count(n)) * kMaxBlocks * sizeof(double);
}

extern "C" int mxg_grad_norm(const mxg_tensor* tensors, int n, float* norm, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!norm || !workspace) return MXG_ERR_ARG;
  if (const int err = check_tensors(tensors, n, false)) return err;
  if (!api::aligned32(workspace) || !api::aligned32(norm)) return MXG_ERR_ALIGN;
  if (workspace_bytes < mxg_grad_norm_workspace_bytes(n)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.grad_norm");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int nparts = 0;
  double* part = static_cast<double*>(workspace);
  MXG_TRY(launch_square_sums(tensors, n, part, &nparts, s));
  MXG_TRY(launch_after(norm_kernel, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(part), nparts, norm));
  return MXG_OK;
}

extern "C" int mxg_grad_clip(const mxg_tensor* tensors, int n, float max_norm, const float* norm_in, float* norm_out,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (!(max_norm > 0.f) || (!norm_in && !workspace) || (norm_in && norm_out)) return MXG_ERR_ARG;
  if (const int err = check_tensors(tensors, n, true)) return err;
  if (!api::aligned32(workspace) || !api::aligned32(norm_in) || !api::aligned32(norm_out)) return MXG_ERR_ALIGN;
  if (!norm_in && workspace_bytes < mxg_grad_norm_workspace_bytes(n)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.grad_clip");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int nparts = 0;
  double* part = static_cast<double*>(workspace);
  if (!norm_in) MXG_TRY(launch_square_sums(tensors, n, part, &nparts, s));
  bool told = norm_out == nullptr;
  MXG_TRY(for_tables(tensors, n, [&](const auto& tab, auto vec) {
    constexpr int N = sizeof(tab.t) / sizeof(tab.t[0]);
    float* to = told ? nullptr : norm_out;
    told = true;
    return launch_after(scale_kernel<N, vec.value>, dim3(blocks_of(tab.chunks)), dim3(kThreads), 0, s, tab,
                        static_cast<const double*>(norm_in ? nullptr : part), nparts, norm_in, max_norm, to);
  }));
  if (!told)                                      // no tensor has elements: the norm is zero
    MXG_TRY(launch_after(norm_kernel, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(part), nparts, norm_out));
  return MXG_OK;
}
