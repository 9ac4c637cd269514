// The global norm of many tensors and their scaling to a largest norm.
//
// Two passes: a workgroup squares and adds a chunk of one tensor in 64 bits
// and leaves one partial sum; then each workgroup of the second pass adds all
// partial sums (some thousands, from the caches) in one fixed order, takes the
// factor from them, and scales its chunk.  No atomics, no flags between
// workgroups: the same bits on every run.
//
// Bound by HBM: a square costs a conversion and a 64-bit fma, a fraction of its
// load.  The second pass takes the chunks in the opposite order, so that what
// the first read last comes from the last-level cache; where nothing is clipped
// in place it reads no gradient at all.
#include "clip.h"
#include "common.hpp"

namespace muon {
namespace clip {

namespace {

constexpr int NT = 256;
typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));

template <typename E> __device__ __forceinline__ float wide(E v);
template <> __device__ __forceinline__ float wide<uint16_t>(uint16_t v) { return bf16_bits_to_f32(v); }
template <> __device__ __forceinline__ float wide<float>(float v) { return v; }
template <typename E> __device__ __forceinline__ E narrow(float v);
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }

// The sum over the workgroup, the same order each time, in every thread.
__device__ __forceinline__ double group_sum(double v) {
  __shared__ double s_sum[NT / 64];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if (threadIdx.x % 64 == 0) s_sum[threadIdx.x / 64] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) v += s_sum[w];
  return v;
}

// The tensor that workgroup b belongs to.
__device__ __forceinline__ int find(const Table& t, uint32_t b) {
  int lo = 0, hi = t.num - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.t[mid].first <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Calls f(place, elements, n) for the run's 16-byte pieces, U of a thread's in
// flight, and for the elements left over.  `elements` holds n of them.
template <typename E, typename F>
__device__ __forceinline__ void each(const E* g, int64_t n, F f) {
  constexpr int PV = 16 / sizeof(E), U = 4;
  int64_t i = (int64_t)threadIdx.x * PV;
  for (; i + (int64_t)(U - 1) * NT * PV + PV <= n; i += (int64_t)U * NT * PV) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = *(const V*)(g + i + (int64_t)u * NT * PV);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      E e[PV];
      __builtin_memcpy(e, &v[u], 16);
      f(i + (int64_t)u * NT * PV, e, PV);
    }
  }
  for (; i < n; i += (int64_t)NT * PV) {
    E e[PV];
    const int m = (int)(n - i < PV ? n - i : PV);
    if (m == PV) {
      __builtin_memcpy(e, g + i, 16);
    } else {
#pragma unroll
      for (int j = 0; j < PV; ++j) e[j] = j < m ? g[i + j] : (E)0;
    }
    f(i, e, m);
  }
}

template <typename E>
__device__ __forceinline__ double squares(const E* g, int64_t n) {
  constexpr int PV = 16 / sizeof(E);
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  each(g, n, [&](int64_t, const E* e, int) {  // (zeros behind the last)
#pragma unroll
    for (int j = 0; j < PV; ++j) {
      const double d = (double)wide<E>(e[j]);
      sum[j % 4] = __builtin_fma(d, d, sum[j % 4]);
    }
  });
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

__global__ void __launch_bounds__(NT) squares_kernel(const Table t, double* part) {
  const Tensor& x = t.t[find(t, blockIdx.x)];
  const int64_t at = (int64_t)(blockIdx.x - x.first) * t.chunk, n = x.n - at < t.chunk ? x.n - at : t.chunk;
  double v = x.gbf16 ? squares((const uint16_t*)x.g + at, n) : squares((const float*)x.g + at, n);
  v = group_sum(v);
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

// The norm from all partial sums.
__device__ __forceinline__ double norm_of(const double* part, int64_t count) {
  double v = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < count; i += NT) v += part[i];
  return sqrt(group_sum(v));
}

__global__ void __launch_bounds__(NT) norm_kernel(const double* part, int64_t count, float* norm) {
  const double v = norm_of(part, count);
  if (threadIdx.x == 0) norm[0] = (float)v;
}

template <typename E, typename O>
__device__ __forceinline__ void scale(const E* g, O* out, int64_t n, float by) {
  constexpr int PV = 16 / sizeof(E);
  each(g, n, [&](int64_t i, const E* e, int m) {
    O o[PV];
#pragma unroll
    for (int j = 0; j < PV; ++j) o[j] = narrow<O>(wide<E>(e[j]) * by);
    if (m == PV) {
      __builtin_memcpy(out + i, o, sizeof(o));
    } else {
#pragma unroll
      for (int j = 0; j < PV; ++j)
        if (j < m) out[i + j] = o[j];
    }
  });
}

__global__ void __launch_bounds__(NT) scale_kernel(const Table t, const double* part, int64_t count, float max_norm,
                                                   float* norm) {
  const uint32_t b = t.groups - 1 - blockIdx.x;
  const double v = norm_of(part, count);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)v;
  const bool kept = v <= (double)max_norm;
  const float by = kept ? 1.0f : (float)((double)max_norm / v);
  const Tensor& x = t.t[find(t, b)];
  if (kept && x.g == x.out) return;
  const int64_t at = (int64_t)(b - x.first) * t.chunk, n = x.n - at < t.chunk ? x.n - at : t.chunk;
  if (x.gbf16) {
    const uint16_t* g = (const uint16_t*)x.g + at;
    if (x.obf16) scale(g, (uint16_t*)x.out + at, n, by);
    else scale(g, (float*)x.out + at, n, by);
  } else {
    const float* g = (const float*)x.g + at;
    if (x.obf16) scale(g, (uint16_t*)x.out + at, n, by);
    else scale(g, (float*)x.out + at, n, by);
  }
}

}  // namespace

hipError_t launch_squares(const Table& t, double* part, int64_t from, hipStream_t s) {
  hipLaunchKernelGGL(squares_kernel, dim3(t.groups), dim3(NT), 0, s, t, part + from);
  return hipGetLastError();
}
hipError_t launch_norm(const double* part, int64_t count, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(NT), 0, s, part, count, norm);
  return hipGetLastError();
}
hipError_t launch_scale(const Table& t, const double* part, int64_t count, float max_norm, float* norm, bool first,
                        hipStream_t s) {
  hipLaunchKernelGGL(scale_kernel, dim3(t.groups), dim3(NT), 0, s, t, part, count, max_norm, first ? norm : nullptr);
  return hipGetLastError();
}

}  // namespace clip
}  // namespace muon
