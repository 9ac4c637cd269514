// The global norm of many tensors and their scaling to a largest norm.
//
// Two passes: a workgroup squares and adds a chunk of one tensor in 64 bits
// and leaves one partial sum; then each workgroup of the second pass adds all
// partial sums (some thousands, from the caches) in one fixed order, takes the
// factor from them, and scales its chunk.  No atomics, no flags between
// workgroups: the same bits on every run.
//
// Bound by HBM (932 M fp32 elements: 600 us, 6.2 TB/s, and 1377, 5.4): a square
// costs a conversion and a 64-bit fma, a fraction of its load.  The second pass goes through the tensors backwards, so that what the
// first read last comes from the last-level cache; where nothing is clipped in
// place it reads no gradient at all.
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

// The sum over a workgroup of W waves, the same order each time, in every thread.
template <int W = NT / 64>
__device__ __forceinline__ double group_sum(double v) {
  __shared__ double s_sum[W];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if (threadIdx.x % 64 == 0) s_sum[threadIdx.x / 64] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int w = 0; w < W; ++w) v += s_sum[w];
  return v;
}

// The factor by * 2^exp that takes a norm to at most max_norm.  exp is 0 unless
// the factor lies under fp32's normal numbers (a norm of 2^126 max_norm and more),
// where fp32 alone would hold few of its bits; by is then in [1/2, 1].
struct Factor {
  bool kept;
  float by;
  int exp;
};
__device__ __forceinline__ Factor factor(double norm, float max_norm) {
  const bool kept = norm <= (double)max_norm;
  double by = kept ? 1.0 : (double)max_norm / norm;
  int exp = 0;
  if (by > 0.0 && by < 0x1p-126) by = frexp(by, &exp);
  return {kept, (float)by, exp};
}
// (a product under fp32's normal numbers is rounded once more, and vanishes if exp is not 0)
__device__ __forceinline__ float times(float v, const Factor& f) { return __builtin_amdgcn_ldexpf(v * f.by, f.exp); }

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

// Calls f(place, elements, n) for what workgroup j of `groups` takes of n
// elements: every groups-th piece of U 16-byte loads per thread (all workgroups
// sweep the tensor side by side: streams of their own, a chunk apart, reached
// 4.8 TB/s), from the last to the first if BACK; and one of them what is left
// over.  `elements` holds n of them, zeros behind.
template <bool BACK, typename E, typename F>
__device__ __forceinline__ void each(const E* g, int64_t n, uint32_t j, uint32_t groups, F f) {
  constexpr int PV = 16 / sizeof(E), U = 4, PIECE = NT * PV * U;
  const int64_t pieces = n / PIECE;
  const int64_t mine = pieces > j ? (pieces - j + groups - 1) / groups : 0;
  for (int64_t k = 0; k < mine; ++k) {
    const int64_t i = (j + (BACK ? mine - 1 - k : k) * groups) * PIECE + (int64_t)threadIdx.x * PV;
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (BACK) v[u] = __builtin_nontemporal_load((const V*)(g + i + u * NT * PV));
      else v[u] = *(const V*)(g + i + u * NT * PV);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      E e[PV];
      __builtin_memcpy(e, &v[u], 16);
      f(i + u * NT * PV, e, PV);
    }
  }
  if (j != pieces % groups) return;
  for (int64_t i = pieces * PIECE + (int64_t)threadIdx.x * PV; i < n; i += NT * PV) {
    E e[PV];
    const int m = (int)(n - i < PV ? n - i : PV);
    if (m == PV) {
      __builtin_memcpy(e, g + i, 16);
    } else {
#pragma unroll
      for (int l = 0; l < PV; ++l) e[l] = l < m ? g[i + l] : (E)0;
    }
    f(i, e, m);
  }
}

template <typename E>
__device__ __forceinline__ double squares(const E* g, int64_t n, uint32_t j, uint32_t groups) {
  constexpr int PV = 16 / sizeof(E);
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  each<false>(g, n, j, groups, [&](int64_t, const E* e, int) {
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
  const uint32_t j = blockIdx.x - x.first, groups = (uint32_t)((x.n + t.chunk - 1) / t.chunk);
  double v = x.gbf16 ? squares((const uint16_t*)x.g, x.n, j, groups) : squares((const float*)x.g, x.n, j, groups);
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
__device__ __forceinline__ void scale(const E* g, O* out, int64_t n, uint32_t j, uint32_t groups, const Factor& f) {
  constexpr int PV = 16 / sizeof(E);
  each<true>(g, n, j, groups, [&](int64_t i, const E* e, int m) {
    O o[PV];
#pragma unroll
    for (int l = 0; l < PV; ++l) o[l] = narrow<O>(times(wide<E>(e[l]), f));
    if (m == PV) {
      // (past the caches, which hold what the first pass read last)
      constexpr int WB = sizeof(O) * PV < 16 ? 8 : 16, NW = sizeof(O) * PV / WB;
      typedef uint32_t W __attribute__((ext_vector_type(WB / 4), aligned(2)));
      W w[NW];
      __builtin_memcpy(w, o, NW * WB);
#pragma unroll
      for (int j = 0; j < NW; ++j) __builtin_nontemporal_store(w[j], (W*)(out + i) + j);
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
  const Factor f = factor(v, max_norm);
  const Tensor& x = t.t[find(t, b)];
  if (f.kept && x.g == x.out) return;
  const uint32_t j = b - x.first, groups = (uint32_t)((x.n + t.chunk - 1) / t.chunk);
  if (x.gbf16) {
    const uint16_t* g = (const uint16_t*)x.g;
    if (x.obf16) scale(g, (uint16_t*)x.out, x.n, j, groups, f);
    else scale(g, (float*)x.out, x.n, j, groups, f);
  } else {
    const float* g = (const float*)x.g;
    if (x.obf16) scale(g, (uint16_t*)x.out, x.n, j, groups, f);
    else scale(g, (float*)x.out, x.n, j, groups, f);
  }
}

// Few elements: one workgroup does all of it, a wave per kSmallChunk elements, so
// that a call is one launch.  `scaled` says whether there is anything to write
// but the norm.
template <typename E, typename F>
__device__ __forceinline__ void wave_each(const E* g, int n, F f) {
  constexpr int PV = 16 / sizeof(E), U = kSmallChunk / (64 * PV);
  const int lane = threadIdx.x % 64;
  V v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * 64 + lane) * PV;
    if (i + PV <= n) v[u] = *(const V*)(g + i);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * 64 + lane) * PV, m = n - i < PV ? n - i : PV;
    E e[PV];
    if (m == PV) {
      __builtin_memcpy(e, &v[u], 16);
    } else {
#pragma unroll
      for (int l = 0; l < PV; ++l) e[l] = l < m ? g[i + l] : (E)0;
    }
    if (m > 0) f(i, e, m);
  }
}
template <typename E, typename O>
__device__ __forceinline__ void wave_scale(const E* g, O* out, int n, const Factor& f) {
  constexpr int PV = 16 / sizeof(E);
  wave_each(g, n, [&](int i, const E* e, int m) {
    O o[PV];
#pragma unroll
    for (int l = 0; l < PV; ++l) o[l] = narrow<O>(times(wide<E>(e[l]), f));
    if (m == PV) {
      __builtin_memcpy(out + i, o, sizeof(o));
    } else {
#pragma unroll
      for (int l = 0; l < PV; ++l)
        if (l < m) out[i + l] = o[l];
    }
  });
}
constexpr int kSmallWaves = kSmallGroups;
__global__ void __launch_bounds__(64 * kSmallWaves) small_kernel(const Table t, int scaled, float max_norm, float* norm) {
  const uint32_t wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
  const bool busy = wave < t.groups;
  const Tensor& x = t.t[find(t, busy ? wave : 0)];
  const int64_t at = busy ? (int64_t)(wave - x.first) * kSmallChunk : 0;
  const int n = busy ? (int)(x.n - at < kSmallChunk ? x.n - at : kSmallChunk) : 0;
  double sum = 0.0;
  auto square = [&](float v) { sum = __builtin_fma((double)v, (double)v, sum); };
  if (x.gbf16) {
    wave_each((const uint16_t*)x.g + at, n, [&](int, const uint16_t* e, int) {
#pragma unroll
      for (int l = 0; l < 8; ++l) square(wide<uint16_t>(e[l]));
    });
  } else {
    wave_each((const float*)x.g + at, n, [&](int, const float* e, int) {
#pragma unroll
      for (int l = 0; l < 4; ++l) square(e[l]);
    });
  }
  const double v = sqrt(group_sum<kSmallWaves>(sum));
  if (threadIdx.x == 0) norm[0] = (float)v;
  if (!scaled) return;
  // (a wave writes what it alone has read)
  const Factor f = factor(v, max_norm);
  if (f.kept && x.g == x.out) return;
  if (x.gbf16) {
    const uint16_t* g = (const uint16_t*)x.g + at;
    if (x.obf16) wave_scale(g, (uint16_t*)x.out + at, n, f);
    else wave_scale(g, (float*)x.out + at, n, f);
  } else {
    const float* g = (const float*)x.g + at;
    if (x.obf16) wave_scale(g, (uint16_t*)x.out + at, n, f);
    else wave_scale(g, (float*)x.out + at, n, f);
  }
}

}  // namespace

hipError_t launch_small(const Table& t, bool scaled, float max_norm, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(small_kernel, dim3(1), dim3(64 * kSmallWaves), 0, s, t, scaled ? 1 : 0, max_norm, norm);
  return hipGetLastError();
}
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
