// The 8-bit floating-point form of rows and of weights, and back.
//
// A block (128 values of a row, or 128 x 128 of a matrix) gets scale = 2^e with
// the smallest e >= -126 for which max|v| <= 448 * 2^e, held as the byte e +
// 127, and q = v / scale in e4m3.  A power of two makes the division and the
// restored value exact, so the conversion's rounding (nearest even, in the
// hardware) is the only one.  448 = 1.75 * 2^8: with max|v| = m * 2^E, e = E - 8,
// one more if m > 1.75, which reads off the bits of the largest magnitude.
//
// Bound by HBM.  Every value is held in registers between the search for the
// block's largest and its conversion, so it is read once.
#include <algorithm>

#include "common.hpp"
#include "float8.h"

namespace muon {
namespace f8 {

namespace {

template <typename T> struct Elem;
template <> struct Elem<BF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ uint32_t bits(uint16_t v) { return (uint32_t)v << 16; }
  static __device__ __forceinline__ uint16_t from(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
template <> struct Elem<F32> {
  typedef float type;
  static __device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
  static __device__ __forceinline__ float from(float v) { return v; }
};

// Eight consecutive elements of a row, n of which exist, zeros behind; at any
// alignment of the element's own.
template <typename T>
__device__ __forceinline__ void load8(const typename Elem<T>::type* p, int n, uint32_t v[8]) {
  typename Elem<T>::type e[8];
  if (n >= 8) {
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    constexpr int NV = 8 * sizeof(e[0]) / 16;
    V w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i] = __builtin_nontemporal_load((const V*)p + i);
    __builtin_memcpy(e, w, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : (typename Elem<T>::type)0;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = Elem<T>::bits(e[i]);
}

__device__ __forceinline__ uint32_t largest(const uint32_t v[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, v[i] & 0x7fffffffu);
  return top;
}
// Over aligned groups of L lanes.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

// A block's scale byte from the bits of its largest magnitude: infinity and NaN
// are on top.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int b = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return top >= 0x7f800000u ? 255u : (uint32_t)max(b, 1);
}
// Eight values times 1 / scale in e4m3 (2^-e from the byte e + 127 <= 247), n
// of which are written.
__device__ __forceinline__ void store8(uint8_t* q, int n, const uint32_t v[8], uint32_t byte) {
  const float by = __uint_as_float((254u - byte) << 23);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[4 * i + j]) * by;
    uint32_t d = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    d = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], (int)d, true);
    w[i] = byte == 255u ? 0x7f7f7f7fu : d;
  }
  if (n >= 8) {
    typedef uint32_t V __attribute__((ext_vector_type(2), aligned(1)));
    *(V*)q = V{w[0], w[1]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// Rows: 16 lanes per block of 128, N blocks per lane a step apart, all loads in
// flight before the first use.
template <typename T, int N>
__global__ void __launch_bounds__(256) rows_kernel(const FormParams p, int64_t from, int64_t blocks, int kb) {
  const int64_t step = (int64_t)gridDim.x * 16;
  int64_t b = from + (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
  const int at = threadIdx.x % 16 * 8;
  uint32_t v[N][8];
  int64_t row[N];
  int col[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t k = b + i * step;
    row[i] = k / kb;
    col[i] = (int)(k - row[i] * kb) * kBlock + at;
    const int n = k < blocks ? (int)min((int64_t)8, p.cols - col[i]) : 0;
    load8<T>((const typename Elem<T>::type*)p.x + row[i] * p.ldx + col[i], n, v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t k = b + i * step;
    const uint32_t byte = scale_byte(lanes_max<16>(largest(v[i])));
    if (k >= blocks) continue;
    store8(p.q + row[i] * p.ldq + col[i], (int)min((int64_t)8, p.cols - col[i]), v[i], byte);
    if (at == 0) p.scale[k] = (uint8_t)byte;
  }
}

// Weights: a workgroup per 128 x 128 values, 64 of them per thread.
template <typename T>
__global__ void __launch_bounds__(256) squares_kernel(const FormParams p, int64_t from, int kb, int nb) {
  __shared__ uint32_t s_top[4];
  const int64_t k = from + blockIdx.x;
  const int64_t m = k / ((int64_t)kb * nb);
  const int in = (int)(k - m * kb * nb), r0 = in / kb * kBlock, c = in % kb * kBlock + threadIdx.x % 16 * 8;
  const int n = (int)min((int64_t)8, p.cols - c);
  const typename Elem<T>::type* x = (const typename Elem<T>::type*)p.x + m * p.sx + c;
  uint32_t v[8][8], top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i * 16 + threadIdx.x / 16;
    load8<T>(x + r * p.ldx, r < p.rows ? n : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, largest(v[i]));
  top = lanes_max<64>(top);
  if (threadIdx.x % 64 == 0) s_top[threadIdx.x / 64] = top;
  __syncthreads();
  top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
  const uint32_t byte = scale_byte(top);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i * 16 + threadIdx.x / 16;
    if (r < p.rows) store8(p.q + m * p.sq + r * p.ldq + c, n, v[i], byte);
  }
  if (threadIdx.x == 0) p.scale[k] = (uint8_t)byte;
}

// Back: 16 values of a row per thread and step.
template <typename T, int N>
__global__ void __launch_bounds__(256) back_kernel(const FormParams p, int64_t from, int64_t chunks, int cpr, int kb,
                                                   int nb) {
  typedef typename Elem<T>::type E;
  const int64_t step = (int64_t)gridDim.x * 256;
  const int64_t first = from + (int64_t)blockIdx.x * 256 + threadIdx.x;
  u32x4 v[N];
  uint32_t byte[N];
  E* out[N];
  int n[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t k = first + i * step;
    n[i] = 0;
    byte[i] = 0;
    v[i] = u32x4{0, 0, 0, 0};
    if (k < chunks) {
      const int64_t row = k / cpr, m = row / p.rows, r = row - m * p.rows;
      const int c = (int)(k - row * cpr) * 16;
      n[i] = (int)min((int64_t)16, p.cols - c);
      // (rows start at 16 bytes and may be read to the next 16)
      v[i] = *(const u32x4*)(p.q + m * p.sq + r * p.ldq + c);
      byte[i] = p.scale[(p.block_rows == 1 ? row : m * nb + r / kBlock) * kb + c / kBlock];
      out[i] = (E*)p.x + m * p.sx + r * p.ldx + c;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (n[i] == 0) continue;
    // (2^-127 is no normal number)
    const float f = byte[i] == 255u ? __uint_as_float(0x7fc00000u)
                    : byte[i] == 0u ? __uint_as_float(1u << 22)
                                    : __uint_as_float(byte[i] << 23);
    E e[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4 w = {__builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 0), __builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 1),
                       __builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 2), __builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 3)};
#pragma unroll
      for (int l = 0; l < 4; ++l) e[4 * j + l] = Elem<T>::from(w[l] * f);
    }
    if (n[i] >= 16) {
      typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
      constexpr int NV = (int)sizeof(e) / 16;
      V w[NV];
      __builtin_memcpy(w, e, sizeof(e));
#pragma unroll
      for (int j = 0; j < NV; ++j) __builtin_nontemporal_store(w[j], (V*)out[i] + j);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < n[i]) out[i][j] = e[j];
    }
  }
}

// Workgroups of a launch: a launch has fewer than 2^32 threads.
constexpr int64_t kMaxGroups = (1ll << 32) / 256 - 1;

// launch(first, workgroups) over `total` items of which a workgroup takes `per`.
template <typename L>
hipError_t in_parts(int64_t total, int64_t per, L launch) {
  for (int64_t from = 0; from < total; from += kMaxGroups * per) {
    launch(from, (uint32_t)std::min(kMaxGroups, (total - from + per - 1) / per));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize(const FormParams& p, bool bf16, hipStream_t s) {
  const int kb = (int)((p.cols + kBlock - 1) / kBlock), nb = (int)((p.rows + kBlock - 1) / kBlock);
  if (p.block_rows == kBlock)
    return in_parts(p.count * nb * kb, 1, [&](int64_t from, uint32_t groups) {
      if (bf16) hipLaunchKernelGGL((squares_kernel<BF16>), dim3(groups), dim3(256), 0, s, p, from, kb, nb);
      else hipLaunchKernelGGL((squares_kernel<F32>), dim3(groups), dim3(256), 0, s, p, from, kb, nb);
    });
  // matrices of rows: rows of one matrix after another
  for (int64_t m = 0; m < p.count; ++m) {
    FormParams o = p;
    o.x = (char*)p.x + m * p.sx * (bf16 ? 2 : 4);
    o.q = p.q + m * p.sq;
    o.scale = p.scale + m * p.rows * kb;
    const int64_t blocks = p.rows * kb;
    auto go = [&](auto kernel, int per) {
      return in_parts(blocks, per, [&](int64_t from, uint32_t groups) {
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(256), 0, s, o, from, std::min(blocks, from + kMaxGroups * per), kb);
      });
    };
    hipError_t e;
    if (blocks >= 16 * 4 * 1024) e = bf16 ? go(rows_kernel<BF16, 4>, 64) : go(rows_kernel<F32, 4>, 64);
    else e = bf16 ? go(rows_kernel<BF16, 1>, 16) : go(rows_kernel<F32, 1>, 16);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dequantize(const FormParams& p, bool bf16, hipStream_t s) {
  const int kb = (int)((p.cols + kBlock - 1) / kBlock), nb = (int)((p.rows + kBlock - 1) / kBlock);
  const int cpr = (int)((p.cols + 15) / 16);
  const int64_t chunks = p.count * p.rows * cpr;
  auto go = [&](auto kernel, int per) {
    return in_parts(chunks, per, [&](int64_t from, uint32_t groups) {
      hipLaunchKernelGGL(kernel, dim3(groups), dim3(256), 0, s, p, from, std::min(chunks, from + kMaxGroups * per), cpr,
                         kb, nb);
    });
  };
  if (chunks >= 256 * 2 * 1024) return bf16 ? go(back_kernel<BF16, 2>, 512) : go(back_kernel<F32, 2>, 512);
  return bf16 ? go(back_kernel<BF16, 1>, 256) : go(back_kernel<F32, 1>, 256);
}

}  // namespace f8
}  // namespace muon
