// Row-wise kernels of the 8-bit linear layer: root-mean-square norm (with
// the residual's addition and an 8-bit output), its backward pass, and the
// 8-bit form of a row and back.
//
// Every kernel is bound by HBM: a row is read once, held in registers, and
// written once.  A row belongs to one wave (no barrier) up to 4096 columns,
// to 4 or 16 waves above; each lane holds NC chunks of 8 consecutive columns
// (16 bytes of bf16).  Rows need no alignment: gfx950 takes 16-byte global
// accesses at any address of the element's own alignment, and the ragged
// last chunk of a row goes element by element.
//
// The 8-bit form of a row v is scale = 2^e with the smallest e >= -126 for
// which max|v| <= 127 * 2^e, and q = rint(v / scale).  A power of two makes
// the division and the restored value q * scale exact, so rint is the only
// rounding (at most scale / 2), and lets the gradient products fold the scale
// into a bf16 operand without rounding.
#include "common.hpp"
#include "linear8.h"

namespace muon {
namespace l8 {

namespace {

template <typename T> struct Elem;
template <> struct Elem<BF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float to(uint16_t v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t from(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);  // v_cvt: nearest even
  }
};
template <> struct Elem<F32> {
  typedef float type;
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
struct I8 {};
template <> struct Elem<I8> {
  typedef int8_t type;
  static __device__ __forceinline__ float to(int8_t v) { return (float)v; }
};

// Eight consecutive elements at p, of which n (>= 1) exist; the others are 0.
template <typename T>
__device__ __forceinline__ void load8(const typename Elem<T>::type* p, int n, float v[8]) {
  typename Elem<T>::type e[8];
  if (n >= 8) {
    __builtin_memcpy(e, p, sizeof(e));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Elem<T>::to(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? Elem<T>::to(p[i]) : 0.0f;
  }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, int n, const E e[8]) {
  if (n >= 8) {
    __builtin_memcpy(p, e, 8 * sizeof(E));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
using muon::wave_sum;

// Biased exponent of the scale for a row whose largest magnitude has the
// bits `top` (finite): 127 = 1.984375 * 2^6, so 127 * 2^e >= top needs
// e = E - 6, one more if top's mantissa exceeds 1.984375's.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) {
  const int f = (int)(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)max(f, 1);
}

// MODE 0: quantize x; 1: norm to T; 2: norm to 8 bits.  W waves per row, NC
// chunks per lane.
//
// Norm: the sum of squares is taken in 64 bits and rstd = 1 / sqrt(mean +
// eps) kept there for the 8-bit output, where q = rint(h * (rstd * w /
// scale)) is taken in 64 bits too: a value next to a rounding border then
// rounds as the formula's does, whatever order the row was summed in.  Each
// lane's 64-bit operations (five per element) run at the fp32 rate on this
// part and hide behind the row's loads.
template <typename T, int MODE, bool RES, int W, int NC>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) norm_kernel(const NormParams p) {
  typedef typename Elem<T>::type E;
  constexpr int RPB = W == 1 ? 4 : 1;  // rows per workgroup
  __shared__ double s_sum[W];
  __shared__ uint32_t s_top[W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * RPB + (W == 1 ? wave : 0);
  if (W == 1 && row >= p.rows) return;  // one wave per row: no barrier below
  const int cols = (int)p.cols;
  const int c0 = (W == 1 ? lane : (int)threadIdx.x) * 8;
  constexpr int STEP = 64 * W * 8;

  const E* x = (const E*)p.x + row * p.ldx;
  float v[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
    if (c < cols) {
      load8<T>(x + c, cols - c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
  if constexpr (RES) {
    const E* r = (const E*)p.res + row * p.ldr;
    E* h = (E*)p.h + row * p.ldh;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        float a[8];
        E e[8];
        load8<T>(r + c, cols - c, a);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = Elem<T>::from(v[i][j] + a[j]);
          v[i][j] = Elem<T>::to(e[j]);  // the norm sees the stored stream
        }
        store8(h + c, cols - c, e);
      }
    }
  }
  float w[NC][8];
  if constexpr (MODE != 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) load8<F32>(p.w + c, cols - c, w[i]);
    }
  }

  double sum = 0.0;
  uint32_t top = 0;  // largest |v| (|h w| for MODE 2) as bits: NaN stays on top
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (c0 + i * STEP < cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (MODE != 0) {
          const double d = (double)v[i][j];
          sum = __builtin_fma(d, d, sum);
        }
        if constexpr (MODE == 0) top = max(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
        if constexpr (MODE == 2) top = max(top, __float_as_uint(v[i][j] * w[i][j]) & 0x7fffffffu);
      }
    }
  }
  if constexpr (MODE != 0) sum = wave_sum(sum);
  if constexpr (MODE != 1) top = wave_max(top);
  if constexpr (W > 1) {
    if (lane == 0) {
      s_sum[wave] = sum;
      s_top[wave] = top;
    }
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      sum += s_sum[k];
      top = max(top, s_top[k]);
    }
  }

  double rstd = 1.0;
  if constexpr (MODE != 0) {
    rstd = 1.0 / sqrt(sum / (double)cols + p.eps);
    if (threadIdx.x % (64 * W) == 0) p.rstd[row] = (float)rstd;
  }
  if constexpr (MODE == 1) {
    const float r = (float)rstd;
    E* y = (E*)p.y + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        E e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = Elem<T>::from(v[i][j] * r * w[i][j]);
        store8(y + c, cols - c, e);
      }
    }
  } else {
    if constexpr (MODE == 2) top = __float_as_uint((float)((double)__uint_as_float(top) * rstd)) & 0x7fffffffu;
    const bool finite = top < 0x7f800000u;
    const uint32_t f = finite ? scale_field(top) : 127u;
    const float inv = __uint_as_float((254u - f) << 23);  // 2^-e; f <= 249, so never subnormal
    if (threadIdx.x % (64 * W) == 0)
      p.scale[row] = finite ? __uint_as_float(f << 23) : __uint_as_float(0x7fc00000u);
    const double k = rstd * (double)inv;
    int8_t* q = p.q + row * p.ldq;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        int8_t e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          int n;
          if constexpr (MODE == 2) n = (int)rint((double)v[i][j] * ((double)w[i][j] * k));
          else n = (int)rintf(v[i][j] * inv);
          e[j] = finite ? (int8_t)n : (int8_t)0;
        }
        store8(q + c, cols - c, e);
      }
    }
  }
}

// Backward of y = h * rstd * w (rstd from h):
//   g = dy * w, hat = h * rstd, dx = rstd (g - hat * mean(g hat)) + dh,
//   dw = sum over rows of dy * hat.
// A workgroup of W waves takes rows blockIdx, blockIdx + groups, ...; a
// thread keeps its columns of w and the running dw in registers over all of
// them and writes one row of partial sums at the end, added up in a fixed
// order by norm_back_sum_kernel (no atomics: the result does not depend on
// timing).  The next row's loads are issued before the current row's
// reduction, so they are in flight across its barrier.
template <typename T, typename TH, int W, int NC>
__global__ void __launch_bounds__(64 * W) norm_back_kernel(const NormBackParams p) {
  typedef typename Elem<T>::type E;
  typedef typename Elem<TH>::type EH;
  __shared__ float s_dot[2][W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = (int)p.cols;
  const int c0 = threadIdx.x * 8;
  constexpr int STEP = 64 * W * 8;
  const float inv_cols = 1.0f / (float)cols;

  float w[NC][8], dw[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = dw[i][j] = 0.0f;
    if (c < cols) load8<F32>(p.w + c, cols - c, w[i]);
  }

  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.groups, flip ^= 1) {
    const float rstd = p.rstd[row];
    float hs = rstd;  // hat = h * hs
    if constexpr (sizeof(EH) == 1) hs = p.hscale[row];
    const E* dyr = (const E*)p.dy + row * p.lddy;
    const EH* hr = (const EH*)p.h + row * p.ldh;
    float dy[NC][8], hat[NC][8], dh[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
#pragma unroll
      for (int j = 0; j < 8; ++j) dy[i][j] = hat[i][j] = dh[i][j] = 0.0f;
      if (c < cols) {
        load8<T>(dyr + c, cols - c, dy[i]);
        load8<TH>(hr + c, cols - c, hat[i]);
        if (p.dh) load8<T>((const E*)p.dh + row * p.lddh + c, cols - c, dh[i]);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hat[i][j] *= hs;
        if constexpr (sizeof(EH) == 1) hat[i][j] *= rstd;
        dw[i][j] = __builtin_fmaf(dy[i][j], hat[i][j], dw[i][j]);
        dy[i][j] *= w[i][j];
        dot = __builtin_fmaf(dy[i][j], hat[i][j], dot);
      }
    }
    dot = wave_sum(dot);
    if constexpr (W > 1) {
      if (lane == 0) s_dot[flip][wave] = dot;
      __syncthreads();  // one per row: the next row writes the other half
      dot = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) dot += s_dot[flip][k];
    }
    dot *= inv_cols;
    E* dxr = (E*)p.dx + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        E e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          e[j] = Elem<T>::from(__builtin_fmaf(rstd, __builtin_fmaf(-hat[i][j], dot, dy[i][j]), dh[i][j]));
        store8(dxr + c, cols - c, e);
      }
    }
  }
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
    if (c < cols) store8(part + c, cols - c, dw[i]);
  }
}

// dw[c] = sum over groups of part[g][c]: 16 lanes of columns x 64 strands of
// groups, each strand in order, then the strands pairwise.
__global__ void __launch_bounds__(1024) norm_back_sum_kernel(const float* part, float* dw, int groups,
                                                             int64_t cols) {
  __shared__ float s[64][17];
  const int cl = threadIdx.x & 15, g0 = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + cl;
  float a = 0.0f;
  if (c < cols)
    for (int g = g0; g < groups; g += 64) a += part[(int64_t)g * cols + c];
  s[g0][cl] = a;
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (g0 < o) s[g0][cl] += s[g0 + o][cl];
    __syncthreads();
  }
  if (g0 == 0 && c < cols) dw[c] = s[0][cl];
}

// x = q * scale, 8 columns per thread; blockIdx.y strides over the rows.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const int8_t* q, int64_t ldq, const float* scale,
                                                         void* x, int64_t ldx, int64_t rows, int64_t cols) {
  typedef typename Elem<T>::type E;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= cols) return;
  const int n = (int)min((int64_t)8, cols - c);
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    float v[8];
    E e[8];
    load8<I8>(q + r * ldq + c, n, v);
    const float s = scale[r];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = Elem<T>::from(v[j] * s);
    store8((E*)x + r * ldx + c, n, e);
  }
}

template <typename T, int MODE, bool RES, int W, int NC>
hipError_t go_norm(const NormParams& p, hipStream_t s) {
  const int64_t blocks = W == 1 ? (p.rows + 3) / 4 : p.rows;
  hipLaunchKernelGGL((norm_kernel<T, MODE, RES, W, NC>), dim3((uint32_t)blocks),
                     dim3(W == 1 ? 256 : 64 * W), 0, s, p);
  return hipGetLastError();
}

// Waves and chunks per lane by width: the narrowest that hold the row.
template <typename T, int MODE, bool RES>
hipError_t pick_norm(const NormParams& p, hipStream_t s) {
  const int64_t d = p.cols;
  if (d <= 512) return go_norm<T, MODE, RES, 1, 1>(p, s);
  if (d <= 1024) return go_norm<T, MODE, RES, 1, 2>(p, s);
  if (d <= 2048) return go_norm<T, MODE, RES, 4, 1>(p, s);
  if (d <= 4096) return go_norm<T, MODE, RES, 4, 2>(p, s);
  if (d <= 8192) return go_norm<T, MODE, RES, 4, 4>(p, s);
  if (d <= 16384) return go_norm<T, MODE, RES, 16, 2>(p, s);
  return go_norm<T, MODE, RES, 16, 4>(p, s);
}

template <typename T>
hipError_t pick_norm_mode(const NormParams& p, hipStream_t s) {
  if (p.q) return p.res ? pick_norm<T, 2, true>(p, s) : pick_norm<T, 2, false>(p, s);
  return p.res ? pick_norm<T, 1, true>(p, s) : pick_norm<T, 1, false>(p, s);
}

template <typename T, typename TH, int W, int NC>
hipError_t go_back(const NormBackParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_back_kernel<T, TH, W, NC>), dim3((uint32_t)p.groups), dim3(64 * W), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename TH>
hipError_t pick_back(const NormBackParams& p, hipStream_t s) {
  const int64_t d = p.cols;
  if (d <= 512) return go_back<T, TH, 1, 1>(p, s);
  if (d <= 2048) return go_back<T, TH, 4, 1>(p, s);
  if (d <= 4096) return go_back<T, TH, 4, 2>(p, s);
  if (d <= 8192) return go_back<T, TH, 16, 1>(p, s);
  if (d <= 16384) return go_back<T, TH, 16, 2>(p, s);
  return go_back<T, TH, 16, 4>(p, s);
}

}  // namespace

hipError_t launch_norm(const NormParams& p, bool bf16, hipStream_t s) {
  return bf16 ? pick_norm_mode<BF16>(p, s) : pick_norm_mode<F32>(p, s);
}

// Workgroups of the backward pass: enough to fill the chip, few enough that
// the partial dw rows stay small beside the rows themselves.
int norm_back_groups(int64_t rows, int64_t cols) {
  const int64_t full = cols <= 512 ? 4096 : cols <= 4096 ? 768 : 512;
  return (int)(rows < full ? rows : full);
}

hipError_t launch_norm_back(const NormBackParams& p, bool bf16, hipStream_t s) {
  if (bf16) return p.hscale ? pick_back<BF16, I8>(p, s) : pick_back<BF16, BF16>(p, s);
  return p.hscale ? pick_back<F32, I8>(p, s) : pick_back<F32, F32>(p, s);
}

hipError_t launch_norm_back_sum(const float* part, float* dw, int groups, int64_t cols, hipStream_t s) {
  hipLaunchKernelGGL(norm_back_sum_kernel, dim3((uint32_t)((cols + 15) / 16)), dim3(1024), 0, s, part, dw,
                     groups, cols);
  return hipGetLastError();
}

hipError_t launch_quantize(const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                           int64_t rows, int64_t cols, bool bf16, hipStream_t s) {
  NormParams p = {};
  p.x = x;
  p.ldx = ldx;
  p.q = q;
  p.ldq = ldq;
  p.scale = scale;
  p.rows = rows;
  p.cols = cols;
  return bf16 ? pick_norm<BF16, 0, false>(p, s) : pick_norm<F32, 0, false>(p, s);
}

hipError_t launch_dequantize(const int8_t* q, int64_t ldq, const float* scale, void* x, int64_t ldx,
                             int64_t rows, int64_t cols, bool bf16, hipStream_t s) {
  const dim3 grid((uint32_t)((cols + 2047) / 2048), (uint32_t)(rows < 32768 ? rows : 32768));
  if (bf16)
    hipLaunchKernelGGL(dequantize_kernel<BF16>, grid, dim3(256), 0, s, q, ldq, scale, x, ldx, rows, cols);
  else
    hipLaunchKernelGGL(dequantize_kernel<F32>, grid, dim3(256), 0, s, q, ldq, scale, x, ldx, rows, cols);
  return hipGetLastError();
}

}  // namespace l8
}  // namespace muon
