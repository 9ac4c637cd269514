// Row-wise kernels of the 8-bit linear layer: root-mean-square norm (with
// the residual's addition and an 8-bit output), its backward pass, and the
// 8-bit form of a row and back.
//
// Every kernel is bound by HBM: a row is read once, held in registers, and
// written once.  A row belongs to 8 to 64 lanes of a wave up to 1024 columns (no
// barrier), to 2, 4 or 16 waves above; each lane holds NC chunks of 8
// consecutive columns (16 bytes of bf16).  Rows need no alignment: gfx950 takes 16-byte global
// accesses at any address of the element's own alignment (measured: 6.1 TB/s
// off 16 bytes against 6.7 for a bare copy), and the ragged last chunk of a
// row is read whole from where it fits and written element by element.
//
// The 8-bit form of a row v is scale = 2^e with the smallest e >= -126 for
// which max|v| <= 127 * 2^e, and q = rint(v / scale).  A power of two makes
// the division and the restored value q * scale exact, so rint is the only
// rounding (at most scale / 2), and lets the gradient products fold the scale
// into a bf16 operand without rounding.
#include <algorithm>

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

// Eight consecutive elements as they lie in memory.
template <typename T> struct Chunk { typename Elem<T>::type e[8]; };

// The chunk at column c of a row of `cols`.  A chunk that the row's end cuts is
// read whole from where it still fits, and one past the end as well (in
// flight like any other; predicated element reads cost a latency each), and
// mend8 puts it in place when it is used.  Rows under 8 columns go element by
// element.  Non-temporal where a row is read once per step: it keeps the
// stream from displacing what the next kernel reads.
template <typename T, bool NT = false>
__device__ __forceinline__ void fetch8(const typename Elem<T>::type* row, int c, int cols, Chunk<T>& k) {
  typedef typename Elem<T>::type E;
  if (cols >= 8) {
    const E* p = row + min(c, cols - 8);
    if constexpr (NT && sizeof(E) > 1) {
      typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
      constexpr int NV = 8 * sizeof(E) / 16;
      V v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = __builtin_nontemporal_load((const V*)p + i);
      __builtin_memcpy(k.e, v, sizeof(k.e));
    } else {
      __builtin_memcpy(k.e, p, sizeof(k.e));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) k.e[i] = c + i < cols ? row[c + i] : (E)0;
  }
}
// Elements c .. cols - 1 first, zeros behind them.
template <typename T>
__device__ __forceinline__ void mend8(Chunk<T>& k, int c, int cols) {
  typedef typename Elem<T>::type E;
  const int d = c + 8 - cols;  // elements that it was moved back by
  if (d <= 0 || cols < 8) return;
  if constexpr (sizeof(E) == 4) {
    E e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = d & 4 ? (i < 4 ? k.e[i + 4] : 0.0f) : k.e[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = d & 2 ? (i < 6 ? e[i + 2] : 0.0f) : e[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = d & 1 ? (i < 7 ? e[i + 1] : 0.0f) : e[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) k.e[i] = d >= 8 ? 0.0f : e[i];
  } else if constexpr (sizeof(E) == 2) {
    uint64_t w[2];
    __builtin_memcpy(w, k.e, 16);
    const int sh = (d & 3) * 16;
    w[0] = d & 4 ? w[1] : w[0];
    w[1] = d & 4 ? 0 : w[1];
    w[0] = sh ? (w[0] >> sh) | (w[1] << (64 - sh)) : w[0];
    w[1] >>= sh;
    if (d >= 8) w[0] = w[1] = 0;
    __builtin_memcpy(k.e, w, 16);
  } else {
    uint64_t w;
    __builtin_memcpy(&w, k.e, 8);
    w = d >= 8 ? 0 : w >> (d * 8);
    __builtin_memcpy(k.e, &w, 8);
  }
}
// (widens a chunk in place in its row)
template <typename T>
__device__ __forceinline__ void widen8(Chunk<T>& k, int c, int cols, float v[8]) {
  mend8<T>(k, c, cols);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = Elem<T>::to(k.e[i]);
}
template <typename T>
__device__ __forceinline__ void load8(const typename Elem<T>::type* row, int c, int cols, float v[8]) {
  Chunk<T> k;
  fetch8<T>(row, c, cols, k);
  widen8<T>(k, c, cols, v);
}

template <bool NT = false, typename E>
__device__ __forceinline__ void store8(E* p, int n, const E e[8]) {
  if (n >= 8) {
    if constexpr (NT && sizeof(E) > 1) {
      typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
      constexpr int NV = 8 * sizeof(E) / 16;
      V v[NV];
      __builtin_memcpy(v, e, 8 * sizeof(E));
#pragma unroll
      for (int i = 0; i < NV; ++i) __builtin_nontemporal_store(v[i], (V*)p + i);
    } else {
      __builtin_memcpy(p, e, 8 * sizeof(E));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
}

// Over aligned groups of L lanes of a wave.
template <int L, typename V>
__device__ __forceinline__ V lanes_max(V v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v = max(v, __shfl_xor(v, off, 64));
  return v;
}
template <int L, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// How a row lies on a workgroup: LPR lanes per row (a power of two), RPB rows
// side by side, NT threads.  Up to 64 lanes a row needs no barrier; above, a
// workgroup has one row.
template <int LPR>
struct Rows {
  static constexpr int NT = LPR <= 64 ? 256 : LPR;
  static constexpr int RPB = NT / LPR;
  static constexpr int L = LPR < 64 ? LPR : 64;  // its lanes in one wave
  static constexpr int W = LPR / 64;             // its waves, if whole ones
  static constexpr bool JOIN = W > 1;
};

// Magnitudes as bits, whose order is theirs, with infinity and NaN on top: a
// row's values in 32 bits, products of two of them in 64, where they are exact.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint64_t magnitude(double v) {
  return (uint64_t)__double_as_longlong(v) & 0x7fffffffffffffffull;
}

// Biased exponent of the scale for a row whose largest magnitude has the
// bits `top` (finite): 127 = 1.984375 * 2^6, so 127 * 2^e >= top needs
// e = E - 6, one more if top's mantissa exceeds 1.984375's.
__device__ __forceinline__ uint32_t scale_field(uint32_t top) {
  const int f = (int)(top >> 23) - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)max(f, 1);
}
__device__ __forceinline__ uint32_t scale_field(uint64_t top) {
  const int f = (int)(top >> 52) - (1023 - 127) - 6 + ((top & 0xfffffffffffffull) > 0xfc00000000000ull ? 1 : 0);
  return (uint32_t)max(f, 1);
}

// Whether y = top * rstd, top a row's largest |h w| as rounded in fp32, may
// have another scale than the unrounded one: where top is under 2^-120 (its
// rounding may be of any size), where y comes near fp32's end (infinities and
// NaN among them), and within 2^-22 of 127 * 2^e (rounding moves y by 2^-24).
__device__ __forceinline__ bool in_doubt(uint32_t top, double y) {
  const int64_t from = (int64_t)(magnitude(y) & 0xfffffffffffffull) - 0xfc00000000000ll;
  return top < 7u << 23 || !(y < 0x1p127) || (from < 1ll << 31 && from > -(1ll << 31));
}

// MODE 0: quantize x; 1: norm to T; 2: norm to 8 bits.  LPR lanes per row, NC
// chunks per lane.
//
// Norm: the sum of squares is taken in 64 bits and rstd = 1 / sqrt(mean +
// eps) kept there for the 8-bit output, where q = rint(h * (rstd * w /
// scale)) is taken in 64 bits too: a value next to a rounding border then
// rounds as the formula's does, whatever order the row was summed in.  Each
// lane's 64-bit operations (five per element) run at the fp32 rate on this
// part and hide behind the row's loads.  The scale follows from the largest
// |h w|, found in fp32, where that leaves no doubt (`in_doubt`); rows where it
// does find it again in 64 bits (doing so for every row took 8192 x 3584 bf16,
// no residual, from 28.0 to 32.5 us, 1500 x 18944 from 37.8 to 44.4).
template <typename T, int MODE, bool RES, int LPR, int NC>
__global__ void __launch_bounds__(Rows<LPR>::NT) norm_kernel(const NormParams p) {
  typedef typename Elem<T>::type E;
  typedef Rows<LPR> RW;
  constexpr int W = RW::JOIN ? RW::W : 1;
  __shared__ double s_sum[W];
  __shared__ uint32_t s_top[W];
  __shared__ uint64_t s_exact[W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, at = threadIdx.x % LPR;
  const int64_t row = p.row0 + (int64_t)blockIdx.x * RW::RPB + threadIdx.x / LPR;
  if (row >= p.rows) return;  // RPB > 1 only, which has no barrier below
  const int cols = (int)p.cols;
  const int c0 = at * 8;
  constexpr int STEP = LPR * 8;

  // every load of the row is in flight before the first one is used
  const E* x = (const E*)p.x + row * p.ldx;
  const E* res = RES ? (const E*)p.res + row * p.ldr : nullptr;
  Chunk<T> cx[NC], cr[NC];
  // the widest rows (16 x 4 chunks, 128 registers per lane) read the weights
  // again from the caches where they are used
  constexpr bool KEEPW = LPR * NC < 4096;
  Chunk<F32> cw[KEEPW ? NC : 1];
  float v[NC][8];
  auto weights = [&](int i, float w[8]) {
    if constexpr (KEEPW) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = cw[i].e[j];
    } else {
      load8<F32>(p.w, c0 + i * STEP, cols, w);
    }
  };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
    fetch8<T, true>(x, c, cols, cx[i]);
    if constexpr (RES) fetch8<T, true>(res, c, cols, cr[i]);
  }
  if constexpr (MODE != 0 && KEEPW) {
#pragma unroll
    for (int i = 0; i < NC; ++i) fetch8<F32>(p.w, c0 + i * STEP, cols, cw[i]);
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
    widen8<T>(cx[i], c, cols, v[i]);
    if constexpr (RES) {
      float a[8];
      E e[8];
      widen8<T>(cr[i], c, cols, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = Elem<T>::from(v[i][j] + a[j]);
        v[i][j] = Elem<T>::to(e[j]);  // the norm sees the stored stream
      }
      store8<true>((E*)p.h + row * p.ldh + c, cols - c, e);
    }
    if constexpr (MODE != 0 && KEEPW) mend8<F32>(cw[i], c, cols);
  }

  double sum = 0.0;
  uint32_t top = 0;  // largest |v| (|h w| for MODE 2)
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (c0 + i * STEP < cols) {
      float w[8];
      if constexpr (MODE == 2) weights(i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (MODE != 0) {
          const double d = (double)v[i][j];
          sum = __builtin_fma(d, d, sum);
        }
        if constexpr (MODE == 0) top = max(top, magnitude(v[i][j]));
        if constexpr (MODE == 2) top = max(top, magnitude(v[i][j] * w[j]));
      }
    }
  }
  if constexpr (MODE != 0) sum = lanes_sum<RW::L>(sum);
  if constexpr (MODE != 1) top = lanes_max<RW::L>(top);
  if constexpr (RW::JOIN) {
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
    if (at == 0) p.rstd[row] = (float)rstd;
  }
  if constexpr (MODE == 1) {
    // (outside fp32's normal numbers r loses what y needs: all 64 bits there)
    const float r = (float)rstd;
    const bool normal = magnitude(r) >= 1u << 23 && magnitude(r) < 0x7f800000u;
    E* y = (E*)p.y + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        E e[8];
        float w[8];
        weights(i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = Elem<T>::from(v[i][j] * r * w[j]);
        if (!normal) {
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = Elem<T>::from((float)((double)v[i][j] * rstd * (double)w[j]));
        }
        store8<true>(y + c, cols - c, e);
      }
    }
  } else {
    bool finite = top < 0x7f800000u;
    uint32_t f = scale_field(top);
    if constexpr (MODE == 2) {
      double y = (double)__uint_as_float(top) * rstd;
      if (in_doubt(top, y)) {  // the whole row's lanes
        uint64_t exact = 0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (c0 + i * STEP < cols) {
            float w[8];
            weights(i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) exact = max(exact, magnitude((double)v[i][j] * (double)w[j]));
          }
        }
        exact = lanes_max<RW::L>(exact);
        if constexpr (RW::JOIN) {
          if (lane == 0) s_exact[wave] = exact;
          __syncthreads();
#pragma unroll
          for (int k = 0; k < W; ++k) exact = max(exact, s_exact[k]);
        }
        y = __longlong_as_double((long long)exact) * rstd;
      }
      finite = magnitude((float)y) < 0x7f800000u;
      f = scale_field(magnitude(y));
    }
    f = finite ? f : 127u;
    const float inv = __uint_as_float((254u - f) << 23);  // 2^-e; f <= 249, so never subnormal
    if (at == 0)
      p.scale[row] = finite ? __uint_as_float(f << 23) : __uint_as_float(0x7fc00000u);
    const double k = rstd * (double)inv;
    int8_t* q = p.q + row * p.ldq;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        int8_t e[8];
        float w[8];
        if constexpr (MODE == 2) weights(i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          int n;
          if constexpr (MODE == 2) n = (int)rint((double)v[i][j] * ((double)w[j] * k));
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
// Of the groups of RPB rows, a workgroup takes every p.groups-th; a thread
// keeps its columns of w and the running dw in registers over all of them,
// the workgroup writes one row of partial sums at the end, and
// norm_back_sum_kernel adds those up in a fixed order (no atomics: the result
// does not depend on timing).  The next row's loads are issued before the
// current row's reduction, so they are in flight across its barrier.
//
// Rows over 8192 columns (16 waves, 128 registers per lane): the running dw
// lies in LDS, the weights come from the caches, nothing is fetched ahead, and
// the row stays in its storage type, widened again for the second pass.  Over
// 16384 columns it does not fit even so, and the second pass reads it again
// (from L2: one row per compute unit, 3 MB per XCD).
template <typename T, typename TH, int LPR, int NC>
__global__ void __launch_bounds__(Rows<LPR>::NT) norm_back_kernel(const NormBackParams p) {
  typedef typename Elem<T>::type E;
  typedef typename Elem<TH>::type EH;
  typedef Rows<LPR> RW;
  constexpr bool WIDE = LPR * NC > 1024;
  constexpr bool AGAIN = LPR * NC > 2048;
  constexpr int W = RW::JOIN ? RW::W : 1;
  __shared__ float s_dot[2][W];
  __shared__ float4 s_dw[WIDE || RW::RPB > 1 ? NC * 2 * RW::NT : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = (int)p.cols;
  const int c0 = (threadIdx.x % LPR) * 8;
  constexpr int STEP = LPR * 8;
  const float inv_cols = 1.0f / (float)cols;

  float wk[WIDE ? 1 : NC][8], dwk[WIDE ? 1 : NC][8];
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i) s_dw[i * LPR + threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      load8<F32>(p.w, c0 + i * STEP, cols, wk[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) dwk[i][j] = 0.0f;
    }
  }

  constexpr int KEPT = AGAIN ? 1 : NC;  // chunks of the row in registers
  Chunk<T> cdy[KEPT], cdh[KEPT];
  Chunk<TH> ch[KEPT];
  auto fetch_one = [&](int64_t row, int i) {
    const E* dyr = (const E*)p.dy + row * p.lddy;
    const EH* hr = (const EH*)p.h + row * p.ldh;
    const E* dhr = (const E*)p.dh + row * p.lddh;
    const int c = c0 + i * STEP, k = AGAIN ? 0 : i;
    fetch8<T, !AGAIN>(dyr, c, cols, cdy[k]);
    fetch8<TH, !AGAIN>(hr, c, cols, ch[k]);
    if (p.dh) fetch8<T, !AGAIN>(dhr, c, cols, cdh[k]);
  };
  auto fetch = [&](int64_t row) {
    if constexpr (!AGAIN) {
#pragma unroll
      for (int i = 0; i < NC; ++i) fetch_one(row, i);
    }
  };
  const int64_t first = (int64_t)blockIdx.x * RW::RPB + threadIdx.x / LPR, stride = (int64_t)p.groups * RW::RPB;
  if (!WIDE && first < p.rows) fetch(first);
  int flip = 0;
  for (int64_t row = first; row < p.rows; row += stride, flip ^= 1) {
    if constexpr (WIDE) fetch(row);
    const float rstd = p.rstd[row];
    float hs = rstd;  // hat = h * hs
    if constexpr (sizeof(EH) == 1) hs = p.hscale[row];
    // g and hat of chunk i
    auto terms = [&](int i, const float w[8], float dy[8], float g[8], float hat[8]) {
      Chunk<T> k = cdy[AGAIN ? 0 : i];  // (copies: the wide rows widen theirs twice)
      Chunk<TH> kh = ch[AGAIN ? 0 : i];
      widen8<T>(k, c0 + i * STEP, cols, dy);
      widen8<TH>(kh, c0 + i * STEP, cols, hat);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hat[j] *= hs;
        if constexpr (sizeof(EH) == 1) hat[j] *= rstd;
        g[j] = dy[j] * w[j];
      }
    };
    float g[WIDE ? 1 : NC][8], hat[WIDE ? 1 : NC][8];
    Chunk<T> cadd[WIDE ? 1 : NC];
    float dot = 0.0f;
#pragma unroll AGAIN ? 1 : NC
    for (int i = 0; i < NC; ++i) {
      if constexpr (AGAIN) fetch_one(row, i);
      float dy[8];
      float *gi = g[WIDE ? 0 : i], *hi = hat[WIDE ? 0 : i];
      if constexpr (WIDE) {
        float w[8], dw[8];
        float4* l = s_dw + 2 * i * LPR + threadIdx.x;
        load8<F32>(p.w, c0 + i * STEP, cols, w);
        terms(i, w, dy, gi, hi);
        __builtin_memcpy(dw, l, 16);
        __builtin_memcpy(dw + 4, l + LPR, 16);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = __builtin_fmaf(dy[j], hi[j], dw[j]);
        __builtin_memcpy(l, dw, 16);
        __builtin_memcpy(l + LPR, dw + 4, 16);
      } else {
        terms(i, wk[i], dy, gi, hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) dwk[i][j] = __builtin_fmaf(dy[j], hi[j], dwk[i][j]);
        cadd[i] = cdh[i];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(gi[j], hi[j], dot);
    }
    if (!WIDE && row + stride < p.rows) fetch(row + stride);
    dot = lanes_sum<RW::L>(dot);
    if constexpr (RW::JOIN) {
      if (lane == 0) s_dot[flip][wave] = dot;
      __syncthreads();  // one per row: the next row writes the other half
      dot = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) dot += s_dot[flip][k];
    }
    dot *= inv_cols;
    E* dxr = (E*)p.dx + row * p.lddx;
#pragma unroll AGAIN ? 1 : NC
    for (int i = 0; i < NC; ++i) {
      const int c = c0 + i * STEP;
      if (c < cols) {
        if constexpr (AGAIN) fetch_one(row, i);
        E e[8];
        float dh[8];
        float *gi = g[WIDE ? 0 : i], *hi = hat[WIDE ? 0 : i];
        if constexpr (WIDE) {
          float w[8], dy[8];
          load8<F32>(p.w, c, cols, w);
          terms(i, w, dy, gi, hi);
        }
        if (p.dh) {
          widen8<T>(WIDE ? cdh[AGAIN ? 0 : i] : cadd[WIDE ? 0 : i], c, cols, dh);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) dh[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          e[j] = Elem<T>::from(__builtin_fmaf(rstd, __builtin_fmaf(-hi[j], dot, gi[j]), dh[j]));
        store8<true>(dxr + c, cols - c, e);
      }
    }
  }

  // one row of partial sums per workgroup
  float* part = p.part + (int64_t)blockIdx.x * p.cols;
  if constexpr (RW::RPB > 1) {  // NC = 1 or 2, LPR <= 64: join the rows' sums
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      __builtin_memcpy(s_dw + 2 * (i * RW::NT + threadIdx.x), dwk[i], 32);
    }
    __syncthreads();
    if (threadIdx.x < LPR) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        for (int r = 1; r < RW::RPB; ++r) {
          float o[8];
          __builtin_memcpy(o, s_dw + 2 * (i * RW::NT + r * LPR + threadIdx.x), 32);
#pragma unroll
          for (int j = 0; j < 8; ++j) dwk[i][j] += o[j];
        }
      }
    }
    if (threadIdx.x >= LPR) return;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = c0 + i * STEP;
    float dw[8];
    if constexpr (WIDE) {
      __builtin_memcpy(dw, s_dw + 2 * i * LPR + threadIdx.x, 16);
      __builtin_memcpy(dw + 4, s_dw + (2 * i + 1) * LPR + threadIdx.x, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[j] = dwk[i][j];
    }
    if (c < cols) store8(part + c, cols - c, dw);
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
    for (int g = g0; g < groups; g += 256) {  // four reads in flight
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = part[(int64_t)min(g + 64 * u, groups - 1) * cols + c];
#pragma unroll
      for (int u = 0; u < 4; ++u) a += g + 64 * u < groups ? v[u] : 0.0f;
    }
  s[g0][cl] = a;
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    if (g0 < o) s[g0][cl] += s[g0 + o][cl];
    __syncthreads();
  }
  if (g0 == 0 && c < cols) dw[c] = s[0][cl];
}

// x = q * scale.  The matrix is cut into chunks of 16 stored bytes (8 bf16 or 4
// fp32 columns), one per thread, from chunk `first` on.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const int8_t* q, int64_t ldq, const float* scale,
                                                         typename Elem<T>::type* x, int64_t ldx, int64_t rows,
                                                         int cols, int64_t first) {
  typedef typename Elem<T>::type E;
  constexpr int C = 16 / sizeof(E);
  const uint32_t cpr = (uint32_t)(cols + C - 1) / C;
  const int64_t id = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id >> 32 ? id / cpr : (int64_t)((uint32_t)id / cpr);
  if (row >= rows) return;
  const int col = (int)(id - row * cpr) * C, n = cols - col;
  const int8_t* a = q + row * ldq + col;
  E* o = x + row * ldx + col;
  const float s = scale[row];
  if (n >= C) {
    int8_t v[C];
    E e[C];
    __builtin_memcpy(v, a, C);
#pragma unroll
    for (int j = 0; j < C; ++j) e[j] = Elem<T>::from((float)v[j] * s);
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    V w;
    __builtin_memcpy(&w, e, 16);
    __builtin_nontemporal_store(w, (V*)o);
  } else {
    for (int j = 0; j < n; ++j) o[j] = Elem<T>::from((float)a[j] * s);
  }
}

// Calls launch(first block, blocks) until all are out.  A launch has fewer than
// 2^32 threads: given more, the runtime drops the upper bits of their number,
// runs what is left and reports no error.
template <typename F>
hipError_t in_launches(int64_t blocks, int threads, F launch) {
  const int64_t most = 0xffffffffll / threads;
  hipError_t e = hipSuccess;
  for (int64_t b = 0; b < blocks && e == hipSuccess; b += most) {
    launch(b, (uint32_t)std::min(blocks - b, most));
    e = hipGetLastError();
  }
  return e;
}

template <typename T, int MODE, bool RES, int LPR, int NC>
hipError_t go_norm(NormParams p, hipStream_t s) {
  typedef Rows<LPR> RW;
  return in_launches((p.rows + RW::RPB - 1) / RW::RPB, RW::NT, [&](int64_t first, uint32_t blocks) {
    p.row0 = first * RW::RPB;
    hipLaunchKernelGGL((norm_kernel<T, MODE, RES, LPR, NC>), dim3(blocks), dim3(RW::NT), 0, s, p);
  });
}

// Lanes and chunks by width: the fewest lanes that hold the row in two chunks
// (four from 4096 columns on).  Measured over 29.4 M elements: with one chunk
// per lane quantize reaches 4.1 TB/s at 512 columns, with two 5.1; at 8192
// four chunks on 4 waves 5.4 TB/s, one on 16 waves 4.1.
template <typename T, int MODE, bool RES>
hipError_t pick_norm(const NormParams& p, hipStream_t s) {
  const int64_t d = p.cols;
  if (d <= 64) return go_norm<T, MODE, RES, 8, 1>(p, s);
  if (d <= 128) return go_norm<T, MODE, RES, 8, 2>(p, s);
  if (d <= 256) return go_norm<T, MODE, RES, 16, 2>(p, s);
  if (d <= 512) return go_norm<T, MODE, RES, 32, 2>(p, s);
  if (d <= 1024) return go_norm<T, MODE, RES, 64, 2>(p, s);
  if (d <= 2048) return go_norm<T, MODE, RES, 128, 2>(p, s);
  if (d <= 4096) return go_norm<T, MODE, RES, 256, 2>(p, s);
  if (d <= 8192) return go_norm<T, MODE, RES, 256, 4>(p, s);
  if (d <= 16384) return go_norm<T, MODE, RES, 512, 4>(p, s);
  return go_norm<T, MODE, RES, 1024, 4>(p, s);
}

template <typename T>
hipError_t pick_norm_mode(const NormParams& p, hipStream_t s) {
  if (p.q) return p.res ? pick_norm<T, 2, true>(p, s) : pick_norm<T, 2, false>(p, s);
  return p.res ? pick_norm<T, 1, true>(p, s) : pick_norm<T, 1, false>(p, s);
}

template <typename T, typename TH, int LPR, int NC>
hipError_t go_back(const NormBackParams& p, hipStream_t s) {
  hipLaunchKernelGGL((norm_back_kernel<T, TH, LPR, NC>), dim3((uint32_t)p.groups), dim3(Rows<LPR>::NT), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename TH>
hipError_t pick_back(const NormBackParams& p, hipStream_t s) {
  const int64_t d = p.cols;
  if (d <= 64) return go_back<T, TH, 8, 1>(p, s);
  if (d <= 128) return go_back<T, TH, 8, 2>(p, s);
  if (d <= 256) return go_back<T, TH, 16, 2>(p, s);
  if (d <= 512) return go_back<T, TH, 32, 2>(p, s);
  if (d <= 1024) return go_back<T, TH, 64, 2>(p, s);
  if (d <= 2048) return go_back<T, TH, 256, 1>(p, s);
  if (d <= 4096) return go_back<T, TH, 256, 2>(p, s);
  if (d <= 8192) return go_back<T, TH, 1024, 1>(p, s);
  if (d <= 16384) return go_back<T, TH, 1024, 2>(p, s);
  return go_back<T, TH, 1024, 4>(p, s);
}

}  // namespace

hipError_t launch_norm(const NormParams& p, bool bf16, hipStream_t s) {
  return bf16 ? pick_norm_mode<BF16>(p, s) : pick_norm_mode<F32>(p, s);
}

// Workgroups of the backward pass: enough to fill the chip, few enough that
// the partial dw rows stay small beside the rows themselves.  Measured over
// 29.4 M bf16 elements (us, sums included) for 256 / 512 / 768 / 1024 groups,
// with dh: 59 / 48 / 47 / 53 at 1024 columns, 64 / 50 / 50 / 60 at 3584, 49 /
// 54 / 60 / 66 at 8192; from 8-bit rows without dh: 52 / 37 / 33 / 41, 59 / 41
// / 37 / 48 and 40 / 45 / 51 / 56.  Fp32 rows (twice the bytes in flight) and
// short batches do better with 512 (f32, 8192 x 3584, dh: 90 against 107; bf16,
// 2048 x 4096: 21 against 24).  Between, rows of over 1024 columns come two or
// four to a workgroup, so that the partial rows stay fewer than the rows (512 x
// 3584: 10.8 us with 256 groups, 13.2 with 512; 1024 x 3584: 13.8 and 15.0).
int norm_back_groups(int64_t rows, int64_t cols, bool bf16) {
  const int64_t side = cols <= 128 ? 32 : cols <= 256 ? 16 : cols <= 512 ? 8 : cols <= 1024 ? 4 : 1;  // RPB
  const int64_t need = (rows + side - 1) / side;
  const int64_t full = cols > 4096 ? 256 : bf16 && need >= 4096 ? 768 : 512;
  if (side > 1 || need <= 128) return (int)std::min(need, full);
  return (int)std::min(full, std::max({(int64_t)128, std::min<int64_t>((need + 1) / 2, 256), (need + 3) / 4}));
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
  const int64_t per = bf16 ? 8 : 4;
  return in_launches((rows * ((cols + per - 1) / per) + 255) / 256, 256, [&](int64_t first, uint32_t blocks) {
    if (bf16)
      hipLaunchKernelGGL(dequantize_kernel<BF16>, dim3(blocks), dim3(256), 0, s, q, ldq, scale, (uint16_t*)x, ldx,
                         rows, (int)cols, first * 256);
    else
      hipLaunchKernelGGL(dequantize_kernel<F32>, dim3(blocks), dim3(256), 0, s, q, ldq, scale, (float*)x, ldx, rows,
                         (int)cols, first * 256);
  });
}

}  // namespace l8
}  // namespace muon
