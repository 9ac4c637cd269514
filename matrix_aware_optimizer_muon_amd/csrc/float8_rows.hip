// The 8-bit floating-point form of rows and of weights, and back.
//
// A block (128 values of a row, or 128 x 128 of a matrix) gets scale = 2^e with
// the smallest e >= -126 for which max|v| <= 448 * 2^e, held as the byte e +
// 127, and q = v / scale in e4m3.  A power of two makes the division and the
// restored value exact, so the conversion's rounding (nearest even, in the
// hardware) is the only one.  448 = 1.75 * 2^8: with max|v| = m * 2^E, e = E - 8,
// one more if m > 1.75, which reads off the bits of the largest magnitude.
//
// Bound by HBM: 18944 x 3584 fp32 weights to 8 bits in 54 us, back in 53, 6.4
// TB/s.  Every value is held in registers between the search for the
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

// 16 bytes of a row's elements, n of which exist, zeros behind; at any alignment
// of the element's own.  (A wave's loads are one run: with eight fp32 values per
// lane, two loads 32 bytes apart, 18944 x 3584 weights took 70 us, not 57.)
template <typename T>
constexpr int kChunk = 16 / sizeof(typename Elem<T>::type);
template <typename T>
__device__ __forceinline__ void load(const typename Elem<T>::type* p, int n, uint32_t v[kChunk<T>]) {
  constexpr int CH = kChunk<T>;
  typename Elem<T>::type e[CH];
  if (n >= CH) {
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    const V w = __builtin_nontemporal_load((const V*)p);
    __builtin_memcpy(e, &w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) e[i] = i < n ? p[i] : (typename Elem<T>::type)0;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) v[i] = Elem<T>::bits(e[i]);
}

template <int CH>
__device__ __forceinline__ uint32_t largest(const uint32_t (&v)[CH]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) top = max(top, v[i] & 0x7fffffffu);
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
// A chunk's values times 1 / scale in e4m3 (2^-e from the byte e + 127 <= 247), n
// of which are written.
template <int CH>
__device__ __forceinline__ void store(uint8_t* q, int n, const uint32_t (&v)[CH], uint32_t byte) {
  const float by = __uint_as_float((254u - byte) << 23);
  uint32_t w[CH / 4];
#pragma unroll
  for (int i = 0; i < CH / 4; ++i) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[4 * i + j]) * by;
    uint32_t d = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    d = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], (int)d, true);
    w[i] = byte == 255u ? 0x7f7f7f7fu : d;
  }
  if (n >= CH) {
    __builtin_memcpy(__builtin_assume_aligned(q, CH), w, CH);  // (rows start at 16 bytes)
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (i < n) q[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// k / d for 32-bit k and d by a multiplication: m = floor(2^64 / d) + 1 is off by
// at most d / 2^64 of a quotient, less than its distance to the next whole one.
// (A 64-bit division is some hundred instructions: they took three quarters of
// a restored matrix's time.)
struct Div {
  uint64_t m;
  uint32_t d;
  Div(int64_t by) : m(by > 1 ? ~0ull / (uint64_t)by + 1 : 0), d((uint32_t)by) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t k) const { return d > 1 ? (uint32_t)__umul64hi(m, k) : k; }
};

// Rows: a block of 128 on 16 (bf16) or 32 lanes, N blocks per lane a step apart,
// all loads in flight before the first use.
template <typename T, int N>
__global__ void __launch_bounds__(256) rows_kernel(const FormParams p, uint32_t blocks, Div kb) {
  constexpr int CH = kChunk<T>, L = kBlock / CH, PER = 256 / L;
  const uint32_t step = gridDim.x * PER, b = blockIdx.x * PER + threadIdx.x / L;
  const int at = threadIdx.x % L * CH;
  uint32_t v[N][CH], row[N];
  int col[N], n[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t k = b + i * step;
    row[i] = kb(k);
    col[i] = (int)(k - row[i] * kb.d) * kBlock + at;
    n[i] = k < blocks ? (int)min((int64_t)CH, p.cols - col[i]) : 0;
    load<T>((const typename Elem<T>::type*)p.x + row[i] * p.ldx + col[i], n[i], v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t k = b + i * step;
    const uint32_t byte = scale_byte(lanes_max<L>(largest(v[i])));
    if (k >= blocks) continue;
    store(p.q + row[i] * p.ldq + col[i], n[i], v[i], byte);
    if (at == 0) p.scale[k] = (uint8_t)byte;
  }
}

// Weights: a workgroup per 128 x 128 values, 64 of them per thread.
template <typename T>
__global__ void __launch_bounds__(256) squares_kernel(const FormParams p, Div per, Div kb) {
  constexpr int CH = kChunk<T>, L = kBlock / CH, ROWS = 256 / L, N = kBlock / ROWS;
  __shared__ uint32_t s_top[4];
  const uint32_t k = blockIdx.x, m = per(k), in = k - m * per.d, rb = kb(in);
  const int c = (int)(in - rb * kb.d) * kBlock + threadIdx.x % L * CH, r0 = (int)rb * kBlock + threadIdx.x / L;
  const int n = (int)min((int64_t)CH, p.cols - c);
  const typename Elem<T>::type* x = (const typename Elem<T>::type*)p.x + m * p.sx + c;
  uint32_t v[N][CH], top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t r = r0 + i * ROWS;
    load<T>(x + r * p.ldx, r < p.rows ? n : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, largest(v[i]));
  top = lanes_max<64>(top);
  if (threadIdx.x % 64 == 0) s_top[threadIdx.x / 64] = top;
  __syncthreads();
  top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
  const uint32_t byte = scale_byte(top);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t r = r0 + i * ROWS;
    if (r < p.rows) store(p.q + m * p.sq + r * p.ldq + c, n, v[i], byte);
  }
  if (threadIdx.x == 0) p.scale[k] = (uint8_t)byte;
}

// Back: 16 bytes of output per thread and step, so that a wave's stores are one
// run (16 values each, four fp32 stores 64 bytes apart, took 313 us instead of
// 57 for 18944 x 3584).
template <typename T, int N>
__global__ void __launch_bounds__(256) back_kernel(const FormParams p, uint32_t chunks, Div cpr, Div rows, int kb, int nb) {
  typedef typename Elem<T>::type E;
  constexpr int CH = 16 / sizeof(E);
  const uint32_t step = gridDim.x * 256, first = blockIdx.x * 256 + threadIdx.x;
  uint32_t v[N][CH / 4], byte[N];
  E* out[N];
  int n[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t k = first + i * step, at = min(k, chunks - 1);
    const uint32_t row = cpr(at), m = rows(row), r = row - m * rows.d;
    const int c = (int)(at - row * cpr.d) * CH;
    n[i] = k < chunks ? (int)min((int64_t)CH, p.cols - c) : 0;
    // (rows start at 16 bytes and may be read to the next 16)
    __builtin_memcpy(v[i], __builtin_assume_aligned(p.q + m * p.sq + r * p.ldq + c, CH), CH);
    byte[i] = p.scale[(p.block_rows == 1 ? (int64_t)row : (int64_t)m * nb + r / kBlock) * kb + c / kBlock];
    out[i] = (E*)p.x + m * p.sx + r * p.ldx + c;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // (2^-127 is no normal number)
    const float f = byte[i] == 255u ? __uint_as_float(0x7fc00000u)
                    : byte[i] == 0u ? __uint_as_float(1u << 22)
                                    : __uint_as_float(byte[i] << 23);
    E e[CH];
#pragma unroll
    for (int j = 0; j < CH / 4; ++j) {
      const f32x4 w = {__builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 0), __builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 1),
                       __builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 2), __builtin_amdgcn_cvt_f32_fp8((int)v[i][j], 3)};
#pragma unroll
      for (int l = 0; l < 4; ++l) e[4 * j + l] = Elem<T>::from(w[l] * f);
    }
    if (n[i] >= CH) {
      typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
      V w;
      __builtin_memcpy(&w, e, 16);
      __builtin_nontemporal_store(w, (V*)out[i]);
    } else {
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (j < n[i]) out[i][j] = e[j];
    }
  }
}

// Calls f(part) for parts of the matrices whose items (`per_row` a row) a launch
// can number and hold: whole matrices where they fit, else rows of one after
// another (a multiple of 128 of them, so that blocks stay whole).
template <typename F>
hipError_t in_parts(const FormParams& p, int64_t per_row, int64_t item, F f) {
  constexpr int64_t kMost = 1ll << 28;
  // (a launch has fewer than 2^32 threads, 256 for a block of 128 rows)
  const int64_t matrix = (p.block_rows == kBlock ? (p.rows + kBlock - 1) / kBlock * kBlock : p.rows) * per_row;
  const int64_t many = std::max<int64_t>(1, kMost / matrix), some = std::max<int64_t>(1, kMost / per_row / kBlock) * kBlock;
  const int kb = (int)((p.cols + kBlock - 1) / kBlock), nb = (int)((p.rows + kBlock - 1) / kBlock);
  for (int64_t m = 0; m < p.count; m += many)
    for (int64_t r = 0; r < p.rows; r += matrix <= kMost ? p.rows : some) {
      FormParams o = p;
      o.count = std::min(many, p.count - m);
      o.rows = matrix <= kMost ? p.rows : std::min(some, p.rows - r);
      o.x = (char*)p.x + (m * p.sx + r * p.ldx) * item;
      o.q = p.q + m * p.sq + r * p.ldq;
      o.scale = p.scale + (p.block_rows == 1 ? m * p.rows + r : m * nb + r / kBlock) * kb;
      const hipError_t e = f(o, kb, (int)((o.rows + kBlock - 1) / kBlock));
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace

hipError_t launch_quantize(const FormParams& p, bool bf16, hipStream_t s) {
  const int64_t kb = (p.cols + kBlock - 1) / kBlock;
  if (p.block_rows == kBlock)
    return in_parts(p, kb, bf16 ? 2 : 4, [&](const FormParams& o, int kb, int nb) {
      const dim3 grid((uint32_t)(o.count * nb * kb));
      if (bf16) hipLaunchKernelGGL((squares_kernel<BF16>), grid, dim3(256), 0, s, o, Div((int64_t)kb * nb), Div(kb));
      else hipLaunchKernelGGL((squares_kernel<F32>), grid, dim3(256), 0, s, o, Div((int64_t)kb * nb), Div(kb));
      return hipGetLastError();
    });
  // (the rows kernel numbers the rows of one matrix)
  for (int64_t m = 0; m < p.count; ++m) {
    FormParams one = p;
    one.count = 1;
    one.x = (char*)p.x + m * p.sx * (bf16 ? 2 : 4);
    one.q = p.q + m * p.sq;
    one.scale = p.scale + m * p.rows * kb;
    const hipError_t e = in_parts(one, kb, bf16 ? 2 : 4, [&](const FormParams& o, int kb, int) {
      const uint32_t blocks = (uint32_t)(o.rows * kb);
      auto go = [&](auto kernel, uint32_t per) {
        hipLaunchKernelGGL(kernel, dim3((blocks + per - 1) / per), dim3(256), 0, s, o, blocks, Div(kb));
        return hipGetLastError();
      };
      if (blocks >= 16 * 4 * 1024) return bf16 ? go(rows_kernel<BF16, 4>, 64) : go(rows_kernel<F32, 4>, 32);
      return bf16 ? go(rows_kernel<BF16, 1>, 16) : go(rows_kernel<F32, 1>, 8);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dequantize(const FormParams& p, bool bf16, hipStream_t s) {
  const int64_t per = bf16 ? 8 : 4, cpr = (p.cols + per - 1) / per;
  return in_parts(p, cpr, bf16 ? 2 : 4, [&](const FormParams& o, int kb, int nb) {
    const uint32_t chunks = (uint32_t)(o.count * o.rows * cpr);
    auto go = [&](auto kernel, uint32_t each) {
      hipLaunchKernelGGL(kernel, dim3((chunks + each - 1) / each), dim3(256), 0, s, o, chunks, Div(cpr), Div(o.rows), kb, nb);
      return hipGetLastError();
    };
    // (several per thread once all threads of the card have one)
    if (chunks >= 256 * 4 * 2048) return bf16 ? go(back_kernel<BF16, 4>, 1024) : go(back_kernel<F32, 4>, 1024);
    return bf16 ? go(back_kernel<BF16, 1>, 256) : go(back_kernel<F32, 1>, 256);
  });
}

}  // namespace f8
}  // namespace muon
