// What the products of the 8-bit layers share (gfx950): the LDS ring's layout,
// operands fed by direct global->LDS loads, fragment reads, and the stores of
// finished rows.
#pragma once

#include "common.hpp"

namespace muon {
namespace l8 {

namespace {

constexpr int KB = 64;        // bytes of K per stage and contiguous row
constexpr int KROWS = 32;     // rows of K per stage of a K-major operand

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_ptr_t;
typedef const __attribute__((address_space(1))) void gbl_ptr_t;

__device__ __attribute__((aligned(64))) const char g_zero[64] = {0};

// s_waitcnt immediate (gfx9 encoding): vmcnt in [3:0] and [15:14], expcnt
// [6:4] left at its maximum, lgkmcnt [11:8].
constexpr int wait_imm(int vm, int lgkm) {
  return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | ((lgkm & 15) << 8);
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

// 16-byte chunk swizzles.  A K-contiguous row has 4 chunks: bit 1 flips with
// row bit 2 (fragment reads of 16 rows x 4 chunks are conflict free).  A
// K-major row has 16 or 32: an even XOR from row bits 0, 1 and 3, so the 16
// rows of 32 bytes that a transposing read takes (bit 2 is fixed) fall on
// eight pair places; with 8 chunks (64 columns) row bit 0 is the upper half
// of the banks already, and bits 1 and 3 make four pair places.
__device__ __forceinline__ int swz_c(int row) { return ((row >> 2) & 1) << 1; }
template <int T>
__device__ __forceinline__ int swz_k(int k) {
  return T == 64 ? ((k >> 1) & 1) << 1 | ((k >> 3) & 1) << 2 : ((k & 3) | (((k >> 3) & 1) << 2)) << 1;
}

__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// One operand of T rows (columns, if K-major) fed by direct global->LDS loads:
// where a lane's instructions read, stage by stage.  In LDS a stage is 64
// bytes per row, or 32 rows of 2 T bytes.  Needs 16-byte aligned rows.
template <bool KM, int T, int NW>
struct DmaOperand {
  static constexpr int NDMA = T * KB / 1024 / NW;  // 1-KB instructions per wave and stage
  const char* src[NDMA];   // stage 0
  const char* tail[NDMA];  // the stage that K's end falls into
  int64_t step;            // bytes from stage to stage

  __device__ __forceinline__ void init(const char* base, int64_t ld, int row0, int count, int kd,
                                       int kbytes, int full, int tid) {
    const int wave = tid >> 6, lane = tid & 63;
    step = KM ? KROWS * ld : (int64_t)KB;
#pragma unroll
    for (int i = 0; i < NDMA; ++i) {
      bool in;
      if constexpr (KM) {
        constexpr int RB = T * 2, RPI = 1024 / RB, CH = RB / 16;
        const int k = (wave * NDMA + i) * RPI + lane / CH;
        const int ch = (lane % CH) ^ swz_k<T>(k);
        const int c = min(row0 + ch * 8, (count - 1) & ~7);  // whole chunks, in the padded row
        in = full * KROWS + k < kd;
        // where there is no whole stage, `src` is never read
        src[i] = base + (int64_t)min(k, kd - 1) * ld + (int64_t)c * 2;
      } else {
        const int r = (wave * NDMA + i) * 16 + (lane >> 2);
        const int ch = (lane & 3) ^ swz_c(r);
        in = full * KB + ch * 16 < kbytes;
        src[i] = base + (int64_t)min(row0 + r, count - 1) * ld + ch * 16;
      }
      tail[i] = in ? src[i] + full * step : g_zero;
    }
  }
  __device__ __forceinline__ void load(int i, char* stage, int ks, int full, int wave) const {
    const char* s = ks < full ? src[i] + ks * step : tail[i];
    // The compiler puts a wait for every earlier DMA before a read of the LDS
    // object that the DMA names (the ring's other stages, which are in use).
    // An address that it cannot follow leaves the waits to this kernel's own
    // vmcnt count and barrier.
    uint32_t to = (uint32_t)(uintptr_t)(lds_ptr_t*)(stage + (wave * NDMA + i) * 1024);
    asm("" : "+s"(to));
    __builtin_amdgcn_global_load_lds((gbl_ptr_t*)s, (lds_ptr_t*)(uintptr_t)to, 16, 0, 0);
  }
};

// The first n bytes wanted of a 16-byte read (8 bytes: the low half) that was
// moved back by d bytes to stay inside its matrix, zeros beyond (none: n <= 0).
__device__ __forceinline__ u32x4 put_in_place(u32x4 v, int d, int n) {
  uint64_t w0 = (uint64_t)v[1] << 32 | v[0], w1 = (uint64_t)v[3] << 32 | v[2];
  const int sh = (d & 7) * 8;
  w0 = d & 8 ? w1 : w0;
  w1 = d & 8 ? 0 : w1;
  w0 = sh ? (w0 >> sh) | (w1 << (64 - sh)) : w0;
  w1 >>= sh;
  const uint64_t m = (1ull << ((n & 7) * 8)) - 1;  // the cut half's bytes
  w0 &= n >= 8 ? ~0ull : n > 0 ? m : 0ull;
  w1 &= n >= 16 ? ~0ull : n > 8 ? m : 0ull;
  return u32x4{(uint32_t)w0, (uint32_t)(w0 >> 32), (uint32_t)w1, (uint32_t)(w1 >> 32)};
}
// last: the last place of the matrix where 16 bytes can be read.
__device__ __forceinline__ u32x4 load_part(const char* a, int n, const char* last) {
  const char* at = a < last ? a : last;
  u32x4 v;
  __builtin_memcpy(&v, at, 16);
  return put_in_place(v, (int)(a - at) & 15, n);  // (over 15 only where n <= 0)
}

// Fragment f (16 rows) of a wave's part of an operand stage.
template <bool KM, int T>
struct Reader {
  int off, sw, col;
  __device__ __forceinline__ void init(int ring, int first, int q4, int c16) {
    if constexpr (KM) {
      // two transposing reads, k 8 q4 .. +3 and +4 .. +7 (swz_k equal: bit 2
      // does not enter it); the lane addresses row 8 q4 + c16 / 4 (+ 4) and
      // columns first + 16 f + 4 (c16 % 4) .. +3
      const int k = 8 * q4 + (c16 >> 2);
      off = k * T * 2 + ((c16 & 3) >> 1) * 16 + (c16 & 1) * 8;
      sw = swz_k<T>(k) << 4;
      col = first >> 3;
    } else {
      const int r = first + c16;
      off = r * KB + ((q4 ^ swz_c(r)) << 4);
    }
    off += ring;
    asm("" : "+v"(off));  // (see get: keeps `ring` from becoming a base of its own)
  }
  // (one addition to the LDS object's address: through a longer chain the
  // compiler loses which object is read, and waits for every DMA)
  __device__ __forceinline__ u32x4 get(const char* lds, int stage, int f) const {
    if constexpr (KM) {
      const int a = stage + off + (((col + 2 * f) << 4) ^ sw);
      const uint2 lo = tr_read(lds + a), hi = tr_read(lds + a + 4 * T * 2);
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
      return *(const u32x4*)(lds + (stage + off + f * 16 * KB));
    }
  }
};

// Four consecutive outputs of one row, n of which exist.  STREAM: past the
// caches, for stores that fill whole lines (partial ones have to meet in L2:
// streamed, an output of 18944 x 3584 took 94 us instead of 60).
template <bool STREAM = false, typename Params>
__device__ __forceinline__ void put4(const Params& p, int64_t at, int n, const float v[4]) {
  if (p.obf16) {
    uint16_t* o = (uint16_t*)p.out + at;
    uint16_t e[4] = {0, 0, 0, 0};
    if (n >= 4) {
      if (p.accumulate) __builtin_memcpy(e, o, 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = to_bf16(p.accumulate ? bf16_bits_to_f32(e[i]) + v[i] : v[i]);
      __builtin_memcpy(o, e, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = to_bf16(p.accumulate ? bf16_bits_to_f32(o[i]) + v[i] : v[i]);
    }
  } else {
    float* o = (float*)p.out + at;
    if (n >= 4) {
      typedef float V __attribute__((ext_vector_type(4), aligned(4)));
      V e = {v[0], v[1], v[2], v[3]};
      if (p.accumulate) e += *(const V*)o;
      if constexpr (STREAM) __builtin_nontemporal_store(e, (V*)o);
      else *(V*)o = e;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = p.accumulate ? o[i] + v[i] : v[i];
    }
  }
}
// Eight of a bf16 row.
template <typename Params>
__device__ __forceinline__ void put8(const Params& p, int64_t at, int n, const float v[8]) {
  if (n < 8) {
    put4(p, at, n, v);
    if (n > 4) put4(p, at + 4, n - 4, v + 4);
    return;
  }
  typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
  uint16_t* o = (uint16_t*)p.out + at;
  uint16_t e[8];
  if (p.accumulate) __builtin_memcpy(e, o, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = to_bf16(p.accumulate ? bf16_bits_to_f32(e[i]) + v[i] : v[i]);
  V w;
  __builtin_memcpy(&w, e, 16);
  __builtin_nontemporal_store(w, (V*)o);
}

template <bool C> struct Cut { static constexpr bool value = C; };

constexpr int waves_of(int T) { return T == 256 ? 8 : 4; }

}  // namespace

}  // namespace l8
}  // namespace muon
