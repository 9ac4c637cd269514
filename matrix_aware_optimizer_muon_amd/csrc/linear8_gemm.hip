// Products of the 8-bit linear layer:
//   Y  = (xq wq^T) xs ws     int8 MFMA, exact int32 sums       (KIND_I8)
//   dX = dY (ws wq)          bf16 MFMA, fp32 sums              (KIND_DX)
//   dW = dY^T (xs xq)        bf16 MFMA, fp32 sums              (KIND_DW)
// all as C[q][p] = sum_k P(p, k) Q(q, k) with p contiguous in C.  P takes the
// MFMA's A side, so each lane ends with four consecutive columns of one row.
//
// For the gradients P is the 8-bit operand widened to bf16 with its scale
// folded in (exact for power-of-two scales: an int8 fits bf16's 8 significant
// bits), so every product of a dY value and a restored one is exact in the
// fp32 sum.  The widening is a pass of its own: the tile kernel then feeds
// both operands straight from HBM into LDS, and the pass moves 3 bytes per
// element of the 8-bit operand, 300 / N of the product's time.
//
// Tiles: 256 x 256 (8 waves, 2 x 4, each 128 x 64) or 128 x 128 (4 waves,
// 2 x 2, each 64 x 64).  A stage is 64 bytes of K per operand row (64 int8,
// 32 bf16): one MFMA K step.  Stages stream through a four-deep LDS ring
// filled by direct global->LDS loads; one barrier per stage, placed so that it
// publishes the next stage and retires the reads of the current one, and a
// constant vmcnt (stages past the end are loaded like any other, from valid
// addresses, and never read).
//
// Ragged sizes: output rows and columns past the end re-read the last valid
// one and are not stored; K past the end reads a zeroed line on both sides,
// so no value of a masked place (not even NaN) enters a sum.
#include "common.hpp"
#include "linear8.h"

namespace muon {
namespace l8 {

namespace {

constexpr int KB = 64;        // bytes of K per stage and contiguous row
constexpr int KROWS = 32;     // rows of K per stage of a K-major operand
constexpr int STAGES = 4;

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
// rows of 32 bytes that a transposing read takes fall on eight pair places.
__device__ __forceinline__ int swz_c(int row) { return ((row >> 2) & 1) << 1; }
__device__ __forceinline__ int swz_k(int k) { return ((k & 3) | (((k >> 3) & 1) << 2)) << 1; }

template <bool I8K> struct Mfma;
template <> struct Mfma<true> {
  typedef i32x4 Acc;
  static __device__ __forceinline__ void go(const u32x4& a, const u32x4& b, Acc& c) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};
template <> struct Mfma<false> {
  typedef f32x4 Acc;
  static __device__ __forceinline__ void go(const u32x4& a, const u32x4& b, Acc& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};

// Where a lane's DMA instructions read, and how a stage of one operand of T
// rows (columns, if K-major) is laid out in LDS: 64 bytes per row, or 32 rows
// of 2 T bytes.
template <bool KM, int T, int NW>
struct Operand {
  static constexpr int BYTES = T * KB;
  static constexpr int NDMA = BYTES / 1024 / NW;  // 1-KB instructions per wave and stage
  const char* src[NDMA];   // stage 0
  const char* tail[NDMA];  // the stage that K's end falls into
  int64_t step;            // bytes from stage to stage

  __device__ __forceinline__ void init(const char* base, int64_t ld, int row0, int count, int kd,
                                       int kbytes, int full, int wave, int lane) {
    step = KM ? KROWS * ld : (int64_t)KB;
#pragma unroll
    for (int i = 0; i < NDMA; ++i) {
      bool in;
      if constexpr (KM) {
        constexpr int RB = T * 2, RPI = 1024 / RB, CH = RB / 16;
        const int k = (wave * NDMA + i) * RPI + lane / CH;
        const int ch = (lane % CH) ^ swz_k(k);
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
    __builtin_amdgcn_global_load_lds((gbl_ptr_t*)s, (lds_ptr_t*)(stage + (wave * NDMA + i) * 1024), 16, 0, 0);
  }
};

// Fragment f (16 rows) of a wave's part of an operand stage.
template <bool KM, int T>
struct Reader {
  int off, sw, col;
  __device__ __forceinline__ void init(int first, int q4, int c16) {
    if constexpr (KM) {
      // two transposing reads, k 8 q4 .. +3 and +4 .. +7 (swz_k equal: bit 2
      // does not enter it); the lane addresses row 8 q4 + c16 / 4 (+ 4) and
      // columns first + 16 f + 4 (c16 % 4) .. +3
      const int k = 8 * q4 + (c16 >> 2);
      off = k * T * 2 + ((c16 & 3) >> 1) * 16 + (c16 & 1) * 8;
      sw = swz_k(k) << 4;
      col = first >> 3;
    } else {
      const int r = first + c16;
      off = r * KB + ((q4 ^ swz_c(r)) << 4);
    }
  }
  __device__ __forceinline__ u32x4 get(const char* stage, int f) const {
    if constexpr (KM) {
      const char* a = stage + off + (((col + 2 * f) << 4) ^ sw);
      const uint2 lo = tr_read(a), hi = tr_read(a + 4 * T * 2);
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
      return *(const u32x4*)(stage + off + f * 16 * KB);
    }
  }
};

__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Four consecutive outputs of one row, n of which exist.
__device__ __forceinline__ void put4(const MmParams& p, int64_t at, int n, const float v[4]) {
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
      float e[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p.accumulate) __builtin_memcpy(e, o, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = p.accumulate ? e[i] + v[i] : v[i];
      __builtin_memcpy(o, e, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = p.accumulate ? o[i] + v[i] : v[i];
    }
  }
}

template <bool I8K, bool PKM, bool QKM, int T>
__global__ void __launch_bounds__(T == 256 ? 512 : 256, T == 256 ? 1 : 2) mm_kernel(const MmParams p) {
  typedef Mfma<I8K> M;
  typedef typename M::Acc Acc;
  constexpr int NW = T == 256 ? 8 : 4;
  constexpr int WQ = NW / 2;                     // waves along Q (2 along P)
  constexpr int FP = T / 2 / 16, FQ = T / WQ / 16;  // 16 x 16 blocks per wave
  constexpr int H = FP / 2;                      // block rows per half stage
  typedef Operand<PKM, T, NW> OpP;
  typedef Operand<QKM, T, NW> OpQ;
  constexpr int DPS = OpP::NDMA + OpQ::NDMA;
  constexpr int STAGE = OpP::BYTES + OpQ::BYTES;
  __shared__ __attribute__((aligned(1024))) char smem[STAGES * STAGE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wp = wave / WQ, wq = wave % WQ;
  const int q4 = lane >> 4, c16 = lane & 15;

  const int tiles_p = (p.np + T - 1) / T, tiles_q = (p.nq + T - 1) / T;
  const uint32_t bid = xcd_remap_chunked(blockIdx.x, gridDim.x, 32);
  const int split = bid / (uint32_t)(tiles_p * tiles_q);
  int tp, tq;
  full_tile_grouped((int)bid - split * tiles_p * tiles_q, tiles_p, tiles_q, 8, &tp, &tq);

  constexpr int KE = I8K ? 64 : 32;              // K elements per stage
  const int full = p.kd / KE;
  const int nk = (p.kd + KE - 1) / KE;
  const int k0 = (int)((int64_t)nk * split / p.splits), k1 = (int)((int64_t)nk * (split + 1) / p.splits);

  OpP op;
  OpQ oq;
  op.init(p.P, p.ldp, tp * T, p.np, p.kd, p.kd * (I8K ? 1 : 2), full, wave, lane);
  oq.init(p.Q, p.ldq, tq * T, p.nq, p.kd, p.kd * (I8K ? 1 : 2), full, wave, lane);
  auto dma = [&](int q, int buf, int ks) {
    char* st = smem + buf * STAGE;
    if (q < OpP::NDMA) op.load(q, st, ks, full, wave);
    else oq.load(q - OpP::NDMA, st + OpP::BYTES, ks, full, wave);
  };
  Reader<PKM, T> rp;
  Reader<QKM, T> rq;
  rp.init(wp * (T / 2), q4, c16);
  rq.init(wq * (T / WQ), q4, c16);

  Acc acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = Acc{0, 0, 0, 0};
  u32x4 fa[FP], fb0[FQ], fb1[FQ];

  // A stage's DPS instructions go out in two halves, so that every run of
  // MFMAs carries the same share: the first half of stage kt + 4 in the second
  // half of step kt (its buffer is released by that step's barrier), the
  // rest in the first half of step kt + 1.
#pragma unroll
  for (int st = 0; st < STAGES; ++st)
#pragma unroll
    for (int q = 0; q < DPS; ++q)
      if (st < STAGES - 1 || q < DPS / 2) dma(q, st, k0 + st);
  __builtin_amdgcn_s_waitcnt(wait_imm(2 * DPS + DPS / 2, 15));
  barrier();
#pragma unroll
  for (int f = 0; f < H; ++f) fa[f] = rp.get(smem, f);
#pragma unroll
  for (int f = 0; f < FQ; ++f) fb0[f] = rq.get(smem + OpP::BYTES, f);

  auto step = [&](int kt, u32x4* fb, u32x4* fbn) {  // kt counts from k0
    const int buf = kt & (STAGES - 1);
    const char* sb = smem + buf * STAGE;
#pragma unroll
    for (int j = 0; j < FQ; ++j) M::go(fa[0], fb[j], acc[0][j]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = H; f < FP; ++f) fa[f] = rp.get(sb, f);
    __builtin_amdgcn_sched_barrier(0);
    constexpr int N1 = (H - 1) * FQ, G1 = N1 / (DPS / 2);
#pragma unroll
    for (int n = 0; n < N1; ++n) {
      M::go(fa[1 + n / FQ], fb[n % FQ], acc[1 + n / FQ][n % FQ]);
      if (n % G1 == G1 - 1) {
        dma(DPS / 2 + n / G1, (kt + STAGES - 1) & (STAGES - 1), k0 + kt + STAGES - 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // stage kt + 1 has landed for this wave (2 DPS later ones may fly) and its
    // reads of stage kt are done
    __builtin_amdgcn_s_waitcnt(wait_imm(2 * DPS, 0));
    barrier();
    const char* sn = smem + ((kt + 1) & (STAGES - 1)) * STAGE;
#pragma unroll
    for (int f = 0; f < H; ++f) fa[f] = rp.get(sn, f);
#pragma unroll
    for (int f = 0; f < FQ; ++f) fbn[f] = rq.get(sn + OpP::BYTES, f);
    __builtin_amdgcn_sched_barrier(0);
    constexpr int N2 = H * FQ, G2 = N2 / (DPS / 2);
#pragma unroll
    for (int n = 0; n < N2; ++n) {
      M::go(fa[H + n / FQ], fb[n % FQ], acc[H + n / FQ][n % FQ]);
      if (n % G2 == G2 - 1) dma(n / G2, buf, k0 + kt + STAGES);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const int steps = k1 - k0;
  int kt = 0;
  for (; kt + 1 < steps; kt += 2) {
    step(kt, fb0, fb1);
    step(kt + 1, fb1, fb0);
  }
  if (kt < steps) step(kt, fb0, fb1);
  __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));  // no load may land after the workgroup's LDS is given back

  // acc[i][j][e] is column col0 + 16 i + 4 q4 + e of row row0 + 16 j + c16
  const int col0 = tp * T + wp * (T / 2) + 4 * q4, row0 = tq * T + wq * (T / WQ) + c16;
#pragma unroll
  for (int j = 0; j < FQ; ++j) {
    const int r = row0 + 16 * j;
    if (r >= p.nq) continue;
    float sq = 1.0f;
    if (I8K && p.splits == 1) sq = p.sq[r];
#pragma unroll
    for (int i = 0; i < FP; ++i) {
      const int c = col0 + 16 * i;
      const int n = p.np - c;
      if (n <= 0) continue;
      if (p.splits > 1) {
        float* dst = p.part + ((int64_t)split * p.nq + r) * p.np + c;
        if (n >= 4) {
          __builtin_memcpy(dst, &acc[i][j], 16);
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (e < n) __builtin_memcpy(dst + e, (const char*)&acc[i][j] + 4 * e, 4);
        }
        continue;
      }
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = (float)acc[i][j][e];
        if constexpr (I8K) v[e] = v[e] * sq * p.sp[min(c + e, p.np - 1)];
      }
      put4(p, (int64_t)r * p.ldo + c, n, v);
    }
  }
}

// C = the splits' partial sums added in order, with the epilogue's scales.
template <bool I8K>
__global__ void __launch_bounds__(256) mm_sum_kernel(const MmParams p) {
  const int per = (p.np + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t r = id / per;
  if (r >= p.nq) return;
  const int c = (int)(id - r * per) * 4, n = min(4, p.np - c);
  const int64_t plane = (int64_t)p.nq * p.np;
  const float* src = p.part + r * p.np + c;
  typedef typename Mfma<I8K>::Acc Acc;
  Acc a = Acc{0, 0, 0, 0};
  for (int s = 0; s < p.splits; ++s) {
    Acc b = Acc{0, 0, 0, 0};
    if (n == 4) {
      __builtin_memcpy(&b, src + s * plane, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < n) __builtin_memcpy((char*)&b + 4 * e, src + s * plane + e, 4);
    }
    a += b;
  }
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = (float)a[e];
    if constexpr (I8K) v[e] = v[e] * p.sq[r] * p.sp[min(c + e, p.np - 1)];
  }
  put4(p, r * p.ldo + c, n, v);
}

// At most 16 rows of x.  A workgroup takes 16 rows of w; its four waves take
// every fourth 64-byte step of K, straight from HBM into MFMA fragments (a
// row of w is read once, by one workgroup; x stays in the caches), and the
// int32 partial tiles are added through LDS.
__global__ void __launch_bounds__(256) few_kernel(const int8_t* xq, int64_t ldx, const float* xs,
                                                  const int8_t* wq, int64_t ldw, const float* ws, void* y,
                                                  int64_t ldy, int bf16, int t, int n, int k) {
  __shared__ i32x4 s_part[3][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q4 = lane >> 4, c16 = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int8_t* wr = wq + (int64_t)min(n0 + c16, n - 1) * ldw + q4 * 16;
  const int8_t* xr = xq + (int64_t)min(c16, t - 1) * ldx + q4 * 16;
  i32x4 acc = {0, 0, 0, 0};
  const int whole = k / 64;
  int s = wave;
#pragma unroll 4
  for (; s < whole; s += 4) {
    u32x4 a, b;
    __builtin_memcpy(&a, wr + s * 64, 16);
    __builtin_memcpy(&b, xr + s * 64, 16);
    Mfma<true>::go(a, b, acc);
  }
  if (s == whole && k % 64) {  // one wave takes the ragged last step, byte by byte
    union { u32x4 v; int8_t e[16]; } a, b;
    const int left = k - whole * 64 - q4 * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      a.e[i] = i < left ? wr[whole * 64 + i] : (int8_t)0;
      b.e[i] = i < left ? xr[whole * 64 + i] : (int8_t)0;
    }
    Mfma<true>::go(a.v, b.v, acc);
  }
  if (wave > 0) s_part[wave - 1][lane] = acc;
  __syncthreads();
  if (wave == 0 && c16 < t) {
#pragma unroll
    for (int i = 0; i < 3; ++i) acc += s_part[i][lane];
    MmParams p = {};
    p.out = y;
    p.obf16 = bf16;
    const int c = n0 + 4 * q4;
    if (c < n) {
      const float sx = xs[c16];
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)acc[e] * sx * ws[min(c + e, n - 1)];
      put4(p, (int64_t)c16 * ldy + c, n - c, v);
    }
  }
}

__global__ void __launch_bounds__(256) pack_kernel(const char* src, int64_t lds, int64_t bytes, char* dst,
                                                   int64_t ld, int64_t rows) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16;
  if (c >= ld) return;
  const int64_t left = bytes - c;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const char* a = src + r * lds + c;
    union { u32x4 v; char e[16]; } b;
    if (left >= 16) {
      __builtin_memcpy(&b.v, a, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) b.e[i] = i < left ? a[i] : (char)0;
    }
    *(u32x4*)(dst + r * ld + c) = b.v;
  }
}

template <bool I8K, bool PKM, bool QKM>
hipError_t go_mm(const MmParams& p, hipStream_t s) {
  const int T = p.tile;
  const int64_t blocks = (int64_t)((p.np + T - 1) / T) * ((p.nq + T - 1) / T) * p.splits;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  if (T == 256)
    hipLaunchKernelGGL((mm_kernel<I8K, PKM, QKM, 256>), dim3((uint32_t)blocks), dim3(512), 0, s, p);
  else
    hipLaunchKernelGGL((mm_kernel<I8K, PKM, QKM, 128>), dim3((uint32_t)blocks), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm(const MmParams& p, ProductKind kind, hipStream_t s) {
  switch (kind) {
    case KIND_I8: return go_mm<true, false, false>(p, s);
    case KIND_DX: return go_mm<false, true, false>(p, s);
    case KIND_DW: return go_mm<false, true, true>(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_mm_sum(const MmParams& p, ProductKind kind, hipStream_t s) {
  const int64_t threads = (int64_t)((p.np + 3) / 4) * p.nq;
  const dim3 grid((uint32_t)((threads + 255) / 256));
  if (kind == KIND_I8) hipLaunchKernelGGL(mm_sum_kernel<true>, grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(mm_sum_kernel<false>, grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_few(const int8_t* xq, int64_t ldx, const float* xs, const int8_t* wq, int64_t ldw,
                      const float* ws, void* y, int64_t ldy, bool bf16, int t, int n, int k, hipStream_t s) {
  hipLaunchKernelGGL(few_kernel, dim3((uint32_t)((n + 15) / 16)), dim3(256), 0, s, xq, ldx, xs, wq, ldw, ws,
                     y, ldy, bf16 ? 1 : 0, t, n, k);
  return hipGetLastError();
}

hipError_t launch_pack(const void* src, int64_t lds, int64_t bytes, void* dst, int64_t ld, int64_t rows,
                       hipStream_t s) {
  const dim3 grid((uint32_t)((ld / 16 + 255) / 256), (uint32_t)(rows < 32768 ? rows : 32768));
  hipLaunchKernelGGL(pack_kernel, grid, dim3(256), 0, s, (const char*)src, lds, bytes, (char*)dst, ld, rows);
  return hipGetLastError();
}

}  // namespace l8
}  // namespace muon
