// Products of the 8-bit linear layer:
//   Y  = (xq wq^T) xs ws     int8 MFMA, exact int32 sums       (KIND_I8)
//   dX = dY (ws wq)          bf16 MFMA, fp32 sums              (KIND_DX)
//   dW = dY^T (xs xq)        bf16 MFMA, fp32 sums              (KIND_DW)
// all as C[q][p] = sum_k P(p, k) Q(q, k) with p contiguous in C.  P takes the
// MFMA's A side, so each lane ends with four consecutive columns of one row.
//
// For the gradients P is the 8-bit operand, widened to bf16 with its scale
// folded in on its way from HBM through registers into LDS (exact for
// power-of-two scales: an int8 fits bf16's 8 significant bits), so every
// product of a dY value and a restored one is exact in the fp32 sum, and no
// widened copy exists in memory.  2.5 vector instructions per element, once
// per workgroup, run between the MFMAs.
//
// Tiles: 256 x 256 (8 waves, 2 x 4, each 128 x 64), 128 x 128 (one or two
// groups of 4 waves, 2 x 2, each 64 x 64) or 64 x 64 (four groups of 4 waves,
// each 32 x 32).  A stage is 64 bytes of K per operand row (64 int8,
// 32 bf16): one MFMA K step.  Stages stream through a four-deep LDS
// ring filled by direct global->LDS loads or from registers; one barrier per stage, placed so that it
// publishes the next stage and retires the reads of the current one, and a
// constant vmcnt (stages past the end are loaded like any other, from valid
// addresses, and never read).
//
// Bound by the matrix cores' issue and the card's power: a product of 4096 x
// 18944 x 3584 takes 242 to 252 us by the card (2.3 to 2.2 POP/s), the input
// gradient of that size 479 to 492 (1.16 to 1.13 PFLOP/s), the weight gradient
// 493 to 512 (1.13 to 1.09); the matrix cores are busy 59, 58 and 51 % of the
// cycles, LDS 26 to 36 %, at 1.8 to 1.9 GHz.
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

// One operand fed through registers, CH bytes of a row per lane and chunk: at
// any address, and, with CONV, int8 rows times their scale widened to bf16 on
// the way.  Whole reads that leave the row stay inside the matrix for all
// stages before `safe` (load).  load_cut, for any stage, moves a read that
// would leave the matrix back inside, and `store` puts such bytes in place and
// zeros what lies past the row or the sum: without a branch, and only when the
// stage is due, so that loads stay in flight (byte reads behind their
// predicates took 8 us of a one-stage product).  The matrix has at least 16
// bytes (`pad` of them may follow its last row).
template <bool KM, bool CONV, int T, int NT>
struct RegOperand {
  static constexpr int CH = CONV && T == 64 ? 8 : 16;
  static constexpr int CPR = KM ? (CONV ? T : T * 2) / CH : 4;   // chunks per stage row
  static constexpr int SROWS = KM ? KROWS : T;                   // stage rows
  static constexpr int N = SROWS * CPR / NT;                     // chunks per lane
  static_assert(N * NT == SROWS * CPR && (!CONV || N == 1), "whole chunks per lane");
  struct Regs {
    u32x4 v[N];
    float scale;
  };
  const char* src[N];
  const float* scale;
  const char* last;
  int64_t step;
  int safe, kd, left;  // left: bytes of the chunk's row from the chunk on
  int row, col;        // the lane's first stage row, its chunk

  __device__ __forceinline__ void init(const char* base, int64_t ld, int pad, const float* sc, int row0,
                                       int count, int kdim, int kbytes, int full, int tid) {
    last = base - CH + pad +
           (KM ? (int64_t)(kdim - 1) * ld + count * (CONV ? 1 : 2) : (int64_t)(count - 1) * ld + kbytes);
    row = tid / CPR;
    col = tid % CPR;
    kd = kdim;
    scale = sc;
    if constexpr (KM) {
      constexpr int SZ = CONV ? 1 : 2;
      const int rb = count * SZ, end = (rb - 1) & ~(CH - 1);  // row bytes, its last chunk
      const int c = min(row0 * SZ + col * CH, end);
      left = rb - c;
      step = KROWS * ld;
      // rows whose last chunk, read whole, ends inside the matrix
      const int over = end + CH - rb;
      const int64_t rows = over > 0 ? kd - (over + ld - 1) / ld : kd;
      safe = rows > 0 ? (int)(rows / KROWS) : 0;
#pragma unroll
      for (int i = 0; i < N; ++i) src[i] = base + (int64_t)(row + i * (KROWS / N)) * ld + c;
    } else {
      step = KB;
      safe = full;
      left = kbytes - col * CH;
#pragma unroll
      for (int i = 0; i < N; ++i) src[i] = base + (int64_t)min(row0 + row + i * (T / N), count - 1) * ld + col * CH;
    }
  }
  // A stage before `safe`.
  __device__ __forceinline__ void load(Regs& r, int ks) const {
#pragma unroll
    for (int i = 0; i < N; ++i) __builtin_memcpy(&r.v[i], src[i] + ks * step, CH);
    if constexpr (CONV) r.scale = scale[ks * KROWS + row];
  }
  // Any stage.
  __device__ __forceinline__ void load_cut(Regs& r, int ks) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const char* a = src[i] + ks * step;
      __builtin_memcpy(&r.v[i], a < last ? a : last, CH);
    }
    if constexpr (CONV) r.scale = scale[min(ks * KROWS + row, kd - 1)];
  }
  // Chunk i of a stage that load_cut (or load) has read.
  __device__ __forceinline__ void mend(Regs& r, int i, int ks) const {
    const char* a = src[i] + ks * step;
    const int d = a < last ? 0 : (int)(a - last) & (CH - 1);
    int n;
    if constexpr (KM) n = ks * KROWS + row + i * (KROWS / N) < kd ? left : 0;
    else n = left - ks * KB;
    r.v[i] = put_in_place(r.v[i], d, n);
    if constexpr (CONV) r.scale = ks * KROWS + row < kd ? r.scale : 0.0f;
  }
  // Piece q of PIECES of a stage's way into LDS, so that the caller can put
  // MFMAs between them.
  static constexpr int PIECES = CONV ? CH / 4 : N;
  struct Wide {
    uint32_t d[CONV ? CH / 2 : 1];
  };
  template <bool CUT>
  __device__ __forceinline__ void store(Regs& r, Wide& w, char* lds, int stage, int ks, int q) const {
    if (CUT && (!CONV || q == 0)) mend(r, q, ks);
    if constexpr (CONV) {
      // (opaque: the compiler otherwise takes the bytes apart at the load,
      // carries 16 registers for 4 and waits for the load to do so)
      uint32_t b = r.v[0][q];
      asm("" : "+v"(b));
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = (float)(int8_t)(b >> (8 * e)) * r.scale;
      w.d[2 * q] = pack_bf16(f[0], f[1]);
      w.d[2 * q + 1] = pack_bf16(f[2], f[3]);
      if (q == PIECES - 1) {
        // swz_k is even, so a lane's two chunks stay side by side
        const int d = stage + row * (T * 2) + ((col * (CH / 8) ^ swz_k<T>(row)) << 4);
        *(u32x4*)(lds + d) = u32x4{w.d[0], w.d[1], w.d[2], w.d[3]};
        if constexpr (CH == 16) *(u32x4*)(lds + d + 16) = u32x4{w.d[4], w.d[5], w.d[6], w.d[7]};
      }
    } else if constexpr (KM) {
      const int k = row + q * (KROWS / N);
      *(u32x4*)(lds + (stage + k * (T * 2) + ((col ^ swz_k<T>(k)) << 4))) = r.v[q];
    } else {
      const int t = row + q * (T / N);
      *(u32x4*)(lds + (stage + t * KB + ((col ^ swz_c(t)) << 4))) = r.v[q];
    }
  }
};

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
template <bool STREAM = false>
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
__device__ __forceinline__ void put8(const MmParams& p, int64_t at, int n, const float v[8]) {
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

// How the kernel reads its operands: P through registers for the gradients
// (widened), by DMA or, at unaligned addresses, through registers for the
// integer product; Q by DMA or, unaligned, through registers.
//
// G groups of waves share a tile, each with a share of K and LDS rings of its
// own, and join their sums through LDS: where there are no more tiles than
// compute units, a group alone on its SIMDs waits for LDS and barriers most of
// the time (0.37 us per stage of a 128 x 128 tile, a third of it MFMAs), and
// the join costs no second launch.
constexpr int waves_of(int T) { return T == 256 ? 8 : 4; }

template <int KIND, bool UNALIGNED, int T, int G>
__global__ void __launch_bounds__(64 * waves_of(T) * G, T == 128 && G == 1 ? 2 : 1)
    mm_kernel(const MmParams p) {
  constexpr bool I8K = KIND == KIND_I8, PKM = !I8K, QKM = KIND == KIND_DW;
  constexpr bool PREG = !I8K || UNALIGNED, QREG = UNALIGNED;
  typedef Mfma<I8K> M;
  typedef typename M::Acc Acc;
  constexpr int NW = waves_of(T);                // waves of a group
  constexpr int WQ = NW / 2;                     // waves along Q (2 along P)
  constexpr int FP = T / 2 / 16, FQ = T / WQ / 16;  // 16 x 16 blocks per wave
  constexpr int H = FP / 2;                      // block rows per half stage
  typedef DmaOperand<PKM, T, NW> DmaP;
  typedef DmaOperand<QKM, T, NW> DmaQ;
  typedef RegOperand<PKM, PKM, T, 64 * NW> RegP;
  typedef RegOperand<QKM, false, T, 64 * NW> RegQ;
  constexpr int DP = PREG ? 0 : DmaP::NDMA, DPS = DP + (QREG ? 0 : DmaQ::NDMA);
  constexpr int DB = DPS / 2, DA = DPS - DB;     // the two halves of a stage's instructions
  constexpr int OPB = T * KB;                    // one operand's stage in LDS
  constexpr int D = 4;                           // stages of a ring
  constexpr int RS = 2;                          // register sets in flight
  // (two objects: the compiler then knows that a write to one is no write to
  // the other)
  __shared__ __attribute__((aligned(1024))) char s_p[G * D * OPB];
  __shared__ __attribute__((aligned(1024))) char s_q[G * D * OPB];

  const int tid = threadIdx.x % (64 * NW), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = G > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / (64 * NW)) : 0;
  const int ring = group * D * OPB;              // the group's rings
  auto at = [&](int st) { return (st & (D - 1)) * OPB; };  // a stage in them
  const int wp = wave / WQ, wq = wave % WQ;
  const int q4 = lane >> 4, c16 = lane & 15;

  // The first `direct` tiles belong to one workgroup each, the others to
  // `splits` workgroups each, a range of K apiece.
  const int tiles_p = (p.np + T - 1) / T, tiles_q = (p.nq + T - 1) / T;
  const int bid = (int)xcd_remap_chunked(blockIdx.x, gridDim.x, 32);
  int tile = bid, split = 0, splits = 1;
  const int rest = tiles_p * tiles_q - p.direct;
  if (bid >= p.direct) {
    const int u = bid - p.direct;
    split = u / rest;
    tile = p.direct + u - split * rest;
    splits = p.splits;
  }
  int tp, tq;
  full_tile_grouped(tile, tiles_p, tiles_q, 8, &tp, &tq);

  constexpr int KE = I8K ? 64 : 32;              // K elements per stage
  const int full = p.kd / KE;
  const int nk = (p.kd + KE - 1) / KE;
  int k0 = 0, k1 = nk;
  if (splits > 1) {
    k0 = (int)((int64_t)nk * split / splits);
    k1 = (int)((int64_t)nk * (split + 1) / splits);
  }
  // stages per group, and this group's (the last ones may have fewer)
  const int most = (k1 - k0 + G - 1) / G;
  const int steps = G > 1 ? max(0, min(most, k1 - k0 - group * most)) : most;
  k0 += group * most;
  const int kbytes = p.kd * (I8K ? 1 : 2);

  Acc acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = Acc{0, 0, 0, 0};

  // acc[i][j][e] is column 16 i + 4 q4 + e of row 16 j + c16 of the wave's part
  const int colt = wp * (T / 2), rowt = wq * (T / WQ);
  const int col0 = tp * T + colt, row0 = tq * T + rowt;
  // Tiles over 64 leave through LDS in whole rows: a lane's columns there, 8
  // of a bf16 row (`wide`), else 4.  The smaller ones: a lane's own block.
  const bool wide = splits == 1 && p.obf16;
  const int outc = T > 64 ? (wide ? lane % (T / 16) * 8 : lane % (T / 8) * 4) : 16 * (group / FQ) + 4 * q4;
  // (the integer product's scales are here before they are due: read at the
  // end, they cost each tile a trip to memory)
  float sq[T > 64 ? FQ : 1];
  f32x4 sp[2];
  if constexpr (I8K) {
    if (splits == 1) {
#pragma unroll
      for (int j = 0; j < (T > 64 ? FQ : 1); ++j)
        sq[j] = p.sq[min(row0 + 16 * (T > 64 ? j : group % FQ) + c16, p.nq - 1)];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < 4 || T > 64) sp[e / 4][e % 4] = p.sp[min(col0 + outc + e, p.np - 1)];
    }
  }

  if (steps > 0) {  // (an empty sum reads nothing)
    DmaP dp;
    DmaQ dq;
    RegP gp;
    RegQ gq;
    if constexpr (PREG) gp.init(p.P, p.ldp, p.padp, p.sp, tp * T, p.np, p.kd, kbytes, full, tid);
    else dp.init(p.P, p.ldp, tp * T, p.np, p.kd, kbytes, full, tid);
    if constexpr (QREG) gq.init(p.Q, p.ldq, p.padq, nullptr, tq * T, p.nq, p.kd, kbytes, full, tid);
    else dq.init(p.Q, p.ldq, tq * T, p.nq, p.kd, kbytes, full, tid);
    auto dma = [&](int q, int st) __attribute__((always_inline)) {  // instruction q of stage k0 + st
      if (q < DP) dp.load(q, s_p + ring + at(st), k0 + st, full, wave);
      else dq.load(q - DP, s_q + ring + at(st), k0 + st, full, wave);
    };
    typename RegP::Regs rp[RS];
    typename RegQ::Regs rq[RS];
    typename RegP::Wide wp8;
    typename RegQ::Wide wq8;
    auto fetch = [&](auto cut, typename RegP::Regs& a, typename RegQ::Regs& b, int st) __attribute__((always_inline)) {
      if constexpr (PREG) {
        if constexpr (decltype(cut)::value) gp.load_cut(a, k0 + st);
        else gp.load(a, k0 + st);
      }
      if constexpr (QREG) {
        if constexpr (decltype(cut)::value) gq.load_cut(b, k0 + st);
        else gq.load(b, k0 + st);
      }
    };
    // pieces of a register set's way into LDS as stage k0 + st
    constexpr int PP = PREG ? RegP::PIECES : 0, PQ = QREG ? RegQ::PIECES : 0, PIECES = PP + PQ;
    auto put = [&](auto cut, typename RegP::Regs& a, typename RegQ::Regs& b, int st,
                   int q) __attribute__((always_inline)) {
      constexpr bool CUT = decltype(cut)::value;
      if (q < PP) gp.template store<CUT>(a, wp8, s_p, ring + at(st), k0 + st, q);
      else if (q < PIECES) gq.template store<CUT>(b, wq8, s_q, ring + at(st), k0 + st, q - PP);
    };
    Reader<PKM, T> fp;
    Reader<QKM, T> fq;
    fp.init(ring, wp * (T / 2), q4, c16);
    fq.init(ring, wq * (T / WQ), q4, c16);
    u32x4 fa[FP], fb0[FQ], fb1[FQ];

    // DMA: a stage's DPS instructions go out in two halves, so that every run
    // of MFMAs carries the same share: the first half of stage kt + D in the
    // second half of step kt (its buffer is released by that step's barrier),
    // the rest in the first half of step kt + 1.
    // Registers: stage kt + 2 goes into LDS in the second half of step kt, and
    // its set is loaded again with stage kt + 2 + RS, RS steps ahead of its
    // use.
#pragma unroll
    for (int st = 0; st < D; ++st)
      if (st < steps) {
#pragma unroll
        for (int q = 0; q < DPS; ++q)
          if (st < D - 1 || q < DA) dma(q, st);
      }
    if constexpr (PIECES > 0) {
      // stages 0 .. RS + 1 in flight together; everything has landed before
      // the loop, so that the waits inside it only count the loop's own loads
      typename RegP::Regs rp0[2];
      typename RegQ::Regs rq0[2];
#pragma unroll
      for (int st = 0; st < 2; ++st) fetch(Cut<true>(), rp0[st], rq0[st], st);
#pragma unroll
      for (int st = 0; st < RS; ++st) fetch(Cut<true>(), rp[st], rq[st], 2 + st);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int q = 0; q < PIECES; ++q) put(Cut<true>(), rp0[st], rq0[st], st, q);
      __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
    } else if (steps < D) {
      __builtin_amdgcn_s_waitcnt(wait_imm(0, 15));
    } else {
      __builtin_amdgcn_s_waitcnt(wait_imm((D - 2) * DPS + DA, 15));
    }
    barrier();
#pragma unroll
    for (int f = 0; f < H; ++f) fa[f] = fp.get(s_p, at(0), f);
#pragma unroll
    for (int f = 0; f < FQ; ++f) fb0[f] = fq.get(s_q, at(0), f);

    // A step, kt counting from k0, set = kt % RS.  Cut: near the end of the
    // sum; what lies past it is not loaded.
    auto step = [&](auto cut, int kt, int set, u32x4* fb, u32x4* fbn) __attribute__((always_inline)) {
      constexpr bool CUT = decltype(cut)::value;
#pragma unroll
      for (int j = 0; j < FQ; ++j) M::go(fa[0], fb[j], acc[0][j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = H; f < FP; ++f) fa[f] = fp.get(s_p, at(kt), f);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int N1 = (H - 1) * FQ, G1 = DB > 0 && N1 > DB ? N1 / (DB + (DB == 0)) : 1;
#pragma unroll
      for (int n = 0; n < N1; ++n) {
        M::go(fa[1 + n / FQ], fb[n % FQ], acc[1 + n / FQ][n % FQ]);
        if (DB > 0 && n % G1 == G1 - 1 && n / G1 < DB) {
          if (!CUT || kt + D - 1 < steps) dma(DA + n / G1, kt + D - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (N1 == 0) {
#pragma unroll
        for (int q = 0; q < DB; ++q)
          if (!CUT || kt + D - 1 < steps) dma(DA + q, kt + D - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      // This wave's DMAs of stage kt + 1 have landed ((D - 2) DPS later ones
      // may fly; register loads among them make the wait stricter: counting
      // them in measured 2-4 % slower on the weight gradients), its LDS
      // writes of stage kt + 1 and its reads of stage kt are done.
      if (CUT && DPS > 0 && kt + D - 1 >= steps) __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
      else __builtin_amdgcn_s_waitcnt(wait_imm(DPS > 0 ? (D - 2) * DPS : 63, 0));
      barrier();
#pragma unroll
      for (int f = 0; f < H; ++f) fa[f] = fp.get(s_p, at(kt + 1), f);
#pragma unroll
      for (int f = 0; f < FQ; ++f) fbn[f] = fq.get(s_q, at(kt + 1), f);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int N2 = H * FQ, G2 = N2 / (DA > 0 ? DA : 1);
      // pieces after each MFMA (several, where there are few MFMAs)
      constexpr int GP = N2 > PIECES ? N2 / (PIECES + 1) : 1, PB = (PIECES + N2 - 1) / N2;
#pragma unroll
      for (int n = 0; n < N2; ++n) {
        M::go(fa[H + n / FQ], fb[n % FQ], acc[H + n / FQ][n % FQ]);
        if (DA > 0 && n % G2 == G2 - 1 && n / G2 < DA && (!CUT || kt + D < steps)) dma(n / G2, kt + D);
        if (PIECES > 0 && n % GP == GP - 1) {
#pragma unroll
          for (int q = 0; q < PB; ++q)
            if (n / GP * PB + q < PIECES) put(cut, rp[set], rq[set], kt + 2, n / GP * PB + q);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (PIECES > 0) {
        if (!CUT || kt + 2 + RS < steps) fetch(cut, rp[set], rq[set], kt + 2 + RS);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // Two steps per trip: the Q fragments and the register sets alternate
    // without copies.  The trips whose loads stay before the end and the cut
    // stages come first and carry no checks.
    int kt = 0;
    auto trips = [&](auto cut, int end) __attribute__((always_inline)) {
      for (; kt + 1 < end; kt += 2) {
        step(cut, kt, 0, fb0, fb1);
        step(cut, kt + 1, 1, fb1, fb0);
      }
    };
    int safe = steps - D;
    if constexpr (PREG) safe = min(safe, gp.safe - k0 - RS - 2);
    if constexpr (QREG) safe = min(safe, gq.safe - k0 - RS - 2);
    trips(Cut<false>(), safe);
    trips(Cut<true>(), steps);
    if (kt < steps) step(Cut<true>(), kt, 0, fb0, fb1);
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));  // no load may land after the workgroup's LDS is given back
  }
  if constexpr (G > 1) {
    // a group's barriers: one ahead of the loop and one per step; then one
    // that ends all reads of the rings
    if (most > 0) {
      for (int i = steps > 0 ? steps : -1; i < most; ++i) barrier();
    }
    barrier();
    // Block b of every wave is finished by group b % G: the other groups
    // leave theirs in LDS, lane by lane, and it adds them in their order.
    constexpr int B = FP * FQ;
    static_assert(B % G == 0 && B * (G - 1) * NW * 1024 <= G * D * OPB, "the join fits the ring");
    auto slot = [&](int b, int from) -> Acc* {
      const int o = b % G;
      return (Acc*)(s_p + (((b / G) * G + o) * (G - 1) + (from < o ? from : from - 1)) * (NW * 1024) + tid * 16);
    };
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (b % G != group) *slot(b, group) = acc[b / FQ][b % FQ];
    __syncthreads();
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (b % G == group) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (g != b % G) acc[b / FQ][b % FQ] += *slot(b, g);
      }
  }

  float* const part = p.part + ((int64_t)(tile - p.direct) * splits + split) * (T * T);
  if constexpr (T > 64) {
    // A lane's four columns are 16 bytes of a row 16 rows apart from its
    // neighbours'.  Sixteen rows of the wave's part at a time go through LDS,
    // 16-byte chunks swapped within a row by the row's number (no bank
    // conflicts either way), and leave as whole rows: 256 bytes or more each.
    // One loop over the blocks of rows, not unrolled but for its first lines:
    // the code is fetched anew by each launch.
    constexpr int PT = 16 * FP, CPR = PT / 4;  // columns and chunks of a row
    static_assert(NW * 16 * PT * 4 * G <= G * D * OPB, "the staged rows fit a ring");
    if constexpr (G == 1) barrier();  // no wave reads the rings any more
    char* const st = s_q + (group * NW + wave) * (16 * PT * 4);
    auto chunk = [&](int r, int c) { return st + r * (PT * 4) + ((c ^ (r & (CPR - 1))) << 4); };
    const int ch = outc / 4, n = p.np - (col0 + outc);
#pragma clang loop unroll(disable)
    for (int jr = G > 1 ? group : 0; jr < FQ; jr += G) {  // (FQ is a multiple of G: block (i, j) is group j % G's)
#pragma unroll
      for (int j = 0; j < FQ; ++j)
        if (j == jr) {
#pragma unroll
          for (int i = 0; i < FP; ++i) {
            f32x4 v;
            if (I8K && splits == 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * sq[j];
            } else {
              v = __builtin_bit_cast(f32x4, acc[i][j]);
            }
            *(f32x4*)chunk(c16, 4 * i + q4) = v;
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int r0 = row0 + 16 * jr;
      if (!wide) {
        constexpr int RPI = 64 / CPR;  // rows per instruction
        int rr = lane / CPR;
#pragma unroll 4
        for (int it = 0; it < 16 / RPI; ++it, rr += RPI) {
          f32x4 v = *(const f32x4*)chunk(rr, ch);
          if (splits > 1) {
            *(f32x4*)(part + (rowt + 16 * jr + rr) * T + colt + outc) = v;
          } else if (r0 + rr < p.nq && n > 0) {
            if constexpr (I8K) v *= sp[0];
            const float o[4] = {v[0], v[1], v[2], v[3]};
            put4<true>(p, (int64_t)(r0 + rr) * p.ldo + col0 + outc, n, o);
          }
        }
      } else {
        constexpr int RPI = 128 / CPR;
        int rr = lane / (CPR / 2);
#pragma unroll 2
        for (int it = 0; it < 16 / RPI; ++it, rr += RPI) {
          f32x4 v = *(const f32x4*)chunk(rr, ch), w = *(const f32x4*)chunk(rr, ch + 1);
          if constexpr (I8K) v *= sp[0], w *= sp[1];
          const float o[8] = {v[0], v[1], v[2], v[3], w[0], w[1], w[2], w[3]};
          if (r0 + rr < p.nq && n > 0) put8(p, (int64_t)(r0 + rr) * p.ldo + col0 + outc, n, o);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    static_assert(FP * FQ == G, "one block per group");
    const int r = 16 * (group % FQ) + c16, n = p.np - col0 - outc;
    Acc a = acc[0][0];
#pragma unroll
    for (int b = 1; b < FP * FQ; ++b)
      if (b == group) a = acc[b / FQ][b % FQ];
    if (splits > 1) {  // the raw sums
      *(Acc*)(part + (rowt + r) * T + colt + outc) = a;
    } else if (row0 + r < p.nq && n > 0) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = (float)a[e];
        if constexpr (I8K) v[e] = v[e] * sq[0] * sp[0][e];
      }
      put4(p, (int64_t)(row0 + r) * p.ldo + col0 + outc, n, v);
    }
  }
}

// C = the splits' partial sums added in order, with the epilogue's scales:
// blockIdx.y a split tile, four columns of a row per thread.
template <bool I8K, int T>
__global__ void __launch_bounds__(256) mm_sum_kernel(const MmParams p) {
  const int at = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
  const int tiles_p = (p.np + T - 1) / T, tiles_q = (p.nq + T - 1) / T;
  int tp, tq;
  full_tile_grouped(p.direct + (int)blockIdx.y, tiles_p, tiles_q, 8, &tp, &tq);
  const int r = tq * T + at / T, c = tp * T + at % T, n = p.np - c;
  if (r >= p.nq || n <= 0) return;
  typedef typename Mfma<I8K>::Acc Acc;
  const float* src = p.part + (int64_t)blockIdx.y * p.splits * (T * T) + at;
  Acc a = *(const Acc*)src;
#pragma unroll 4
  for (int s = 1; s < p.splits; ++s) a += *(const Acc*)(src + (int64_t)s * (T * T));
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = (float)a[e];
    if constexpr (I8K) v[e] = v[e] * p.sq[r] * p.sp[min(c + e, p.np - 1)];
  }
  put4(p, (int64_t)r * p.ldo + c, n, v);
}

// Few rows of x (at most 16 QB).  A workgroup takes 16 rows of w; its W waves
// take every W-th 64-byte step of K, straight from memory into MFMA fragments
// at any alignment (a row of w is read once, by one workgroup; x comes from
// the caches), and the int32 partial tiles are added through LDS.  Bound by
// the read of w: one row of x against 18944 x 3584 takes 13.9 us from memory
// (4.9 TB/s) and 12.1 where the last-level cache holds w.
template <int QB, int W>
__global__ void __launch_bounds__(64 * W) few_kernel(const int8_t* xq, int64_t ldx, const float* xs,
                                                  const int8_t* wq, int64_t ldw, const float* ws, void* y,
                                                  int64_t ldy, int bf16, int t, int n, int k) {
  __shared__ i32x4 s_part[W - 1][QB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q4 = lane >> 4, c16 = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int8_t* const wr = wq + (int64_t)min(n0 + c16, n - 1) * ldw + q4 * 16;
  const int8_t* xr[QB];
#pragma unroll
  for (int j = 0; j < QB; ++j) xr[j] = xq + (int64_t)min(16 * j + c16, t - 1) * ldx + q4 * 16;
  i32x4 acc[QB];
#pragma unroll
  for (int j = 0; j < QB; ++j) acc[j] = i32x4{0, 0, 0, 0};
  const int whole = k / 64;
  int s = wave;
#pragma unroll 4
  for (; s < whole; s += W) {
    u32x4 a, b[QB];
    __builtin_memcpy(&a, wr + s * 64, 16);
#pragma unroll
    for (int j = 0; j < QB; ++j) __builtin_memcpy(&b[j], xr[j] + s * 64, 16);
#pragma unroll
    for (int j = 0; j < QB; ++j) Mfma<true>::go(a, b[j], acc[j]);
  }
  if (s == whole && k % 64) {  // one wave takes the ragged last step
    u32x4 a, b[QB];
    const int left = k - whole * 64 - q4 * 16;
    auto part = [&](const int8_t* r, const int8_t* base, int64_t total) {
      const char* c = (const char*)r + whole * 64;
      if (total >= 16) return load_part(c, left, (const char*)base + total - 16);
      u32x4 v = {0, 0, 0, 0};  // a matrix of less than 16 bytes
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) v[i / 4] |= (uint32_t)(uint8_t)c[i] << (8 * (i % 4));
      return v;
    };
    a = part(wr, wq, (int64_t)(n - 1) * ldw + k);
#pragma unroll
    for (int j = 0; j < QB; ++j) b[j] = part(xr[j], xq, (int64_t)(t - 1) * ldx + k);
#pragma unroll
    for (int j = 0; j < QB; ++j) Mfma<true>::go(a, b[j], acc[j]);
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < QB; ++j) s_part[wave - 1][j][lane] = acc[j];
  }
  __syncthreads();
  if (wave > 0) return;
  MmParams p = {};
  p.out = y;
  p.obf16 = bf16;
  const int c = n0 + 4 * q4;
#pragma unroll
  for (int j = 0; j < QB; ++j) {
    i32x4 a = acc[j];
#pragma unroll
    for (int q = 0; q < W - 1; ++q) a += s_part[q][j][lane];
    const int r = 16 * j + c16;
    if (c < n && r < t) {
      const float sx = xs[r];
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)a[e] * sx * ws[min(c + e, n - 1)];
      put4(p, (int64_t)r * ldy + c, n - c, v);
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

template <int KIND>
hipError_t go_mm(const MmParams& p, hipStream_t s) {
  const int T = p.tile;
  const int64_t tiles = (int64_t)((p.np + T - 1) / T) * ((p.nq + T - 1) / T), rest = tiles - p.direct;
  const int64_t blocks = p.direct + rest * p.splits;
  // (a launch has fewer than 2^32 threads; outputs that need more pass any memory)
  const int threads = 64 * waves_of(T) * p.groups;
  if (blocks > 0xffffffffll / threads || rest < 0 || (T == 256 && p.unaligned)) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)blocks);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, p); };
  if (T == 256) go(mm_kernel<KIND, false, 256, 1>);
  else if (T == 128 && p.groups == 2) p.unaligned ? go(mm_kernel<KIND, true, 128, 2>) : go(mm_kernel<KIND, false, 128, 2>);
  else if (T == 128) p.unaligned ? go(mm_kernel<KIND, true, 128, 1>) : go(mm_kernel<KIND, false, 128, 1>);
  else p.unaligned ? go(mm_kernel<KIND, true, 64, 4>) : go(mm_kernel<KIND, false, 64, 4>);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 sums((uint32_t)(T * T / 1024), (uint32_t)rest);
  constexpr bool I8K = KIND == KIND_I8;
  if (T == 256) hipLaunchKernelGGL((mm_sum_kernel<I8K, 256>), sums, dim3(256), 0, s, p);
  else if (T == 128) hipLaunchKernelGGL((mm_sum_kernel<I8K, 128>), sums, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((mm_sum_kernel<I8K, 64>), sums, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm(const MmParams& p, ProductKind kind, hipStream_t s) {
  switch (kind) {
    case KIND_I8: return go_mm<KIND_I8>(p, s);
    case KIND_DX: return go_mm<KIND_DX>(p, s);
    case KIND_DW: return go_mm<KIND_DW>(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_few(const int8_t* xq, int64_t ldx, const float* xs, const int8_t* wq, int64_t ldw,
                      const float* ws, void* y, int64_t ldy, bool bf16, int t, int n, int k, hipStream_t s) {
  auto go = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((n + 15) / 16)), dim3(64 * waves), 0, s, xq, ldx, xs, wq, ldw, ws, y,
                       ldy, bf16 ? 1 : 0, t, n, k);
    return hipGetLastError();
  };
  // Eight waves read a row's K faster than four until there are four
  // workgroups per compute unit (one row of x, w from memory: 8192 x 8192 14.5
  // and 21.4 us, 12000 x 8192 20.2 and 23.9, 16384 x 4096 15.8 and 15.7, 18944 x
  // 3584 16.1 and 13.9).
  if (t > 16) return go(few_kernel<2, 8>, 8);
  return n < 16 * 1024 ? go(few_kernel<1, 8>, 8) : go(few_kernel<1, 4>, 4);
}

hipError_t launch_pack(const void* src, int64_t lds, int64_t bytes, void* dst, int64_t ld, int64_t rows,
                       hipStream_t s) {
  const dim3 grid((uint32_t)((ld / 16 + 255) / 256), (uint32_t)(rows < 32768 ? rows : 32768));
  hipLaunchKernelGGL(pack_kernel, grid, dim3(256), 0, s, (const char*)src, lds, bytes, (char*)dst, ld, rows);
  return hipGetLastError();
}

}  // namespace l8
}  // namespace muon
