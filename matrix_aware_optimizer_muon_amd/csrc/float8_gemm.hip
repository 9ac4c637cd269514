// Products of the 8-bit floating-point layer, dense or grouped by expert:
//   Y  = x w^T      e4m3 MFMA, scales in the instruction    (FWD)
//                   or bf16 MFMA on widened fragments       (FWD32)
//   dX = dY w       bf16 MFMA                               (DX)
//   dW = dY^T x     bf16 MFMA                               (DW)
// all as C[q][p] = sum_k P(p, k) Q(q, k) with p contiguous in C.  P takes the
// MFMA's A side, so each lane ends with four consecutive columns of one row.
//
// Scales are powers of two for 128 values of K, two stages of FWD.  FWD hands
// them to the MFMA, which adds exponents: no scaled copy, no instruction of its
// own.  Its sums inside eight products are cut 13 bits under the largest one's
// power of two (seen in-bounds on the card for both shapes and for the older
// e4m3 MFMAs alike; the accumulator itself is fp32), so results in fp32 go through FWD32, and so do
// few rows, which wait for memory either way.  Elsewhere a value times its
// scale is widened to bf16, exactly (4 significant bits), two per instruction.
//
// Grouped: rows of x and dy are sorted by expert, and only the device knows
// where an expert ends.  The launch holds as many workgroups as the rows can
// need however they fall (one partly filled tile per expert); each finds its
// expert by a scan of the ends, and the ones left over zero the rows that
// belong to none.
//
// Ragged sizes: output rows and columns past the end re-read the last valid
// one and are not stored; K past the end is zero on both sides, so no value of
// a masked place (not even NaN) enters a sum.
#include <algorithm>

#include "common.hpp"
#include "float8.h"
#include "mm_tiles.hpp"

namespace muon {
namespace f8 {

using namespace l8;

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The scale that a byte stands for (255: NaN, as in e8m0).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four e4m3 values times a scale, as bf16: exact, two per instruction.  (A
// scale's sign and fraction are not looked at; scale 2^-127 included.)
__device__ __forceinline__ uint2 widen4(uint32_t v, float scale) {
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, true)));
}
__device__ __forceinline__ u32x4 widen8(uint32_t a, uint32_t b, float scale) {
  const uint2 x = widen4(a, scale), y = widen4(b, scale);
  return u32x4{x.x, x.y, y.x, y.y};
}

__device__ __forceinline__ void mfma(const u32x4& a, const u32x4& b, f32x4& c) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The first n bytes of a chunk, zeros behind.
__device__ __forceinline__ u32x4 first(u32x4 v, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    v[i] &= left >= 4 ? ~0u : left > 0 ? (1u << (8 * left)) - 1 : 0u;
  }
  return v;
}

// Where row tile u lies: its expert, that one's rows [lo, lo + rows) and the
// number of row tiles ahead of it.  Each lane looks at an expert; an end
// outside [0, total] is moved there, and one before its start gives no rows.
// False past the last tile (`ahead` then counts them all).
struct Part {
  int expert, lo, rows, ahead;
};
template <int T>
__device__ __forceinline__ bool find_part(const int* ends, int experts, int total, int u, Part& f) {
  const int lane = threadIdx.x & 63;
  int ahead = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    const int e = e0 + lane;
    int hi = e < experts ? ends[e] : 0, lo = e > 0 && e < experts ? ends[e - 1] : 0;
    hi = min(max(hi, 0), total);
    lo = min(max(lo, 0), total);
    const int rows = max(hi - lo, 0), tiles = (rows + T - 1) / T;
    int upto = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(upto, off, 64);
      upto += lane >= off ? v : 0;
    }
    const int all = __builtin_amdgcn_readlane(upto, 63);
    if (u < ahead + all) {
      const int l = __builtin_ctzll(__ballot(ahead + upto > u));
      f.expert = e0 + l;
      f.lo = __builtin_amdgcn_readlane(lo, l);
      f.rows = __builtin_amdgcn_readlane(rows, l);
      f.ahead = ahead + __builtin_amdgcn_readlane(upto - tiles, l);
      return true;
    }
    ahead += all;
  }
  f.ahead = ahead;
  return false;
}

// Rows from the last end on, by the z-th of n workgroups.
__device__ __forceinline__ void zero_rows(const MmParams& p, int z, int n) {
  const int from = min(max(p.ends[p.experts - 1], 0), p.nq);
  const float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  MmParams o = p;
  o.accumulate = false;
  for (int64_t r = (int64_t)from + z; r < p.nq; r += n)
    for (int64_t c = (int64_t)threadIdx.x * 4; c < p.np; c += (int64_t)blockDim.x * 4)
      put4(o, r * p.ldo + c, (int)min((int64_t)4, p.np - c), v);
}

// P of the gradients: e4m3 rows along K, 16 columns (8 of 64-wide tiles) per
// lane and stage, widened with their scale on the way through registers into
// LDS.  SQUARE: a scale per 128 rows (weights), else per row.  A chunk lies
// within 128 columns, and within the readable part of its row.
template <bool SQUARE, int T, int NT>
struct WideOperand {
  static constexpr int CH = T == 64 ? 8 : 16;
  static constexpr int CPR = T / CH;
  static_assert(KROWS * CPR == NT, "one chunk per lane");
  static constexpr int PIECES = CH / 4;
  struct Regs {
    u32x4 v;
    uint32_t scale;
  };
  struct Wide {
    uint32_t d[CH / 2];
  };
  const char* src;
  const uint8_t* scale;
  int64_t ld;
  int lds, kd, row, col;

  __device__ __forceinline__ void init(const char* base, int64_t ld_, const uint8_t* sc, int lds_, int col0, int np,
                                       int kd_, int tid) {
    row = tid / CPR;
    col = tid % CPR;
    ld = ld_;
    lds = lds_;
    kd = kd_;
    const int c = min(col0 + col * CH, (np - 1) & ~(CH - 1));
    src = base + c;
    scale = sc + c / kBlock;
  }
  // CUT: some of the stage's rows may lie past the end, where the last one is read.
  template <bool CUT>
  __device__ __forceinline__ void load(Regs& r, int ks) const {
    int k = ks * KROWS + row;
    if (CUT) k = min(k, kd - 1);
    __builtin_memcpy(&r.v, src + (int64_t)k * ld, CH);
    r.scale = scale[(int64_t)(SQUARE ? k / kBlock : k) * lds];
  }
  // Piece q of a stage's way into LDS.
  template <bool CUT>
  __device__ __forceinline__ void store(const Regs& r, Wide& w, char* lds_at, int stage, int ks, int q) const {
    uint32_t b = r.v[q];
    if (CUT) b = ks * KROWS + row < kd ? b : 0u;
    // (opaque: see the waits of the 8-bit integer layer's operands; the bytes
    // are taken apart here, not at the load)
    asm("" : "+v"(b));
    // (a scale of NaN past the end would make NaN of the zeros)
    const float f = scale_of(CUT && ks * KROWS + row >= kd ? 127u : r.scale);
    const uint2 d = widen4(b, f);
    w.d[2 * q] = d.x;
    w.d[2 * q + 1] = d.y;
    if (q == PIECES - 1) {
      // swz_k is even, so a lane's two chunks stay side by side
      const int at = stage + row * (T * 2) + ((col * (CH / 8) ^ swz_k<T>(row)) << 4);
      *(u32x4*)(lds_at + at) = u32x4{w.d[0], w.d[1], w.d[2], w.d[3]};
      if constexpr (CH == 16) *(u32x4*)(lds_at + at + 16) = u32x4{w.d[4], w.d[5], w.d[6], w.d[7]};
    }
  }
};

// Fragments of FWD: 32 rows, each lane with 32 of a row's 64 bytes.
struct Reader32 {
  int lo, hi;
  __device__ __forceinline__ void init(int ring, int first_row, int lane) {
    const int r = first_row + (lane & 31), c = (lane >> 5) * 2;
    lo = ring + r * KB + ((c ^ swz_r(r)) << 4);
    hi = ring + r * KB + (((c + 1) ^ swz_r(r)) << 4);
    asm("" : "+v"(lo), "+v"(hi));  // (as in Reader)
  }
  __device__ __forceinline__ u32x4 get(const char* lds, int stage, int f, int half) const {
    return *(const u32x4*)(lds + (stage + (half ? hi : lo) + f * 32 * KB));
  }
};

template <int KIND> struct Frag { typedef u32x4 type; };
template <> struct Frag<FWD> { typedef i32x8 type; };

// What a kernel writes to (put4, put8).
struct Out {
  void* out;
  int obf16, accumulate;
};

// One tile (or a contraction range of one) per workgroup; G groups of waves
// share its K, each with LDS rings of its own, and join their sums through LDS.
template <int KIND, bool GROUPED, int T, int G>
__global__ void __launch_bounds__(64 * waves_of(T) * G, T == 128 && G == 1 ? 2 : 1) mm_kernel(const MmParams p) {
  constexpr bool FORWARD = KIND == FWD || KIND == FWD32;
  constexpr bool PREG = !FORWARD, QKM = KIND == DW;
  constexpr int FR = KIND == FWD ? 32 : 16;        // rows and columns of an MFMA
  constexpr int QUADS = FR == 32 ? 4 : 1;          // a lane's runs of four columns in it
  constexpr int NW = waves_of(T);                  // waves of a group
  constexpr int WQ = NW / 2;                       // waves along Q (2 along P)
  constexpr int FP = T / 2 / FR, FQ = T / WQ / FR; // MFMA blocks per wave
  constexpr int H = (FP + 1) / 2;                  // block rows of a stage's first half
  typedef typename Frag<KIND>::type F;
  typedef std::conditional_t<FR == 32, f32x16, f32x4> Acc;
  typedef DmaOperand<false, T, NW, KIND == FWD> DmaP;
  typedef DmaOperand<QKM, T, NW, KIND == FWD> DmaQ;
  typedef WideOperand<KIND == DX, T, 64 * NW> RegP;
  constexpr int DP = PREG ? 0 : DmaP::NDMA, DPS = DP + DmaQ::NDMA;
  constexpr int DB = DPS / 2, DA = DPS - DB;       // the two halves of a stage's instructions
  constexpr int OPB = T * KB;                      // one operand's stage in LDS
  constexpr int D = 4;                             // stages of a ring
  constexpr int RS = 2;                            // register sets in flight
  // (two objects: the compiler then knows that a write to one is no write to
  // the other)
  __shared__ __attribute__((aligned(1024))) char s_p[G * D * OPB];
  __shared__ __attribute__((aligned(1024))) char s_q[G * D * OPB];

  const int tid = threadIdx.x % (64 * NW), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = G > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / (64 * NW)) : 0;
  const int ring = group * D * OPB;                // the group's rings
  auto at = [&](int st) { return (st & (D - 1)) * OPB; };  // a stage in them
  const int wp = wave / WQ, wq = wave % WQ;
  const int q4 = lane >> 4, c16 = lane & 15;

  // This workgroup's tile, and its part of the operands.
  const char *P = p.P, *Q = p.Q;
  const uint8_t *scp = p.sp, *scq = p.sq;
  Out o = {p.out, p.obf16, p.accumulate};
  const int osize = p.obf16 ? 2 : 4;
  int nq = p.nq, kd = p.kd;
  const int tiles_p = (p.np + T - 1) / T;
  const int bid = (int)xcd_remap_chunked(blockIdx.x, gridDim.x, 32);
  int tile = bid, split = 0, splits = 1, tiles_q = (nq + T - 1) / T;
  if constexpr (GROUPED && KIND == DW) {
    const int per = tiles_p * tiles_q, e = bid / per;
    tile = bid - e * per;
    const int lo = e > 0 ? min(max(p.ends[e - 1], 0), kd) : 0;
    kd = max(min(max(p.ends[e], 0), kd) - lo, 0);
    P += lo * p.ldp;
    Q += lo * p.ldq;
    scp += (int64_t)lo * p.ldsp;
    o.out = (char*)o.out + e * p.stride_o * osize;
  } else if constexpr (GROUPED) {
    Part f;
    if (!find_part<T>(p.ends, p.experts, nq, bid / tiles_p, f)) {
      zero_rows(p, bid - f.ahead * tiles_p, (int)gridDim.x - f.ahead * tiles_p);
      return;
    }
    tile = bid - f.ahead * tiles_p;
    nq = f.rows;
    tiles_q = (nq + T - 1) / T;
    P += f.expert * p.stride_p;
    scp += f.expert * p.stride_sp;
    Q += f.lo * p.ldq;
    if constexpr (FORWARD) scq += (int64_t)f.lo * p.ldsq;
    o.out = (char*)o.out + f.lo * p.ldo * osize;
  } else {
    // The first `direct` tiles belong to one workgroup each, the others to
    // `splits` workgroups each, a range of K apiece.
    const int rest = tiles_p * tiles_q - p.direct;
    if (bid >= p.direct) {
      const int u = bid - p.direct;
      split = u / rest;
      tile = p.direct + u - split * rest;
      splits = p.splits;
    }
  }
  int tp, tq;
  full_tile_grouped(tile, tiles_p, tiles_q, 8, &tp, &tq);

  constexpr int KE = FORWARD ? 64 : 32;            // K elements per stage
  constexpr int EVEN = FORWARD ? 2 : 1;            // ranges hold whole blocks of scales
  const int full = kd / KE;
  const int nk = (kd + KE - 1) / KE;
  int k0 = 0, k1 = nk;
  if (splits > 1) {
    const int nb = (nk + EVEN - 1) / EVEN;
    k0 = (int)((int64_t)nb * split / splits) * EVEN;
    k1 = min(nk, (int)((int64_t)nb * (split + 1) / splits) * EVEN);
  }
  // stages per group, and this group's (the last ones may have fewer)
  const int most = ((k1 - k0 + G - 1) / G + EVEN - 1) / EVEN * EVEN;
  const int steps = G > 1 ? max(0, min(most, k1 - k0 - group * most)) : k1 - k0;
  k0 += group * most;
  const int kbytes = kd * (FORWARD ? 1 : 2);       // of a K-contiguous row
  const bool ragged = !QKM && kbytes % 16 != 0;    // its last chunk holds bytes that are not the row's

  Acc acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j)
#pragma unroll
      for (int e = 0; e < 4 * QUADS; ++e) acc[i][j][e] = 0.0f;

  // Quad g of acc[i][j] is columns FR i + qcol(g) .. +3 of row FR j + qrow of
  // the wave's part.
  const int qrow = lane % FR;
  auto qcol = [&](int g) { return FR == 32 ? 8 * g + 4 * (lane >> 5) : 4 * q4; };
  const int colt = wp * (T / 2), rowt = wq * (T / WQ);
  const int col0 = tp * T + colt, row0 = tq * T + rowt;

  if (steps > 0) {  // (an empty sum reads nothing)
    DmaP dp;
    DmaQ dq;
    RegP gp;
    if constexpr (PREG) gp.init(P, p.ldp, scp, p.ldsp, tp * T, p.np, kd, tid);
    else dp.init(P, p.ldp, tp * T, p.np, kd, kbytes, full, tid);
    dq.init(Q, p.ldq, tq * T, nq, kd, kbytes, full, tid);
    auto dma = [&](int q, int st) __attribute__((always_inline)) {  // instruction q of stage k0 + st
      if (q < DP) dp.load(q, s_p + ring + at(st), k0 + st, full, wave);
      else dq.load(q - DP, s_q + ring + at(st), k0 + st, full, wave);
    };
    // Scales of two stages: the wave's columns lie in one block of weights, its
    // rows have one each.  Asked for one trip ahead.
    const uint8_t* sp_at = scp;
    const uint8_t* sq_at[FQ];
    uint32_t sp1 = 0, sp2 = 0, sq1[FQ], sq2[FQ];
    auto scales = [&](int st) __attribute__((always_inline)) {
      sp1 = sp2;
      const int b = min((k0 + st) / 2, (kd - 1) / kBlock);
      sp2 = sp_at[b];
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        sq1[j] = sq2[j];
        sq2[j] = sq_at[j][b];
      }
    };
    if constexpr (FORWARD) {
      sp_at = scp + (int64_t)(min(col0, p.np - 1) / kBlock) * p.ldsp;
#pragma unroll
      for (int j = 0; j < FQ; ++j) sq_at[j] = scq + (int64_t)min(row0 + FR * j + qrow, nq - 1) * p.ldsq;
      scales(0);
    }
    typename RegP::Regs rp[RS];
    typename RegP::Wide wide;
    constexpr int PIECES = PREG ? RegP::PIECES : 0;
    Reader<PREG, T> fp;
    Reader<QKM, T> fq;
    Reader32 fp32, fq32;
    if constexpr (KIND == FWD) {
      fp32.init(ring, wp * (T / 2), lane);
      fq32.init(ring, wq * (T / WQ), lane);
    } else {
      fp.init(ring, wp * (T / 2), q4, c16);
      fq.init(ring, wq * (T / WQ), q4, c16);
    }
    // Fragment f of stage k0 + st.  Cut: the stage may be the last one, whose
    // last chunk holds what stands behind the row.
    auto chunk = [&](auto cut, u32x4 v, int st, int c) __attribute__((always_inline)) {
      if (decltype(cut)::value && ragged && k0 + st == full) return first(v, kbytes - full * KB - 16 * c);
      return v;
    };
    auto get = [&](auto cut, auto& r, auto& r32, const char* lds, int st, int f, bool km) __attribute__((always_inline)) {
      if constexpr (KIND == FWD) {
        const int c = (lane >> 5) * 2;
        const u32x4 lo = chunk(cut, r32.get(lds, at(st), f, 0), st, c);
        const u32x4 hi = chunk(cut, r32.get(lds, at(st), f, 1), st, c + 1);
        return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
      } else {
        const u32x4 v = r.get(lds, at(st), f);
        return km ? v : chunk(cut, v, st, q4);
      }
    };
    auto getp = [&](auto cut, int st, int f) __attribute__((always_inline)) { return get(cut, fp, fp32, s_p, st, f, PREG); };
    auto getq = [&](auto cut, int st, int f) __attribute__((always_inline)) { return get(cut, fq, fq32, s_q, st, f, QKM); };
    F fa[FP], fb0[FQ], fb1[FQ];
    // FWD32: fragments widened for the present stage
    u32x4 wa[2], wb[FQ][2];
    auto go = [&](int i, int j, const F* fb) __attribute__((always_inline)) {
      if constexpr (KIND == FWD) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[i], fb[j], acc[i][j], 0, 0, 0, (int)sp1, 0, (int)sq1[j]);
      } else if constexpr (KIND == FWD32) {
        if (i == 0) {
          wb[j][0] = widen8(fb[j][0], fb[j][1], scale_of(sq1[j]));
          wb[j][1] = widen8(fb[j][2], fb[j][3], scale_of(sq1[j]));
        }
        if (j == 0) {
          wa[0] = widen8(fa[i][0], fa[i][1], scale_of(sp1));
          wa[1] = widen8(fa[i][2], fa[i][3], scale_of(sp1));
        }
        mfma(wa[0], wb[j][0], acc[i][j]);
        mfma(wa[1], wb[j][1], acc[i][j]);
      } else {
        mfma(fa[i], fb[j], acc[i][j]);
      }
    };

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
    if constexpr (PREG) {
      // stages 0 .. RS + 1 in flight together; everything has landed before
      // the loop, so that the waits inside it only count the loop's own loads
      typename RegP::Regs rp0[2];
#pragma unroll
      for (int st = 0; st < 2; ++st) gp.template load<true>(rp0[st], k0 + st);
#pragma unroll
      for (int st = 0; st < RS; ++st) gp.template load<true>(rp[st], k0 + 2 + st);
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int q = 0; q < PIECES; ++q) gp.template store<true>(rp0[st], wide, s_p, ring + at(st), k0 + st, q);
      __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
    } else if (steps < D) {
      __builtin_amdgcn_s_waitcnt(wait_imm(0, 15));
    } else {
      __builtin_amdgcn_s_waitcnt(wait_imm((D - 2) * DPS + DA, 15));
    }
    barrier();
#pragma unroll
    for (int f = 0; f < H; ++f) fa[f] = getp(Cut<true>(), 0, f);
#pragma unroll
    for (int f = 0; f < FQ; ++f) fb0[f] = getq(Cut<true>(), 0, f);

    // A step, kt counting from k0, set = kt % RS.  Cut: near the end of the
    // sum; what lies past it is not loaded.
    auto step = [&](auto cut, int kt, int set, F* fb, F* fbn) __attribute__((always_inline)) {
      constexpr bool CUT = decltype(cut)::value;
#pragma unroll
      for (int j = 0; j < FQ; ++j) go(0, j, fb);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = H; f < FP; ++f) fa[f] = getp(cut, kt, f);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int N1 = (H - 1) * FQ, G1 = DB > 0 && N1 > DB ? N1 / (DB + (DB == 0)) : 1;
#pragma unroll
      for (int n = 0; n < N1; ++n) {
        go(1 + n / FQ, n % FQ, fb);
        if (DB > 0 && n % G1 == G1 - 1 && n / G1 < DB) {
          if (!CUT || kt + D - 1 < steps) dma(DA + n / G1, kt + D - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int q = N1 > 0 ? std::min(DB, N1 / G1) : 0; q < DB; ++q)
        if (!CUT || kt + D - 1 < steps) dma(DA + q, kt + D - 1);
      __builtin_amdgcn_sched_barrier(0);
      // This wave's DMAs of stage kt + 1 have landed ((D - 2) DPS later ones
      // may fly; other loads among them make the wait stricter), its LDS
      // writes of stage kt + 1 and its reads of stage kt are done.
      if (CUT && kt + D - 1 >= steps) __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
      else __builtin_amdgcn_s_waitcnt(wait_imm((D - 2) * DPS, 0));
      barrier();
#pragma unroll
      for (int f = 0; f < H; ++f) fa[f] = getp(cut, kt + 1, f);
#pragma unroll
      for (int f = 0; f < FQ; ++f) fbn[f] = getq(cut, kt + 1, f);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int N2 = (FP - H) * FQ, N2S = N2 > 0 ? N2 : 1, G2 = N2S > DA ? N2S / DA : 1;
      // pieces after each MFMA (several, where there are few MFMAs)
      constexpr int GP = N2S > PIECES ? N2S / (PIECES + 1) : 1, PB = (PIECES + N2S - 1) / N2S;
      auto piece = [&](int q) __attribute__((always_inline)) {
        if constexpr (PREG) gp.template store<CUT>(rp[set], wide, s_p, ring + at(kt + 2), k0 + kt + 2, q);
      };
#pragma unroll
      for (int n = 0; n < N2; ++n) {
        go(H + n / FQ, n % FQ, fb);
        if (n % G2 == G2 - 1 && n / G2 < DA && (!CUT || kt + D < steps)) dma(n / G2, kt + D);
        if (PIECES > 0 && n % GP == GP - 1) {
#pragma unroll
          for (int q = 0; q < PB; ++q)
            if (n / GP * PB + q < PIECES) piece(n / GP * PB + q);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int q = N2 > 0 ? std::min(DA, N2 / G2) : 0; q < DA; ++q)
        if (!CUT || kt + D < steps) dma(q, kt + D);
#pragma unroll
      for (int q = N2 > 0 ? std::min(PIECES, N2 / GP * PB) : 0; q < PIECES; ++q) piece(q);
      if constexpr (PREG) {
        if (!CUT || kt + 2 + RS < steps) gp.template load<CUT>(rp[set], k0 + kt + 2 + RS);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // Two steps per trip: the Q fragments and the register sets alternate
    // without copies, and the scales stay.  The trips whose loads stay before
    // the last stage come first and carry no checks.
    int kt = 0;
    auto trips = [&](auto cut, int end) __attribute__((always_inline)) {
      for (; kt + 1 < end; kt += 2) {
        if constexpr (FORWARD) scales(kt + 2);
        step(cut, kt, 0, fb0, fb1);
        step(cut, kt + 1, 1, fb1, fb0);
      }
    };
    int safe = min(steps, full - k0) - D;
    if constexpr (PREG) safe = min(safe, full - k0 - RS - 2);
    trips(Cut<false>(), safe);
    trips(Cut<true>(), steps);
    if (kt < steps) {
      if constexpr (FORWARD) scales(kt + 2);
      step(Cut<true>(), kt, 0, fb0, fb1);
    }
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));  // no load may land after the workgroup's LDS is given back
  }

  // A block's quads are finished by group b % G (b: the quad's number): j runs fastest.
  auto quad = [&](int i, int g, int j) __attribute__((always_inline)) {
    if constexpr (FR == 32) return f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    else return acc[i][j];
  };
  constexpr int NB = FP * QUADS * FQ;
  if constexpr (G > 1) {
    // a group's barriers: one ahead of the loop and one per step; then one
    // that ends all reads of the rings
    if (most > 0) {
      for (int i = steps > 0 ? steps : -1; i < most; ++i) barrier();
    }
    barrier();
    // The other groups leave a quad in LDS, lane by lane, and its own adds them
    // in their order.
    static_assert(NB % G == 0 && NB * (G - 1) * NW * 1024 <= G * D * OPB, "the join fits the ring");
    auto slot = [&](int b, int from) -> f32x4* {
      const int own = b % G;
      return (f32x4*)(s_p + (((b / G) * G + own) * (G - 1) + (from < own ? from : from - 1)) * (NW * 1024) + tid * 16);
    };
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b % G != group) *slot(b, group) = quad(b / FQ / QUADS, b / FQ % QUADS, b % FQ);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b % G == group) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (g != b % G) {
            const f32x4 v = *slot(b, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b / FQ / QUADS][b % FQ][b / FQ % QUADS * 4 + e] += v[e];
          }
      }
  }

  float* const part = p.part + ((int64_t)(tile - p.direct) * splits + split) * (T * T);
  if constexpr (T > 64) {
    // A lane's four columns are 16 bytes of a row FR rows apart from its
    // neighbours'.  FR rows of SC columns of the wave's part at a time go
    // through LDS, 16-byte chunks swapped within a row by the row's number,
    // and leave as whole runs of 128 bytes or more.  One loop over them, not
    // unrolled but for its first lines.
    constexpr int PT = T / 2, SC = FR == 32 && PT > 64 ? 64 : PT, NH = PT / SC, CPR = SC / 4;
    static_assert(NW * FR * SC * 4 * G <= G * D * OPB, "the staged rows fit a ring");
    static_assert(FQ % G == 0, "a row's quads are one group's");
    if constexpr (G == 1) barrier();  // no wave reads the rings any more
    const bool wide = splits == 1 && p.obf16;
    const int outc = wide ? lane % (SC / 8) * 8 : lane % (SC / 4) * 4, ch = outc / 4;
    char* const st = s_q + (group * NW + wave) * (FR * SC * 4);
    auto chunk = [&](int r, int c) { return st + r * (SC * 4) + ((c ^ (r & (CPR - 1))) << 4); };
#pragma clang loop unroll(disable)
    for (int it = G > 1 ? group : 0; it < FQ * NH; it += G) {  // it = h FQ + j
      const int jr = it % FQ, h = it / FQ;
#pragma unroll
      for (int b = 0; b < FQ * NH; ++b)
        if (b == it) {
#pragma unroll
          for (int i = b / FQ * (SC / FR); i < (b / FQ + 1) * (SC / FR); ++i)
#pragma unroll
            for (int g = 0; g < QUADS; ++g)
              *(f32x4*)chunk(qrow, (FR * (i - b / FQ * (SC / FR)) + qcol(g)) / 4) = quad(i, g, b % FQ);
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int r0 = row0 + FR * jr, c0 = h * SC + outc, n = p.np - (col0 + c0);
      if (!wide) {
        constexpr int RPI = 64 / CPR;  // rows per instruction
        int rr = lane / CPR;
#pragma unroll 4
        for (int i = 0; i < FR / RPI; ++i, rr += RPI) {
          const f32x4 v = *(const f32x4*)chunk(rr, ch);
          if (splits > 1) {
            *(f32x4*)(part + (rowt + FR * jr + rr) * T + colt + c0) = v;
          } else if (r0 + rr < nq && n > 0) {
            const float e[4] = {v[0], v[1], v[2], v[3]};
            put4<true>(o, (int64_t)(r0 + rr) * p.ldo + col0 + c0, n, e);
          }
        }
      } else {
        constexpr int RPI = 128 / CPR;
        int rr = lane / (CPR / 2);
#pragma unroll 2
        for (int i = 0; i < FR / RPI; ++i, rr += RPI) {
          const f32x4 v = *(const f32x4*)chunk(rr, ch), w = *(const f32x4*)chunk(rr, ch + 1);
          const float e[8] = {v[0], v[1], v[2], v[3], w[0], w[1], w[2], w[3]};
          if (r0 + rr < nq && n > 0) put8(o, (int64_t)(r0 + rr) * p.ldo + col0 + c0, n, e);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    static_assert(NB == G, "one quad per group");
    // quad `group`
    const int i = group / FQ / QUADS, g = group / FQ % QUADS, j = group % FQ;
    f32x4 a = quad(0, 0, 0);
#pragma unroll
    for (int b = 1; b < NB; ++b)
      if (b == group) a = quad(b / FQ / QUADS, b / FQ % QUADS, b % FQ);
    const int r = FR * j + qrow, c = FR * i + qcol(g), n = p.np - col0 - c;
    if (splits > 1) {
      *(f32x4*)(part + (rowt + r) * T + colt + c) = a;
    } else if (row0 + r < nq && n > 0) {
      const float e[4] = {a[0], a[1], a[2], a[3]};
      put4(o, (int64_t)(row0 + r) * p.ldo + col0 + c, n, e);
    }
  }
}

// C = the splits' partial sums added in order: blockIdx.y a split tile, four
// columns of a row per thread.
template <int T>
__global__ void __launch_bounds__(256) mm_sum_kernel(const MmParams p) {
  const int at = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
  const int tiles_p = (p.np + T - 1) / T, tiles_q = (p.nq + T - 1) / T;
  int tp, tq;
  full_tile_grouped(p.direct + (int)blockIdx.y, tiles_p, tiles_q, 8, &tp, &tq);
  const int r = tq * T + at / T, c = tp * T + at % T, n = p.np - c;
  if (r >= p.nq || n <= 0) return;
  const float* src = p.part + (int64_t)blockIdx.y * p.splits * (T * T) + at;
  f32x4 a = *(const f32x4*)src;
#pragma unroll 4
  for (int s = 1; s < p.splits; ++s) a += *(const f32x4*)(src + (int64_t)s * (T * T));
  const float v[4] = {a[0], a[1], a[2], a[3]};
  put4(p, (int64_t)r * p.ldo + c, n, v);
}

// Few rows of x, 16 QB of them against 16 rows of w: a workgroup's W waves take
// every W-th block of 128 of K, straight from memory into MFMA fragments (a
// row of w is read once; x comes from the caches), and the partial tiles are
// added through LDS.  Bound by the read of w.  blockIdx.y: which rows of x.
template <bool GROUPED, int QB, int W>
__global__ void __launch_bounds__(64 * W) few_kernel(const MmParams p) {
  __shared__ f32x4 s_part[W - 1][QB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q4 = lane >> 4, c16 = lane & 15;
  const int n0 = blockIdx.x * 16, k = p.kd;
  const char *P = p.P, *Q = p.Q;
  const uint8_t *scp = p.sp, *scq = p.sq;
  int lo = 0, t = p.nq, row0 = (int)blockIdx.y * 16 * QB;
  if constexpr (GROUPED) {
    Part f;
    if (!find_part<16 * QB>(p.ends, p.experts, p.nq, blockIdx.y, f)) {
      zero_rows(p, (int)(blockIdx.y - f.ahead) * gridDim.x + blockIdx.x, (int)(gridDim.y - f.ahead) * gridDim.x);
      return;
    }
    row0 = ((int)blockIdx.y - f.ahead) * 16 * QB;
    lo = f.lo;
    t = f.rows;
    P += f.expert * p.stride_p;
    scp += f.expert * p.stride_sp;
    Q += lo * p.ldq;
    scq += (int64_t)lo * p.ldsq;
  }
  const char* const wr = P + (int64_t)min(n0 + c16, p.np - 1) * p.ldp + q4 * 32;
  const uint8_t* const wsc = scp + (int64_t)(n0 / kBlock) * p.ldsp;
  const char* xr[QB];
  const uint8_t* xsc[QB];
#pragma unroll
  for (int j = 0; j < QB; ++j) {
    const int r = min(row0 + 16 * j + c16, t - 1);
    xr[j] = Q + (int64_t)r * p.ldq + q4 * 32;
    xsc[j] = scq + (int64_t)r * p.ldsq;
  }
  f32x4 acc[QB];
#pragma unroll
  for (int j = 0; j < QB; ++j) acc[j] = f32x4{0, 0, 0, 0};
  auto block = [&](auto cut, int s) __attribute__((always_inline)) {
    u32x4 a[2], b[QB][2];
    uint32_t sa, sb[QB];
    const int left = k - s * kBlock - q4 * 32;  // bytes of the row from the lane's first on
    auto load = [&](const char* r, u32x4 v[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a chunk past the end: the row's first 16 bytes, put to zero)
        const char* c = r + s * kBlock + h * 16;
        if (decltype(cut)::value) c = left > h * 16 ? c : r - q4 * 32;
        __builtin_memcpy(&v[h], c, 16);
      }
    };
    load(wr, a);
    sa = wsc[s];
#pragma unroll
    for (int j = 0; j < QB; ++j) {
      load(xr[j], b[j]);
      sb[j] = xsc[j][s];
    }
    if constexpr (decltype(cut)::value) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[h] = first(a[h], left - 16 * h);
#pragma unroll
        for (int j = 0; j < QB; ++j) b[j][h] = first(b[j][h], left - 16 * h);
      }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const u32x4 wa = widen8(a[h / 2][h % 2 * 2], a[h / 2][h % 2 * 2 + 1], scale_of(sa));
#pragma unroll
      for (int j = 0; j < QB; ++j)
        mfma(wa, widen8(b[j][h / 2][h % 2 * 2], b[j][h / 2][h % 2 * 2 + 1], scale_of(sb[j])), acc[j]);
    }
  };
  const int whole = k / kBlock;
  int s = wave;
#pragma unroll 2
  for (; s < whole; s += W) block(Cut<false>(), s);
  if (s == whole && k % kBlock) block(Cut<true>(), s);  // one wave takes the ragged last block
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < QB; ++j) s_part[wave - 1][j][lane] = acc[j];
  }
  __syncthreads();
  if (wave > 0) return;
  const int c = n0 + 4 * q4;
#pragma unroll
  for (int j = 0; j < QB; ++j) {
    f32x4 a = acc[j];
#pragma unroll
    for (int q = 0; q < W - 1; ++q) a += s_part[q][j][lane];
    const int r = row0 + 16 * j + c16;
    if (c < p.np && r < t) {
      const float v[4] = {a[0], a[1], a[2], a[3]};
      put4(p, (int64_t)(lo + r) * p.ldo + c, p.np - c, v);
    }
  }
}

template <int KIND>
hipError_t go_mm(const MmParams& p, hipStream_t s) {
  const int T = p.tile;
  const int64_t tp = (p.np + T - 1) / T, tq = (p.nq + T - 1) / T;
  int64_t blocks, rest = 0;
  if (!p.ends) {
    rest = tp * tq - p.direct;
    blocks = p.direct + rest * p.splits;
  } else if (KIND == DW) {
    blocks = tp * tq * p.experts;
  } else {
    // a partly filled tile per expert, and one workgroup per column for rows of none
    blocks = tp * (p.nq / T + std::min(p.experts, p.nq) + 1);
  }
  // (a launch has fewer than 2^32 threads; outputs that need more pass any memory)
  const int threads = 64 * waves_of(T) * p.groups;
  if (blocks > 0xffffffffll / threads || rest < 0) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)blocks);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, p);
    return hipGetLastError();
  };
  hipError_t e = hipErrorInvalidValue;
  if (p.ends) {
    if (T == 256 && p.groups == 1) {
      if constexpr (KIND != FWD32) e = go(mm_kernel<KIND, true, 256, 1>);
    } else if (T == 128 && p.groups == 1) {
      e = go(mm_kernel<KIND, true, 128, 1>);
    }
    return e;
  }
  if (T == 256 && p.groups == 1) {
    if constexpr (KIND != FWD32) e = go(mm_kernel<KIND, false, 256, 1>);
  } else if (T == 128 && p.groups == 1) {
    e = go(mm_kernel<KIND, false, 128, 1>);
  } else if (T == 128 && p.groups == 2) {
    e = go(mm_kernel<KIND, false, 128, 2>);
  } else if (T == 64 && p.groups == 4) {
    e = go(mm_kernel<KIND, false, 64, 4>);
  }
  if (e != hipSuccess || rest == 0 || p.splits == 1) return e;
  const dim3 sums((uint32_t)(T * T / 1024), (uint32_t)rest);
  auto sum = [&](auto kernel) { hipLaunchKernelGGL(kernel, sums, dim3(256), 0, s, p); };
  if (T == 256) sum(mm_sum_kernel<256>);
  else if (T == 128) sum(mm_sum_kernel<128>);
  else sum(mm_sum_kernel<64>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mm(const MmParams& p, Kind kind, hipStream_t s) {
  switch (kind) {
    case FWD: return go_mm<FWD>(p, s);
    case FWD32: return go_mm<FWD32>(p, s);
    case DX: return go_mm<DX>(p, s);
    case DW: return go_mm<DW>(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_few(const MmParams& p, int rows, hipStream_t s) {
  const int64_t n = (p.np + 15) / 16;
  const int64_t y = p.ends ? p.nq / rows + std::min(p.experts, p.nq) + 1 : (p.nq + rows - 1) / rows;
  if (y > 65535 || n * y > 0xffffffffll / 512) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)n, (uint32_t)y);
  auto go = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), 0, s, p);
    return hipGetLastError();
  };
  if (p.ends) {
    if (rows == 16) return go(few_kernel<true, 1, 8>, 8);
    if (rows == 32) return go(few_kernel<true, 2, 8>, 8);
    return go(few_kernel<true, 4, 8>, 8);
  }
  if (rows == 16) return go(few_kernel<false, 1, 8>, 8);
  if (rows == 32) return go(few_kernel<false, 2, 8>, 8);
  return go(few_kernel<false, 4, 8>, 8);
}

}  // namespace f8
}  // namespace muon
