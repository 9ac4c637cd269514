// Forward products of the 8-bit floating-point layer, dense or grouped by
// expert: Y = x w^T as C[q][p] = sum_k P(p, k) Q(q, k) with P = w, Q = x, p
// contiguous in C.  P takes the MFMA's A side, so each lane ends with four
// consecutive columns of one row.
//
// Scales are powers of two for 128 values of K: a stage.  FWD hands them to the
// e4m3 MFMA, which adds exponents: no scaled copy, no instruction of its own.
// Its sums inside eight products are cut 13 bits under the largest one's power
// of two (seen on the card for both of its shapes and for the older e4m3 MFMAs
// alike; the accumulator itself is fp32), so results in fp32 go through FWD32,
// which widens fragments to bf16 with their scale on the way from LDS (exactly,
// but at the ends of bf16's range: widen4), and so do few rows, which wait for
// memory either way.
//
// Ragged sizes: output rows and columns past the end re-read the last valid one
// and are not stored; K past the end is zero on both sides, so no value of a
// masked place (not even NaN) enters a sum.
#include <algorithm>

#include "float8_tiles.hpp"

namespace muon {
namespace f8 {

namespace {

constexpr int SB = 128;  // bytes of K per stage and row: a cache line, a block of scales
constexpr int D = 2;     // stages of a ring

// 16-byte chunks of a stage's row are swapped by the row: reads of 16
// consecutive rows of one chunk fall on the 16 places of two rows.
__device__ __forceinline__ int swz_s(int row) { return (row >> 1) & 7; }

// One operand's T rows by direct global->LDS loads, a whole line of a row per
// eight lanes.
template <int T, int NW>
struct RowOperand {
  static constexpr int NDMA = T * SB / 1024 / NW;  // 1-KB instructions per wave and stage
  Rsrc base;            // the tile's first row
  uint32_t off[NDMA];   // the lane's place in the first stage
  int kbytes;

  __device__ __forceinline__ void init(const char* b, int64_t ld, int row0, int count, int kd, int wave, int lane) {
    base = rsrc(b + row0 * ld);
    kbytes = kd;
#pragma unroll
    for (int i = 0; i < NDMA; ++i) {
      const int r = (wave * NDMA + i) * 8 + lane / 8;
      // (a row distance is at most 2^23, and with it K)
      off[i] = (uint32_t)min(r, count - 1 - row0) * (uint32_t)ld + (((lane & 7) ^ swz_s(r)) << 4);
    }
  }
  // Instruction i of stage ks; if not WHOLE, chunks past the row's end are zeros.
  template <Mode M>
  __device__ __forceinline__ void load(int i, char* stage, int ks, int wave, int lane) const {
    uint32_t at = off[i];
    if (M != WHOLE) {
      const int c = (lane & 7) ^ swz_s((wave * NDMA + i) * 8 + lane / 8);
      at = ks * SB + c * 16 < kbytes ? at : kPast;
    }
    dma16(base, stage + (wave * NDMA + i) * 1024, at, ks * SB);
  }
};

// Fragments of half h of a stage.  FWD: 32 rows, a lane has 32 of the half's 64
// bytes; FWD32: 16 rows, 16 bytes.
template <bool R32> struct HalfReader;
template <> struct HalfReader<true> {
  typedef i32x8 F;
  int row, c, sw;
  __device__ __forceinline__ void init(int ring, int first_row, int lane) {
    const int r = first_row + (lane & 31);
    row = ring + r * SB;
    c = (lane >> 5) * 2;
    sw = swz_s(r);
    asm("" : "+v"(row));
  }
  __device__ __forceinline__ F get(const char* lds, int stage, int f, int h) const {
    const u32x4 a = *(const u32x4*)(lds + (stage + row + f * 32 * SB + (((4 * h + c) ^ sw) << 4)));
    const u32x4 b = *(const u32x4*)(lds + (stage + row + f * 32 * SB + (((4 * h + c + 1) ^ sw) << 4)));
    return F{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  }
};
template <> struct HalfReader<false> {
  typedef u32x4 F;
  int row, c, sw;
  __device__ __forceinline__ void init(int ring, int first_row, int lane) {
    const int r = first_row + (lane & 15);
    row = ring + r * SB;
    c = lane >> 4;
    sw = swz_s(r);
    asm("" : "+v"(row));
  }
  __device__ __forceinline__ F get(const char* lds, int stage, int f, int h) const {
    return *(const u32x4*)(lds + (stage + row + f * 16 * SB + (((4 * h + c) ^ sw) << 4)));
  }
};

// One tile (or a contraction range of one) of T columns and TQ rows by G groups of NW
// waves, which share its K, each with rings of its own, and join their sums
// through LDS.
//
// A ring holds two stages.  A stage has two halves of N blocks of MFMAs each,
// 2 N slots.  During the first half the fragments of the second are read; a
// barrier then says that all waves have, and the stage after the next goes into
// the buffer; later a second one says that the next stage stands in LDS, and the
// fragments of its first half are read behind the last MFMAs.  Nothing that a
// slot needs is asked for less than several slots before, so a wave that has its
// SIMD to itself keeps the matrix core fed.
template <int KIND, int T, int TQ, int G, int NW>
__device__ __forceinline__ void forward_tile(const MmParams& p, const Work& w, char* s_p, char* s_q) {
  constexpr bool R32 = KIND == FWD;
  constexpr int FR = R32 ? 32 : 16;                 // rows and columns of an MFMA
  constexpr int WQ = NW / 2;                        // waves along Q (2 along P)
  constexpr int FP = T / 2 / FR, FQ = TQ / WQ / FR; // MFMA blocks per wave
  typedef RowOperand<T, NW> OpP;
  typedef RowOperand<TQ, NW> OpQ;
  typedef HalfReader<R32> Rd;
  typedef typename Rd::F F;
  typedef std::conditional_t<R32, f32x16, f32x4> Acc;
  constexpr int OPB = T * SB;                       // room of one operand's stage in LDS

  const int tid = threadIdx.x % (64 * NW), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = G > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / (64 * NW)) : 0;
  const int ring = group * D * OPB;                 // the group's rings
  auto at = [&](int st) { return (st & (D - 1)) * OPB; };  // a stage in them
  const int wp = wave / WQ, wq = wave % WQ;
  const int kd = w.kd, nq = w.at.nq, tp = w.at.tp, tq = w.at.tq, split = w.at.split, splits = w.at.splits;

  const int full = kd / SB, nk = (kd + SB - 1) / SB;
  int k0 = 0, k1 = nk;
  if (splits > 1) {
    k0 = (int)((int64_t)nk * split / splits);
    k1 = (int)((int64_t)nk * (split + 1) / splits);
  }
  // stages per group, and this group's (the last ones may have fewer)
  const int most = (k1 - k0 + G - 1) / G;
  const int steps = G > 1 ? max(0, min(most, k1 - k0 - group * most)) : most;
  k0 += group * most;
  const bool ragged = kd % 16 != 0;                // a row's last chunk holds bytes that are not its own

  Acc acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j)
#pragma unroll
      for (int e = 0; e < (R32 ? 16 : 4); ++e) acc[i][j][e] = 0.0f;

  if (steps > 0) {  // (an empty sum reads nothing)
    OpP dp;
    OpQ dq;
    dp.init(w.P, p.ldp, tp * T, p.np, kd, wave, lane);
    dq.init(w.Q, p.ldq, tq * T, nq, kd, wave, lane);
    constexpr int DPS = OpP::NDMA + OpQ::NDMA;             // a stage's instructions
    auto dma = [&](auto in, int q, int st) __attribute__((always_inline)) {  // instruction q of stage k0 + st
      constexpr Mode M = decltype(in)::mode;
      if (q < OpP::NDMA) dp.template load<M>(q, s_p + ring + at(st), k0 + st, wave, lane);
      else dq.template load<M>(q - OpP::NDMA, s_q + ring + at(st), k0 + st, wave, lane);
    };
    // Scales: the wave's columns lie in one block of weights, its rows have one
    // each; four stages' at a time (a gather of a byte per row and stage took 6 %
    // of a long sum), asked for four stages ahead.  The present stage's is the
    // lowest byte.
    const int sp_row = (min(tp * T + wp * (T / 2), p.np - 1) / kBlock) * p.ldsp;
    const uint8_t* sq_at[FQ];
#pragma unroll
    for (int j = 0; j < FQ; ++j)
      sq_at[j] = w.scq + (int64_t)min(tq * T + wq * (TQ / WQ) + FR * j + lane % FR, nq - 1) * p.ldsq;
    struct Scales {
      uint32_t p, q[FQ];
    } now, coming, four1, four2;
    // Blocks b .. b + 3 of a row of nk >= 4, by a dword that ends inside it: to be
    // shifted by `shift` when it is due (at the load, that would wait for it).
    int shift = 0;
    auto ask = [&](int b) __attribute__((always_inline)) {
      const int from = min(b, nk - 4);
      shift = 8 * min(b - from, 3);
      __builtin_memcpy(&four2.p, w.scp + sp_row + from, 4);
#pragma unroll
      for (int j = 0; j < FQ; ++j) __builtin_memcpy(&four2.q[j], sq_at[j] + from, 4);
    };
    auto take = [&]() __attribute__((always_inline)) {
      four1.p = four2.p >> shift;
#pragma unroll
      for (int j = 0; j < FQ; ++j) four1.q[j] = four2.q[j] >> shift;
    };
    // ahead of stage s: the dwords that stage s + 1's scales come from
    auto refill = [&](int s) __attribute__((always_inline)) {
      if (s % 4 == 3 && nk > 4) {
        take();
        ask(k0 + s + 5);
      }
    };
    auto extract = [&](Scales& to) __attribute__((always_inline)) {
      to.p = four1.p & 255;
      four1.p >>= 8;
#pragma unroll
      for (int j = 0; j < FQ; ++j) {
        to.q[j] = four1.q[j] & 255;
        four1.q[j] >>= 8;
      }
    };
    if (nk >= 4) {
      ask(k0);
      take();
      if (nk > 4) ask(k0 + 4);
    } else {  // short rows, byte by byte
      auto bytes = [&](const uint8_t* row) __attribute__((always_inline)) {
        const uint32_t v = row[0] | (uint32_t)row[min(1, nk - 1)] << 8 | (uint32_t)row[min(2, nk - 1)] << 16;
        return v >> (8 * k0);
      };
      four1.p = bytes(w.scp + sp_row);
#pragma unroll
      for (int j = 0; j < FQ; ++j) four1.q[j] = bytes(sq_at[j]);
    }
    extract(now);

    Rd rp, rq;
    rp.init(ring, wp * (T / 2), lane);
    rq.init(ring, wq * (TQ / WQ), lane);
    // Zeros behind the rows' ends in the last stage, which stands in LDS (a
    // barrier has said so).  All waves call it.
    auto zero_tail = [&]() __attribute__((always_inline)) {
      if (tid < T) {
        const int left = kd - full * SB;
        const int b = ring + at(full - k0) + tid * SB + ((left / 16 ^ swz_s(tid)) << 4);
        *(u32x4*)(s_p + b) = first(*(const u32x4*)(s_p + b), left % 16);
        *(u32x4*)(s_q + b) = first(*(const u32x4*)(s_q + b), left % 16);
      }
      __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
      barrier();
    };
    // The schedule (see `stage`): fragments read ahead of a stage, slots that
    // read, the barriers' slots, DMAs that are out at the second one.
    constexpr int N = FP * FQ, R1 = N > 2 ? N / 2 : 1, B1 = N > 4 ? N - N / 4 - 2 : N > 1 ? N - 1 : 1;
    constexpr int B2 = N > 4 ? N + N / 8 : N > 1 ? 2 * N - 2 : 1, DE = 2 * N, RE = N > 4 ? 2 * N - N / 4 : 2 * N;
    constexpr int OUT = ((B2 - B1) * DPS + DE - B1 - 1) / (DE - B1);  // DMAs issued ahead of B2
    static_assert(R1 <= B1 && B1 <= B2 && B2 < RE && RE <= 2 * N, "in this order");
    F fa[2][FP], fb[2][FQ];
    // FWD32: fragments widened for the present half
    u32x4 wa[2], wb[FQ][2];
    auto go = [&](int h, int i, int j, const Scales& sc) __attribute__((always_inline)) {
      if constexpr (R32) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[h][i], fb[h][j], acc[i][j], 0, 0, 0, (int)sc.p, 0,
                                                                    (int)sc.q[j]);
      } else {
        if (i == 0) {
          wb[j][0] = widen8(fb[h][j][0], fb[h][j][1], scale_of(sc.q[j]));
          wb[j][1] = widen8(fb[h][j][2], fb[h][j][3], scale_of(sc.q[j]));
        }
        if (j == 0) {
          wa[0] = widen8(fa[h][i][0], fa[h][i][1], scale_of(sc.p));
          wa[1] = widen8(fa[h][i][2], fa[h][i][3], scale_of(sc.p));
        }
        mfma(wa[0], wb[j][0], acc[i][j]);
        mfma(wa[1], wb[j][1], acc[i][j]);
      }
    };
    // the fragments of a half, in the order of their use
    auto read = [&](int st, int h, int i) __attribute__((always_inline)) {
      if (i == 0) fa[h][0] = rp.get(s_p, at(st), 0, h);
      else if (i <= FQ) fb[h][i - 1] = rq.get(s_q, at(st), i - 1, h);
      else fa[h][i - FQ] = rp.get(s_p, at(st), i - FQ, h);
    };

#pragma unroll
    for (int st = 0; st < D; ++st)
      if (st < steps) {
#pragma unroll
        for (int q = 0; q < DPS; ++q) dma(In<CUT>(), q, st);
      }
    if (steps < D) __builtin_amdgcn_s_waitcnt(wait_imm(0, 15));
    else __builtin_amdgcn_s_waitcnt(wait_imm(DPS, 15));
    barrier();
#pragma unroll
    for (int i = 0; i < FP + FQ; ++i) read(0, 0, i);

    // Slots of a stage: the second half's fragments are read up to R1; ahead of
    // B1 a barrier says that all waves have read the stage, and the DMA of stage
    // s + 2 goes out from there to the end (the L1 takes 16 cycles for each of
    // the waves' instructions: they need the room); ahead of B2 a barrier says
    // that the next stage stands, and the fragments of its first half are read
    // from there to RE.
    auto stage = [&](auto in, int s) __attribute__((always_inline)) {
      constexpr Mode M = decltype(in)::mode;
      refill(s);
      // runs the items i of `items` that fall on the n-th of `slots`
      auto share = [](int n, int slots, int items, auto f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < items && i * slots / items == n) f(i);
      };
#pragma unroll
      for (int n = 0; n < 2 * N; ++n) {
        if (n == B1) {
          __builtin_amdgcn_s_waitcnt(wait_imm(63, 0));
          barrier();
        }
        if (n == B2) {
          // (the DMAs of stage s + 2 that are out may fly; scales are older)
          __builtin_amdgcn_s_waitcnt(wait_imm(M == DRAIN ? 0 : OUT, 15));
          barrier();
        }
        go(n / N, n % N / FQ, n % FQ, now);
        if (n == N / 2) extract(coming);
        if (n < R1) share(n, R1, FP + FQ, [&](int i) __attribute__((always_inline)) { read(s, 1, i); });
        if (M != DRAIN && n >= B1) share(n - B1, DE - B1, DPS, [&](int q) __attribute__((always_inline)) { dma(in, q, s + 2); });
        if (n >= B2 && n < RE) share(n - B2, RE - B2, FP + FQ, [&](int i) __attribute__((always_inline)) { read(s + 1, 0, i); });
        __builtin_amdgcn_sched_barrier(0);
      }
      now = coming;
    };
    int s = 0;
    for (const int whole = min(steps, full - k0) - 2; s < whole; ++s) stage(In<WHOLE>(), s);
    for (; s < steps - 2; ++s) stage(In<CUT>(), s);
    for (; s < steps; ++s) {
      if (ragged && k0 + s == full) {
        zero_tail();
#pragma unroll
        for (int i = 0; i < FP + FQ; ++i) read(s, 0, i);  // (again)
      }
      stage(In<DRAIN>(), s);
    }
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));  // no load may land after the workgroup's LDS is given back
  }

  if constexpr (G > 1) {
    // a group's barriers: one ahead of the loop, two per stage and one ahead of
    // the ragged one
    if (most > 0) {
      const bool had = steps > 0 && ragged && full >= k0 && full < k0 + steps;
      for (int i = steps > 0 ? 2 * steps : -1; i < 2 * most + (ragged && !had ? 1 : 0); ++i) barrier();
    }
  }
  barrier();  // no wave reads the rings any more
  finish_tile<FR, T, TQ, 2, G, NW, G * D * OPB>(acc, p, w.o, w.at, group, tid, s_p, s_q);
}

// A workgroup per tile.  An expert's last row tile of at most 128 rows is computed
// as one of 128: 64 experts of 128 rows, 2816 x 2048, 107 -> 89 us.
//
// Bound by the matrix cores where there are many rows: 8192^3 takes 381 to 397 us
// (2.8 PFLOP/s), 4096 x 18944 x 3584 takes 224 to 241 by card (2.4), 63 % busy at 2.1
// GHz, in 4.6 rounds of tiles of 256, each with 11 us before its first and behind its last
// stage.  128-wide tiles read LDS twice as often per product (0.91 us a stage of
// two tiles against 1.39 of one with four times their size), and start and end
// under each other.
template <int KIND, bool GROUPED, int T, int G, int NW>
__global__ void __launch_bounds__(64 * NW * G, T == 128 && G == 1 ? 2 : 1) forward_kernel(const MmParams p) {
  __shared__ __attribute__((aligned(1024))) char s_p[G * D * T * SB];
  __shared__ __attribute__((aligned(1024))) char s_q[G * D * T * SB];

  // This workgroup's tile, and its part of the operands.
  const char *P = p.P, *Q = p.Q;
  const uint8_t *scp = p.sp, *scq = p.sq;
  Out o = {p.out, p.obf16, 0};
  int nq = p.nq;
  const int kd = p.kd, tiles_p = (p.np + T - 1) / T;
  const int bid = (int)xcd_remap_chunked(blockIdx.x, gridDim.x, 32);
  int tile = bid, split = 0, splits = 1, tiles_q = (nq + T - 1) / T;
  if constexpr (GROUPED) {
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
    scq += (int64_t)f.lo * p.ldsq;
    o.out = (char*)o.out + f.lo * p.ldo * (p.obf16 ? 2 : 4);
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

  const Work w = {P, Q, scp, scq, o, kd, {tile, split, splits, tp, tq, nq}};
  if constexpr (GROUPED && T == 256)
    if (nq - tq * T <= T / 2) return forward_tile<KIND, T, T / 2, G, NW>(p, w, s_p, s_q);
  forward_tile<KIND, T, T, G, NW>(p, w, s_p, s_q);
}

// Few rows of x, 16 QB of them against 16 rows of w: a workgroup's W waves take
// every W-th block of 128 of K, straight from memory into MFMA fragments (a
// row of w is read once; x comes from the caches), and the partial tiles are
// added through LDS.  Bound by the read of w: 18944 x 3584 in 13.2 us for one
// row, 5.1 TB/s.  blockIdx.y: which rows of x.
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
  // One block of 128 of K at a time: with more in flight per wave, fewer waves
  // fit (four: 13.3 -> 15.0 us for one row against 18944 x 3584, 34 -> 44 for 64
  // rows of 64 experts).  CUT: the ragged one.
  auto block = [&](auto cut, int s) __attribute__((always_inline)) {
    constexpr bool CUT = decltype(cut)::value;
    u32x4 a[2], b[QB][2];
    uint32_t sb[QB];
    const int left = k - s * kBlock - q4 * 32;  // bytes of the row from the lane's first on
    auto load = [&](const char* r, u32x4 v[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a chunk past the end: the row's first 16 bytes, put to zero)
        const char* c = r + s * kBlock + h * 16;
        if (CUT) c = left > h * 16 ? c : r - q4 * 32;
        __builtin_memcpy(&v[h], c, 16);
      }
    };
    load(wr, a);
    const uint32_t sa = wsc[s];
#pragma unroll
    for (int j = 0; j < QB; ++j) {
      load(xr[j], b[j]);
      sb[j] = xsc[j][s];
    }
    if constexpr (CUT) {
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
hipError_t go_forward(const MmParams& p, hipStream_t s) {
  const int T = p.tile;
  const int64_t tp = (p.np + T - 1) / T, tq = (p.nq + T - 1) / T;
  const int64_t blocks = p.ends ? tp * row_tiles(p.nq, T, p.experts) : p.direct + (tp * tq - p.direct) * p.splits;
  // (a launch has fewer than 2^32 threads; outputs that need more pass any memory)
  const int threads = 256 * p.groups;
  if (blocks > 0xffffffffll / threads || tp * tq < p.direct) return hipErrorInvalidValue;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks), dim3(threads), 0, s, p);
    return hipGetLastError();
  };
  if (p.ends) {
    if (p.groups != 1) return hipErrorInvalidValue;
    if (T == 128) return go(forward_kernel<KIND, true, 128, 1, 4>);
    if constexpr (KIND == FWD)
      if (T == 256) return go(forward_kernel<KIND, true, 256, 1, 4>);
    return hipErrorInvalidValue;
  }
  hipError_t e = hipErrorInvalidValue;
  if (T == 128 && p.groups == 1) e = go(forward_kernel<KIND, false, 128, 1, 4>);
  else if (T == 128 && p.groups == 2) e = go(forward_kernel<KIND, false, 128, 2, 4>);
  else if (T == 64 && p.groups == 4) e = go(forward_kernel<KIND, false, 64, 4, 4>);
  else if (T == 256 && p.groups == 1) {
    if constexpr (KIND == FWD) e = go(forward_kernel<KIND, false, 256, 1, 4>);
  }
  return e == hipSuccess ? launch_sums(p, s) : e;
}

}  // namespace

hipError_t launch_forward(const MmParams& p, Kind kind, hipStream_t s) {
  return kind == FWD ? go_forward<FWD>(p, s) : kind == FWD32 ? go_forward<FWD32>(p, s) : hipErrorInvalidValue;
}

hipError_t launch_few(const MmParams& p, int rows, hipStream_t s) {
  const int64_t n = (p.np + 15) / 16;
  const int64_t y = p.ends ? row_tiles(p.nq, rows, p.experts) : (p.nq + rows - 1) / rows;
  if (y > 65535 || n * y > 0xffffffffll / 512) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)n, (uint32_t)y);
  auto go = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), 0, s, p);
    return hipGetLastError();
  };
  if (rows == 16) return p.ends ? go(few_kernel<true, 1, 8>, 8) : go(few_kernel<false, 1, 8>, 8);
  if (rows == 32 && !p.ends) return go(few_kernel<false, 2, 8>, 8);
  return hipErrorInvalidValue;
}

}  // namespace f8
}  // namespace muon
