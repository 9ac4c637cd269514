// Gradient products of the 8-bit floating-point layer, dense or grouped by
// expert:
//   dX = dY w     P = w (rows n along K), Q = dY        (DX)
//   dW = dY^T x   P = x (rows t along K), Q = dY^T      (DW)
// as C[q][p] = sum_k P(p, k) Q(q, k) with p contiguous in C, on the bf16 MFMA
// with P on its A side, so each lane ends with four consecutive columns.
//
// P's e4m3 values are widened to bf16 with their scale on the way from memory
// through registers into LDS: exact (4 significant bits, powers of two) but at the
// ends of bf16's range, two values per instruction, once per workgroup.  Q comes by direct global->LDS
// loads.  Tiles, ring and schedule are those of the 8-bit integer layer's
// gradients (64 bytes of K per stage, four stages deep, one barrier per stage).
//
// K past the end is zero on both sides, so no value of a masked place (not even
// NaN) enters a sum; rows and columns past the end re-read the last valid ones
// and are not stored.
#include <algorithm>

#include "float8_tiles.hpp"

namespace muon {
namespace f8 {

namespace {

constexpr int D = 4;  // stages of a ring

// P of the gradients: e4m3 rows along K, 16 columns (8 of 64-wide tiles) per
// lane and chunk, widened with their scale on the way through registers into
// LDS.  SQUARE: a scale per 128 rows (weights), else per row.  A chunk lies
// within 128 columns, and within the readable part of its row.
template <bool SQUARE, int T, int NT>
struct WideOperand {
  static constexpr int CH = T == 64 ? 8 : 16;
  static constexpr int CPR = T / CH;
  static_assert(KROWS * CPR == NT, "a chunk per lane: two loads that no compiler joins");
  static constexpr int PIECES = CH / 4;
  static constexpr int LOADS = 2;  // of a stage: values and scale
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
  // If not WHOLE, some of the stage's rows may lie past the end, where the last
  // one is read.
  template <Mode M>
  __device__ __forceinline__ void load(Regs& r, int ks) const {
    int k = ks * KROWS + row;
    if (M != WHOLE) k = min(k, kd - 1);
    __builtin_memcpy(&r.v, src + (int64_t)k * ld, CH);
    r.scale = scale[(int64_t)(SQUARE ? k / kBlock : k) * lds];
  }
  // Piece q of a stage's way into LDS.
  template <Mode M>
  __device__ __forceinline__ void store(const Regs& r, Wide& w, char* lds_at, int stage, int ks, int q) const {
    const bool past = M != WHOLE && ks * KROWS + row >= kd;
    uint32_t b = past ? 0u : r.v[q];
    // (opaque: the bytes are taken apart here, not at the load, which would be waited for there)
    asm("" : "+v"(b));
    // (a scale of NaN past the end would make NaN of the zeros)
    const uint2 d = widen4(b, scale_of(past ? 127u : r.scale));
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

// Q of the gradients, T rows (columns, if K-major) by direct loads into LDS, laid
// out as DmaOperand does.  A row distance is at most 2^24 bytes.
template <bool KM, int T, int NW>
struct BufferOperand {
  static constexpr int NDMA = T * KB / 1024 / NW;  // 1-KB instructions per wave and stage
  const char* base;    // the tile's first row (column)
  uint32_t off[NDMA];  // the lane's place in a stage,
  int k[NDMA];         // and its row (byte) of K there
  int64_t step;        // bytes from stage to stage
  int kend;

  __device__ __forceinline__ void init(const char* b, int64_t ld, int row0, int count, int kd, int tid) {
    const int wave = tid >> 6, lane = tid & 63;
    step = KM ? KROWS * ld : (int64_t)KB;
    kend = KM ? kd : kd * 2;
    base = KM ? b : b + row0 * ld;
#pragma unroll
    for (int i = 0; i < NDMA; ++i) {
      if constexpr (KM) {
        constexpr int RB = T * 2, RPI = 1024 / RB, CH = RB / 16;
        k[i] = (wave * NDMA + i) * RPI + lane / CH;
        const int ch = (lane % CH) ^ swz_k<T>(k[i]);
        // (whole chunks, in the padded row)
        off[i] = (uint32_t)k[i] * (uint32_t)ld + (uint32_t)min(row0 + ch * 8, (count - 1) & ~7) * 2;
      } else {
        const int r = (wave * NDMA + i) * 16 + (lane >> 2);
        k[i] = ((lane & 3) ^ swz_c(r)) * 16;
        off[i] = (uint32_t)min(r, count - 1 - row0) * (uint32_t)ld + (uint32_t)k[i];
      }
    }
  }
  // Instruction i of stage ks; if not WHOLE, what lies past K's end is zeros.
  template <Mode M>
  __device__ __forceinline__ void load(int i, char* stage, int ks, int wave) const {
    uint32_t at = off[i];
    if (M != WHOLE) at = ks * (KM ? KROWS : KB) + k[i] < kend ? at : kPast;
    dma16(rsrc(base + ks * step), stage + (wave * NDMA + i) * 1024, at, 0);
  }
};

// One tile (or a contraction range of one) of T columns and TQ rows.
template <int KIND, int T, int TQ, int G, int NW>
__device__ __forceinline__ void mm_tile(const MmParams& p, const Work& w, char* s_p, char* s_q) {
  constexpr bool QKM = KIND == DW;
  constexpr int WP = TQ < T ? 4 : 2, WQ = NW / WP;    // waves along P and Q
  constexpr int FP = T / WP / 16, FQ = TQ / WQ / 16;  // 16 x 16 blocks per wave
  constexpr int H = FP / 2;                           // block rows per half stage
  typedef BufferOperand<QKM, TQ, NW> DmaQ;
  typedef WideOperand<KIND == DX, T, 64 * NW> RegP;
  constexpr int DPS = DmaQ::NDMA;                     // a stage's instructions,
  constexpr int DB = DPS / 2, DA = DPS - DB;          // in two halves
  constexpr int PIECES = RegP::PIECES;
  constexpr int OPB = T * KB;                         // room of one operand's stage in LDS
  constexpr int RS = 2;                               // register sets in flight

  const int tid = threadIdx.x % (64 * NW), lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = G > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / (64 * NW)) : 0;
  const int ring = group * D * OPB;                   // the group's rings
  auto at = [&](int st) { return (st & (D - 1)) * OPB; };  // a stage in them
  const int wp = wave / WQ, wq = wave % WQ;
  const int q4 = lane >> 4, c16 = lane & 15;
  const int kd = w.kd, nq = w.at.nq, tp = w.at.tp, tq = w.at.tq, split = w.at.split, splits = w.at.splits;

  const int full = kd / KROWS;
  const int nk = (kd + KROWS - 1) / KROWS;
  int k0 = 0, k1 = nk;
  if (splits > 1) {
    k0 = (int)((int64_t)nk * split / splits);
    k1 = (int)((int64_t)nk * (split + 1) / splits);
  }
  // stages per group, and this group's (the last ones may have fewer)
  const int most = (k1 - k0 + G - 1) / G;
  const int steps = G > 1 ? max(0, min(most, k1 - k0 - group * most)) : k1 - k0;
  k0 += group * most;
  f32x4 acc[FP][FQ];
#pragma unroll
  for (int i = 0; i < FP; ++i)
#pragma unroll
    for (int j = 0; j < FQ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  if (steps > 0) {  // (an empty sum reads nothing)
    DmaQ dq;
    RegP gp;
    gp.init(w.P, p.ldp, w.scp, p.ldsp, tp * T, p.np, kd, tid);
    dq.init(w.Q, p.ldq, tq * T, nq, kd, tid);
    auto dma = [&](auto in, int q, int st) __attribute__((always_inline)) {  // instruction q of stage k0 + st
      dq.template load<decltype(in)::mode>(q, s_q + ring + at(st), k0 + st, wave);
    };
    typename RegP::Regs rp[RS];
    typename RegP::Wide wide;
    auto put = [&](auto in, typename RegP::Regs& r, int st, int q) __attribute__((always_inline)) {
      gp.template store<decltype(in)::mode>(r, wide, s_p, ring + at(st), k0 + st, q);
    };
    Reader<true, T> fp;
    Reader<QKM, TQ> fq;
    fp.init(ring, wp * (T / WP), q4, c16);
    fq.init(ring, wq * (TQ / WQ), q4, c16);
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
          if (st < D - 1 || q < DA) dma(In<CUT>(), q, st);
      }
    // stages 0 .. RS + 1 in flight together; everything has landed before
    // the loop, so that the waits inside it only count the loop's own loads
    typename RegP::Regs rp0[2];
#pragma unroll
    for (int st = 0; st < 2; ++st) gp.template load<CUT>(rp0[st], k0 + st);
#pragma unroll
    for (int st = 0; st < RS; ++st) gp.template load<CUT>(rp[st], k0 + 2 + st);
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int q = 0; q < PIECES; ++q) put(In<CUT>(), rp0[st], st, q);
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
    barrier();
#pragma unroll
    for (int f = 0; f < H; ++f) fa[f] = fp.get(s_p, at(0), f);
#pragma unroll
    for (int f = 0; f < FQ; ++f) fb0[f] = fq.get(s_q, at(0), f);

    // A step, kt counting from k0, set = kt % RS.
    // (A wave in its MFMAs goes ahead of one that waits or loads: 128-wide tiles,
    // 2048 x 4096 x 4096, 69.3 -> 66.5 us; 256-wide, 4096 x 18944 x 3584, 441 -> 435.)
    auto step = [&](auto in, int kt, int set, u32x4* fb, u32x4* fbn) __attribute__((always_inline)) {
      constexpr Mode M = decltype(in)::mode;
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j = 0; j < FQ; ++j) mfma(fa[0], fb[j], acc[0][j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = H; f < FP; ++f) fa[f] = fp.get(s_p, at(kt), f);
      __builtin_amdgcn_sched_barrier(0);
      constexpr int N1 = (H - 1) * FQ, G1 = DB > 0 && N1 > DB ? N1 / (DB + (DB == 0)) : 1;
#pragma unroll
      for (int n = 0; n < N1; ++n) {
        mfma(fa[1 + n / FQ], fb[n % FQ], acc[1 + n / FQ][n % FQ]);
        if (M != DRAIN && DB > 0 && n % G1 == G1 - 1 && n / G1 < DB) {
          dma(in, DA + n / G1, kt + D - 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if constexpr (N1 == 0 && M != DRAIN) {
#pragma unroll
        for (int q = 0; q < DB; ++q) dma(in, DA + q, kt + D - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      // This wave's DMAs of stage kt + 1 have landed ((D - 2) DPS later ones
      // may fly, and the register loads of two steps), its LDS writes of stage
      // kt + 1 and its reads of stage kt are done.
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_s_waitcnt(wait_imm(M == DRAIN ? 0 : (D - 2) * DPS + 2 * RegP::LOADS, 0));
      barrier();
#pragma unroll
      for (int f = 0; f < H; ++f) fa[f] = fp.get(s_p, at(kt + 1), f);
#pragma unroll
      for (int f = 0; f < FQ; ++f) fbn[f] = fq.get(s_q, at(kt + 1), f);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      constexpr int N2 = H * FQ, G2 = N2 / DA;
      // pieces after each MFMA (several, where there are few MFMAs)
      constexpr int GP = N2 > PIECES ? N2 / (PIECES + 1) : 1, PB = (PIECES + N2 - 1) / N2;
#pragma unroll
      for (int n = 0; n < N2; ++n) {
        mfma(fa[H + n / FQ], fb[n % FQ], acc[H + n / FQ][n % FQ]);
        if (M != DRAIN && n % G2 == G2 - 1 && n / G2 < DA) dma(in, n / G2, kt + D);
        if (n % GP == GP - 1) {
#pragma unroll
          for (int q = 0; q < PB; ++q)
            if (n / GP * PB + q < PIECES) put(in, rp[set], kt + 2, n / GP * PB + q);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      if constexpr (M != DRAIN) gp.template load<M>(rp[set], k0 + kt + 2 + RS);
      __builtin_amdgcn_sched_barrier(0);
    };
    // Two steps per trip: the Q fragments and the register sets alternate
    // without copies.  (The last step that has a stage to ask for is steps - D:
    // the second half of its DMAs.)
    static_assert(RS + 2 <= D, "a register load reaches no further than a DMA");
    int kt = 0;
    auto trip = [&](auto in) __attribute__((always_inline)) {
      step(in, kt, 0, fb0, fb1);
      step(in, kt + 1, 1, fb1, fb0);
      kt += 2;
    };
    const int whole = min(steps, full - k0) - D;
    while (kt + 1 < whole) trip(In<WHOLE>());
    while (kt <= steps - D) trip(In<CUT>());
    while (kt + 1 < steps) trip(In<DRAIN>());
    if (kt < steps) step(In<DRAIN>(), kt, 0, fb0, fb1);
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));  // no load may land after the workgroup's LDS is given back
  }

  if constexpr (G > 1) {
    // a group's barriers: one ahead of the loop and one per step
    if (most > 0) {
      for (int i = steps > 0 ? steps : -1; i < most; ++i) barrier();
    }
  }
  barrier();  // no wave reads the rings any more
  finish_tile<16, T, TQ, WP, G, NW, G * D * OPB>(acc, p, w.o, w.at, group, tid, s_p, s_q);
}

// A workgroup per tile.  An expert's last row tile of at most 128 rows is computed
// as one of 128: the input gradient of 61 experts of 128 rows, 1408 x 2048, 87 ->
// 60 us.
//
// A 256-wide stage takes 0.79 us, of which its MFMAs are 0.43 at 2.4 GHz and the
// reads and writes of LDS as much: 8192 x 3584 x 3584 (weight gradient) 188 us,
// matrix cores 60 % busy on the 196 units that have a tile; 4096 x 18944 x 3584
// (input gradient) 440, 65 % on 224 units.
template <int KIND, bool GROUPED, int T, int G, int NW>
__global__ void __launch_bounds__(64 * NW * G, T == 128 && G == 1 ? 2 : 1) mm_kernel(const MmParams p) {
  // (two objects: the compiler then knows that a write to one is no write to
  // the other)
  __shared__ __attribute__((aligned(1024))) char s_p[G * D * T * KB];
  __shared__ __attribute__((aligned(1024))) char s_q[G * D * T * KB];

  // This workgroup's tile, and its part of the operands.
  const char *P = p.P, *Q = p.Q;
  const uint8_t* scp = p.sp;
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

  const Work w = {P, Q, scp, nullptr, o, kd, {tile, split, splits, tp, tq, nq}};
  if constexpr (GROUPED && T == 256)
    if (nq - tq * T <= T / 2) return mm_tile<KIND, T, T / 2, G, NW>(p, w, s_p, s_q);
  mm_tile<KIND, T, T, G, NW>(p, w, s_p, s_q);
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

template <int KIND>
hipError_t go_grads(const MmParams& p, hipStream_t s) {
  const int T = p.tile;
  const int64_t tp = (p.np + T - 1) / T, tq = (p.nq + T - 1) / T;
  int64_t blocks;
  if (!p.ends) blocks = p.direct + (tp * tq - p.direct) * p.splits;
  else if (KIND == DW) blocks = tp * tq * p.experts;
  else blocks = tp * row_tiles(p.nq, T, p.experts);
  // (a launch has fewer than 2^32 threads; outputs that need more pass any memory)
  const int threads = 64 * (T == 256 ? 8 : 4) * p.groups;
  if (blocks > 0xffffffffll / threads || tp * tq < p.direct) return hipErrorInvalidValue;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks), dim3(threads), 0, s, p);
    return hipGetLastError();
  };
  if (p.ends) {
    if (p.groups != 1) return hipErrorInvalidValue;
    if (T == 256) return go(mm_kernel<KIND, true, 256, 1, 8>);
    if (T == 128) return go(mm_kernel<KIND, true, 128, 1, 4>);
    return hipErrorInvalidValue;
  }
  hipError_t e = hipErrorInvalidValue;
  if (T == 256 && p.groups == 1) e = go(mm_kernel<KIND, false, 256, 1, 8>);
  else if (T == 128 && p.groups == 1) e = go(mm_kernel<KIND, false, 128, 1, 4>);
  else if (T == 128 && p.groups == 2) e = go(mm_kernel<KIND, false, 128, 2, 4>);
  else if (T == 64 && p.groups == 4) e = go(mm_kernel<KIND, false, 64, 4, 4>);
  return e == hipSuccess ? launch_sums(p, s) : e;
}

}  // namespace

hipError_t launch_grads(const MmParams& p, Kind kind, hipStream_t s) {
  return kind == DX ? go_grads<DX>(p, s) : kind == DW ? go_grads<DW>(p, s) : hipErrorInvalidValue;
}

hipError_t launch_sums(const MmParams& p, hipStream_t s) {
  const int T = p.tile;
  const int64_t rest = (int64_t)((p.np + T - 1) / T) * ((p.nq + T - 1) / T) - p.direct;
  if (p.ends || rest == 0 || p.splits == 1) return hipSuccess;
  const dim3 sums((uint32_t)(T * T / 1024), (uint32_t)rest);
  if (T == 256) hipLaunchKernelGGL(mm_sum_kernel<256>, sums, dim3(256), 0, s, p);
  else if (T == 128) hipLaunchKernelGGL(mm_sum_kernel<128>, sums, dim3(256), 0, s, p);
  else hipLaunchKernelGGL(mm_sum_kernel<64>, sums, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace f8
}  // namespace muon
