// What the products of the 8-bit floating-point layer share: the 8-bit values'
// way to bf16, the place of an expert's rows, and a tile's way to memory.
#pragma once

#include <type_traits>

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

// Direct loads into LDS go through a buffer descriptor: 32-bit places from a base
// that the whole workgroup shares, zeros for a place past the end.  (Beside the
// global form the compiler can count neither the loads of registers nor the reads
// of LDS, and waits for all that are out: with the waits of the kernel's own the same, the
// weight gradient of 8192 x 3584 x 3584 took 195 us instead of 187.)
typedef __amdgpu_buffer_rsrc_t Rsrc;
constexpr uint32_t kPast = 0xfffffff0u;
__device__ __forceinline__ Rsrc rsrc(const char* base) {
  // (word 3: 32-bit elements)
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)kPast, 4 << 15);
}
__device__ __forceinline__ void dma16(Rsrc r, char* to, uint32_t at, uint32_t step) {
  // (an LDS address that the compiler cannot follow: it otherwise puts a wait for
  // every earlier load before a read of the LDS object; the waits are the
  // kernels' own)
  uint32_t lds = (uint32_t)(uintptr_t)(lds_ptr_t*)to;
  asm("" : "+s"(lds));
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t*)(uintptr_t)lds, 16, (int)at, (int)step, 0, 0);
}

// Four e4m3 values times a scale, as bf16, two per instruction: exact under scales
// from 2^-124 to 2^119; else rounded (nearest even) to bf16's subnormals, multiples
// of 2^-133, or infinite.  (A scale's sign and fraction are not looked at: 0 bits
// of exponent are 2^-127.)
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

// What a stage of a sum asks for ahead: whole stages; any, those past the end as
// zeros; or, near the end, none.  Each is code of its own: a branch among the
// MFMAs would make the compiler gather them behind it.
enum Mode { WHOLE, CUT, DRAIN };
template <Mode M> struct In { static constexpr Mode mode = M; };

// What a kernel writes to (put4, put8).
struct Out {
  void* out;
  int obf16, accumulate;
};

// Which tile a workgroup has: `split` of the `splits` ranges of its sum, and the
// rows that its part of the output has.
struct Place {
  int tile, split, splits, tp, tq, nq;
};

// A workgroup's tile and its part of the operands.
struct Work {
  const char *P, *Q;
  const uint8_t *scp, *scq;
  Out o;
  int kd;
  Place at;
};

// A tile's sums to memory, T columns and TQ rows (T of them, or the few that a
// row tile's end has).  Waves stand WP along P and NW / WP along Q; acc[i][j]
// covers FR columns and rows of the wave's part: quad g of it is columns FR i +
// qcol(g) .. +3 of row FR j + qrow.  G groups of NW waves have summed a share of
// K each; s_p and s_q hold RING bytes and nobody reads or writes them any more
// (a barrier stands ahead of the call).
template <int FR, int T, int TQ, int WP, int G, int NW, int RING, int FP, int FQ, typename Acc>
__device__ __forceinline__ void finish_tile(Acc (&acc)[FP][FQ], const MmParams& p, const Out& o, const Place& at,
                                            int group, int tid, char* s_p, char* s_q) {
  constexpr int QUADS = FR == 32 ? 4 : 1, WQ = NW / WP;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), q4 = lane >> 4;
  const int wp = wave / WQ, wq = wave % WQ;
  const int qrow = lane % FR;
  auto qcol = [&](int g) { return FR == 32 ? 8 * g + 4 * (lane >> 5) : 4 * q4; };
  const int colt = wp * (T / WP), rowt = wq * (TQ / WQ);
  const int col0 = at.tp * T + colt, row0 = at.tq * T + rowt;
  // A block's quads are finished by group b % G (b: the quad's number): j runs fastest.
  auto quad = [&](int i, int g, int j) __attribute__((always_inline)) {
    if constexpr (FR == 32) return f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    else return acc[i][j];
  };
  constexpr int NB = FP * QUADS * FQ;
  if constexpr (G > 1) {
    // The other groups leave a quad in LDS, lane by lane, and its own adds them
    // in their order.
    static_assert(NB % G == 0 && NB * (G - 1) * NW * 1024 <= RING, "the join fits the ring");
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

  float* const part = p.part + ((int64_t)(at.tile - p.direct) * at.splits + at.split) * (T * T);
  if constexpr (T > 64) {
    // A lane's four columns are 16 bytes of a row FR rows apart from its
    // neighbours'.  FR rows of SC columns of the wave's part at a time go
    // through LDS, 16-byte chunks swapped within a row by the row's number,
    // and leave as whole runs of 128 bytes or more.  One loop over them, not
    // unrolled but for its first lines.
    constexpr int PT = T / WP, SC = FR == 32 && PT > 64 ? 64 : PT, NH = PT / SC, CPR = SC / 4;
    static_assert(NW * FR * SC * 4 * G <= RING, "the staged rows fit a ring");
    static_assert(FQ % G == 0, "a row's quads are one group's");
    const bool wide = at.splits == 1 && p.obf16;
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
          if (at.splits > 1) {
            *(f32x4*)(part + (rowt + FR * jr + rr) * T + colt + c0) = v;
          } else if (r0 + rr < at.nq && n > 0) {
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
          if (r0 + rr < at.nq && n > 0) put8(o, (int64_t)(r0 + rr) * p.ldo + col0 + c0, n, e);
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  } else {
    static_assert(NB == G, "one quad per group");
    // quad `group`
    const int i = group / FQ / QUADS, g = group / FQ % QUADS, j = group % FQ;
    // (by selections of values: a choice of places would put the sums in memory)
    f32x4 a = quad(0, 0, 0);
#pragma unroll
    for (int b = 1; b < NB; ++b) {
      f32x4 v = quad(b / FQ / QUADS, b / FQ % QUADS, b % FQ);
      asm("" : "+v"(v));
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = b == group ? v[e] : a[e];
    }
    const int r = FR * j + qrow, c = FR * i + qcol(g), n = p.np - col0 - c;
    if (at.splits > 1) {
      *(f32x4*)(part + (rowt + r) * T + colt + c) = a;
    } else if (row0 + r < at.nq && n > 0) {
      const float e[4] = {a[0], a[1], a[2], a[3]};
      put4(o, (int64_t)(row0 + r) * p.ldo + col0 + c, n, e);
    }
  }
}

}  // namespace

}  // namespace f8
}  // namespace muon
