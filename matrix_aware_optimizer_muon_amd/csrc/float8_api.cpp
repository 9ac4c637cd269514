// C ABI of the 8-bit floating-point layer (include/muon_float8.h): validation,
// the choice of kernel, tile and split, and the launch sequence.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <iterator>

#include "float8.h"
#include "linear8.h"
#include "muon_float8.h"

using namespace muon::f8;

namespace {

constexpr int64_t kMaxDim = 1ll << 24;

bool known(muon_dtype t) { return t == MUON_F32 || t == MUON_BF16; }
int64_t size_of(muon_dtype t) { return t == MUON_BF16 ? 2 : 4; }
bool aligned(const void* p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t blocks_of(int64_t v) { return (v + kBlock - 1) / kBlock; }
muon_status hip(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }

// A matrix argument: present, aligned to its elements, rows that do not
// overlap.
bool matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t size) {
  return p && aligned(p, size) && (rows <= 1 || ld >= cols);
}
// Distances that no memory holds, whose products would pass 64 bits.
constexpr int64_t kFar = 1ll << 36;
bool far(int64_t ld, int64_t rows) { return rows > 1 && (ld > kFar || ld < -kFar); }
// 8-bit rows: each starts at a multiple of 16 bytes.  (Kernels add up a tile's
// row distances, and in the forward product K, in 32 bits: kMaxLd, bytes.  dy's
// that lie further apart are laid out again.)
constexpr int64_t kMaxLd = 1ll << 23, kMaxGap = 1ll << 24;
bool matrix8(const void* p, int64_t ld, int64_t rows, int64_t cols) {
  return p && aligned(p, 16) && (rows <= 1 || (ld >= cols && ld % 16 == 0));
}

// How a product runs.  few: rows of the few rows' kernel, or 0.
struct Choice {
  Kind kind = FWD;
  int few = 0;
  bool pack = false;          // a laid out again
  int64_t lda = 0, bytes = 0; // bytes of a's row as the kernel reads it; of the workspace
  int64_t at_part = 0;
  int tile = 128, groups = 1, splits = 1, direct = 0;
  int np = 0, nq = 0, kd = 0;
};

// Measured times of a tile, us: per stage of its sum (128 bytes of K forward, 32
// rows or columns of the gradients), and what is ahead of and behind it, for
// workgroups that run at once: a tile of 256 or a 128-wide one of two wave groups
// per compute unit, two 128-wide ones of one group, one 64-wide of four.
struct Cost {
  double stage, ends;
};
struct Costs {
  Cost t256, t128, t128g2, t64g4;
};
const Costs kCosts[] = {
    {{1.39, 10.8}, {0.91, 6.0}, {1.01, 4.9}, {1.05, 4.1}},  // FWD
    {{0.0, 0.0}, {1.57, 7.2}, {1.63, 6.3}, {1.38, 4.4}},    // FWD32 (no 256-wide tile)
    {{0.79, 8.1}, {0.52, 6.0}, {0.54, 5.6}, {0.53, 3.5}},   // DX
    {{0.80, 7.8}, {0.54, 5.8}, {0.54, 5.8}, {0.45, 4.3}},   // DW
};

// The few rows' kernel, us: the read of w and, growing with the rows, of x; a
// wave's chain of loads where there are few workgroups.
double few_us(double matrices, double rows, int few, int64_t n, int64_t k) {
  const double read = matrices * (double)n * (double)k * (few == 16 ? 1.0 : 1.2) / 6.2e6;
  const double chain = (double)((k + 1023) / 1024) * 0.53;
  return 2.8 + std::max(read, chain) * (1.0 + 0.033 * (rows - 1.0));
}

// The cheapest way for one matrix: workgroups take a tile each in whole rounds;
// the tiles left over may be split along K over one more round, for a second
// launch (4 us) and their partial sums' way to memory and back (at 4 TB/s).
void choose_dense(Choice& c) {
  const Costs& costs = kCosts[c.kind];
  const bool fwd = c.kind == FWD || c.kind == FWD32;
  const int64_t stages = fwd ? blocks_of(c.kd) : (c.kd + 31) / 32;
  auto tiles = [&](int64_t T) { return (int64_t)((c.np + T - 1) / T) * ((c.nq + T - 1) / T); };
  double best = 0.0;
  auto way = [&](int tile, int groups, const Cost& cost) {
    const int64_t all = tiles(tile), slots = tile == 128 && groups == 1 ? 512 : 256, rest = all % slots;
    const int64_t each = (stages + groups - 1) / groups;  // a group's stages
    const double whole = (double)(all / slots) * (cost.stage * (double)each + cost.ends);
    double us = whole + (rest > 0 ? cost.stage * (double)each + cost.ends : 0.0);
    int splits = 1;
    const int64_t most = rest > 0 ? std::min<int64_t>({slots / rest, each / (fwd ? 2 : 4), 32}) : 1;
    for (int64_t n = 2; n <= most; ++n) {
      const double with = whole + cost.stage * (double)((each + n - 1) / n) + cost.ends + 4.0 +
                          (double)tile * tile * 8 / 4e6 * (double)(rest * n);
      if (with < us) {
        us = with;
        splits = (int)n;
      }
    }
    if (best == 0.0 || us < best) {
      best = us;
      c.tile = tile;
      c.groups = groups;
      c.splits = splits;
      c.direct = (int)(splits > 1 ? all - rest : all);
    }
  };
  // (wave groups that share K need a compute unit of their own)
  if (tiles(128) <= 256) way(128, 2, costs.t128g2);
  else way(128, 1, costs.t128);
  if (costs.t256.stage > 0) way(256, 1, costs.t256);
  if (tiles(64) <= 256) way(64, 4, costs.t64g4);
  if (fwd)
    for (const int few : {16, 32})
      if (c.nq <= few && few_us(1.0, (double)c.nq, few, c.np, c.kd) < best) {
        c.few = few;
        c.splits = 1;
        break;
      }
}

// The same for experts, whose rows only the device knows: their number of tiles
// is taken as if they shared the rows evenly, with half a tile more each, and at
// least one (0.45 and 0.75 of 256 rows, of which up to 128 take less time), and
// no whole rounds: 0.4 of one more than their share.  256-wide ones have to win by
// 4 %, since fewer tiles spread worse: over 105 sizes, 4 to 4000 rows per expert of
// uneven numbers, the choice is 1 % off the better one in the mean.  No splits and no
// wave groups, so the tiles have to fill the card by their number: those of few
// experts with small matrices and many rows do not (the weight gradients of 2 experts of
// 16384 rows, 256 x 256, are 8 workgroups and take 285 us; one dense call for
// each, 15).
void choose_experts(Choice& c, int64_t experts, int64_t t) {
  const Costs& costs = kCosts[c.kind];
  const bool fwd = c.kind == FWD || c.kind == FWD32;
  const double busy = (double)std::min(experts, t), rows = (double)t / std::max(busy, 1.0);
  auto rounds = [](double tiles, double slots) { return std::max(1.0, tiles / slots); };
  auto columns = [&](int64_t T, int64_t n) { return (double)((n + T - 1) / T); };
  auto way = [&](int64_t T, const Cost& cost, double slots) {
    if (c.kind == DW) {
      // the tiles' number is known, their sums are not: with less than two rounds
      // the longest expert's counts (taken as twice the mean)
      const double tiles = (double)experts * columns(T, c.np) * columns(T, c.nq);
      return rounds(tiles, slots) * (cost.stage * rows / 32.0 + cost.ends) + (tiles < 2 * slots ? cost.stage * rows / 32.0 : 0.0);
    }
    const double stages = fwd ? (double)blocks_of(c.kd) : (double)((c.kd + 31) / 32);
    const double each = T == 256 ? std::max(0.75, rows / 256.0 + 0.45) : std::max(1.0, rows / (double)T + 0.5);
    const double tiles = busy * each * columns(T, c.np);
    // (alone on its compute unit a 128-wide tile has a stage in two thirds of the time)
    const double stage = T == 128 && tiles <= 256 ? cost.stage * 0.67 : cost.stage;
    return (tiles > 0.8 * slots ? rounds(tiles + 0.4 * slots, slots) : 1.0) * (stage * stages + cost.ends);
  };
  double best = way(128, costs.t128, 512);
  c.tile = 128;
  if (costs.t256.stage > 0) {
    const double us = way(256, costs.t256, 256) * (c.kind == DW ? 1.0 : 1.04);
    if (us < best) {
      best = us;
      c.tile = 256;
    }
  }
  // (an expert's rows vary: up to a mean of half the kernel's)
  if (fwd && rows <= 8.0 && few_us(busy, 4.0 * rows - 3.0, 16, c.np, c.kd) < best) c.few = 16;
}

Choice choose(muon_f8_product product, const void* a, int64_t lda, bool grouped, int64_t experts, int64_t t, int64_t n,
              int64_t k, bool bf16) {
  Choice c;
  const bool fwd = product == MUON_F8_MATMUL, dw = product == MUON_F8_GRAD_WEIGHT;
  c.kind = fwd ? (bf16 ? FWD : FWD32) : dw ? DW : DX;
  c.np = (int)(fwd ? n : k);
  c.nq = (int)(dw ? n : t);
  c.kd = (int)(fwd ? k : dw ? t : n);
  const int64_t a_cols = fwd ? k : n, size = fwd ? 1 : 2;
  c.lda = t <= 1 ? up(a_cols * size, 16) : lda * size;
  if (!fwd && t * n > 0) {
    // bf16 rows that the DMA cannot read: not at 16 bytes, with a last chunk that
    // would leave the matrix, or too far apart
    c.pack = !aligned(a, 16) || c.lda % 16 || a_cols % 8 || c.lda > kMaxGap;
    if (c.pack) {
      c.lda = up(a_cols * 2, 16);
      c.bytes = up(t * c.lda, 256);
    }
  }
  if (grouped) choose_experts(c, experts, t);
  else choose_dense(c);
  // (a launch has fewer than 2^32 threads)
  if (c.few && up(n, 16) / 16 * (grouped ? row_tiles(t, c.few, experts) : 1) > (1ll << 32) / 512 - 1) c.few = 0;
  if (c.splits > 1) {
    c.at_part = c.bytes;
    const int64_t T = c.tile;
    c.bytes += ((c.np + T - 1) / T * ((c.nq + T - 1) / T) - c.direct) * c.splits * T * T * 4;
  }
  return c;
}

muon_status product_sizes(muon_f8_product product, bool grouped, int64_t experts, int64_t t, int64_t n, int64_t k) {
  if (product < MUON_F8_MATMUL || product > MUON_F8_GRAD_WEIGHT) return MUON_ERR_INVALID_ARGUMENT;
  if (t < 0 || n < 0 || k < 0 || experts < 1 || (!grouped && experts != 1)) return MUON_ERR_INVALID_ARGUMENT;
  if (t > kMaxDim || n > kMaxDim || k > kMaxDim || experts > kMaxExperts) return MUON_ERR_UNSUPPORTED;
  if (product != MUON_F8_MATMUL && t > 1 && n * 2 > kMaxGap) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

// a: xq or dy; b: the weights, or the rows of the weight gradient.
struct Call {
  muon_f8_product product;
  const void* a;
  int64_t lda;
  const uint8_t* a_scale;
  const uint8_t* b;
  int64_t ldb, b_stride;
  const uint8_t* b_scale;
  const int32_t* ends;
  int64_t experts, t, n, k;
  void* out;
  int64_t ldo, o_stride;
  muon_dtype dtype;
  bool accumulate;
  void* workspace;
  size_t workspace_bytes;
};

muon_status run(const Call& v, hipStream_t s) {
  const bool fwd = v.product == MUON_F8_MATMUL, dw = v.product == MUON_F8_GRAD_WEIGHT, grouped = v.ends != nullptr;
  const muon_status bad = product_sizes(v.product, grouped, v.experts, v.t, v.n, v.k);
  if (bad != MUON_OK) return bad;
  if (!known(v.dtype) || !aligned(v.ends, 4)) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t t = v.t, n = v.n, k = v.k;
  const int64_t a_cols = fwd ? k : n, b_rows = dw ? t : n;
  const int64_t o_rows = dw ? n : t, o_cols = fwd ? n : k;
  if (o_rows == 0 || o_cols == 0) return MUON_OK;
  if (!matrix(v.out, v.ldo, o_rows, o_cols, size_of(v.dtype))) return MUON_ERR_INVALID_ARGUMENT;
  if ((fwd && t > 1 && v.lda > kMaxLd) || (b_rows > 1 && v.ldb > kMaxLd) || far(v.lda, t) || far(v.ldo, o_rows) ||
      (dw ? far(v.o_stride, v.experts) : far(v.b_stride, v.experts)))
    return MUON_ERR_UNSUPPORTED;
  if (t * a_cols > 0 && !(fwd ? matrix8(v.a, v.lda, t, a_cols) : matrix(v.a, v.lda, t, a_cols, 2)))
    return MUON_ERR_INVALID_ARGUMENT;
  if (b_rows * k > 0 && !matrix8(v.b, v.ldb, b_rows, k)) return MUON_ERR_INVALID_ARGUMENT;
  if ((fwd && t * k > 0 && !v.a_scale) || (b_rows * k > 0 && !v.b_scale)) return MUON_ERR_INVALID_ARGUMENT;
  if (v.experts > 1) {
    // one expert's matrix behind the other's
    if (dw && v.o_stride < (o_rows > 1 ? (o_rows - 1) * v.ldo : 0) + o_cols) return MUON_ERR_INVALID_ARGUMENT;
    if (!dw && n * k > 0 && (v.b_stride % 16 || v.b_stride < (n > 1 ? (n - 1) * v.ldb : 0) + k))
      return MUON_ERR_INVALID_ARGUMENT;
  }
  const Choice c = choose(v.product, v.a, v.lda, grouped, v.experts, t, n, k, v.dtype == MUON_BF16);
  if (c.bytes > 0) {
    if (v.workspace_bytes < (size_t)c.bytes) return MUON_ERR_WORKSPACE_TOO_SMALL;
    if (!v.workspace || !aligned(v.workspace, 256)) return MUON_ERR_INVALID_ARGUMENT;
  }
  char* const w = (char*)v.workspace;
  MmParams p = {};
  p.Q = c.pack ? w : (const char*)v.a;
  p.P = (const char*)v.b;
  p.sp = v.b_scale;
  p.sq = v.a_scale;
  p.ends = v.ends;
  p.ldp = b_rows <= 1 ? up(k, 16) : v.ldb;
  p.ldq = c.lda;
  p.ldsp = (int)blocks_of(k);
  p.ldsq = (int)blocks_of(a_cols);
  p.stride_p = v.b_stride;
  p.stride_sp = blocks_of(n) * blocks_of(k);
  p.stride_o = v.o_stride;
  p.experts = (int)v.experts;
  p.np = c.np;
  p.nq = c.nq;
  p.kd = c.kd;
  p.tile = c.tile;
  p.groups = c.groups;
  p.direct = c.direct;
  p.splits = c.splits;
  p.out = v.out;
  p.ldo = v.ldo;
  p.obf16 = v.dtype == MUON_BF16;
  p.accumulate = v.accumulate;
  p.part = c.splits > 1 ? (float*)(w + c.at_part) : nullptr;
  if (c.few) return hip(launch_few(p, c.few, s));
  hipError_t e = hipSuccess;
  if (c.pack) e = muon::l8::launch_pack(v.a, t > 1 ? v.lda * 2 : 0, a_cols * 2, w, c.lda, t, s);
  if (e == hipSuccess) e = fwd ? launch_forward(p, c.kind, s) : launch_grads(p, c.kind, s);
  return hip(e);
}

// Checks of a call that makes or reads the 8-bit form.
muon_status form_sizes(muon_dtype dtype, int64_t count, int64_t rows, int64_t cols, int block_rows) {
  if (!known(dtype) || count < 0 || rows < 0 || cols < 0 || (block_rows != 1 && block_rows != kBlock))
    return MUON_ERR_INVALID_ARGUMENT;
  if (rows > kMaxDim || cols > kMaxDim || count > kMaxDim) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

}  // namespace

extern "C" {

muon_status muon_f8_quantize(const void* x, int64_t ldx, int64_t x_stride, muon_dtype dtype, int64_t count,
                             int64_t rows, int64_t cols, int block_rows, uint8_t* q, int64_t ldq, int64_t q_stride,
                             uint8_t* scale, hipStream_t stream) {
  const muon_status bad = form_sizes(dtype, count, rows, cols, block_rows);
  if (bad != MUON_OK) return bad;
  if (count == 0 || rows == 0 || cols == 0) return MUON_OK;
  if (far(ldx, rows) || far(ldq, rows) || far(x_stride, count) || far(q_stride, count)) return MUON_ERR_UNSUPPORTED;
  if (!matrix(x, ldx, rows, cols, size_of(dtype)) || !matrix8(q, ldq, rows, cols) || !scale ||
      (count > 1 && (q_stride % 16 || q_stride < (rows > 1 ? (rows - 1) * ldq : 0) + cols)))
    return MUON_ERR_INVALID_ARGUMENT;
  const FormParams p = {(void*)x, q, scale, count, rows, cols, ldx, x_stride, ldq, q_stride, block_rows};
  return hip(launch_quantize(p, dtype == MUON_BF16, stream));
}

muon_status muon_f8_dequantize(const uint8_t* q, int64_t ldq, int64_t q_stride, const uint8_t* scale, int64_t count,
                               int64_t rows, int64_t cols, int block_rows, void* x, int64_t ldx, int64_t x_stride,
                               muon_dtype dtype, hipStream_t stream) {
  const muon_status bad = form_sizes(dtype, count, rows, cols, block_rows);
  if (bad != MUON_OK) return bad;
  if (count == 0 || rows == 0 || cols == 0) return MUON_OK;
  if (far(ldx, rows) || far(ldq, rows) || far(x_stride, count) || far(q_stride, count)) return MUON_ERR_UNSUPPORTED;
  if (!matrix(x, ldx, rows, cols, size_of(dtype)) || !matrix8(q, ldq, rows, cols) || !scale ||
      (count > 1 && (q_stride % 16 || x_stride < (rows > 1 ? (rows - 1) * ldx : 0) + cols)))
    return MUON_ERR_INVALID_ARGUMENT;
  const FormParams p = {x, (uint8_t*)q, (uint8_t*)scale, count, rows, cols, ldx, x_stride, ldq, q_stride, block_rows};
  return hip(launch_dequantize(p, dtype == MUON_BF16, stream));
}

muon_status muon_f8_workspace(muon_f8_product product, const void* a, int64_t lda, int grouped, int64_t experts,
                              int64_t t, int64_t n, int64_t k, muon_dtype dtype, size_t* workspace_bytes) {
  if (!workspace_bytes || !known(dtype)) return MUON_ERR_INVALID_ARGUMENT;
  const muon_status bad = product_sizes(product, grouped != 0, experts, t, n, k);
  if (bad != MUON_OK) return bad;
  if (far(lda, t)) return MUON_ERR_UNSUPPORTED;
  *workspace_bytes = (size_t)choose(product, a, lda, grouped != 0, experts, t, n, k, dtype == MUON_BF16).bytes;
  return MUON_OK;
}

// (float8.h)
void muon_f8_choice(int product, const void* a, int64_t lda, int grouped, int64_t experts, int64_t t, int64_t n,
                    int64_t k, int bf16, int64_t* out) {
  const Choice c = choose((muon_f8_product)product, a, lda, grouped != 0, experts, t, n, k, bf16 != 0);
  const int64_t T = c.tile, tiles = c.few ? 0 : (c.np + T - 1) / T * ((c.nq + T - 1) / T);
  const int64_t v[] = {c.kind, c.few, T, c.groups, c.pack, c.direct, tiles - c.direct, c.splits};
  std::copy(std::begin(v), std::end(v), out);
}

muon_status muon_f8_matmul(const uint8_t* xq, int64_t ldx, const uint8_t* x_scale, const uint8_t* wq, int64_t ldw,
                           int64_t w_stride, const uint8_t* w_scale, const int32_t* ends, int64_t experts, int64_t t,
                           int64_t n, int64_t k, void* y, int64_t ldy, muon_dtype dtype, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  return run({MUON_F8_MATMUL, xq, ldx, x_scale, wq, ldw, w_stride, w_scale, ends, experts, t, n, k, y, ldy, 0, dtype,
              false, workspace, workspace_bytes},
             stream);
}

muon_status muon_f8_grad_input(const void* dy, int64_t lddy, const uint8_t* wq, int64_t ldw, int64_t w_stride,
                               const uint8_t* w_scale, const int32_t* ends, int64_t experts, int64_t t, int64_t n,
                               int64_t k, void* dx, int64_t lddx, muon_dtype dtype, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
  return run({MUON_F8_GRAD_INPUT, dy, lddy, nullptr, wq, ldw, w_stride, w_scale, ends, experts, t, n, k, dx, lddx, 0,
              dtype, false, workspace, workspace_bytes},
             stream);
}

muon_status muon_f8_grad_weight(const void* dy, int64_t lddy, const uint8_t* xq, int64_t ldx, const uint8_t* x_scale,
                                const int32_t* ends, int64_t experts, int64_t t, int64_t n, int64_t k, void* dw,
                                int64_t lddw, int64_t dw_stride, muon_dtype dtype, int accumulate, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  return run({MUON_F8_GRAD_WEIGHT, dy, lddy, nullptr, xq, ldx, 0, x_scale, ends, experts, t, n, k, dw, lddw, dw_stride,
              dtype, accumulate != 0, workspace, workspace_bytes},
             stream);
}

}  // extern "C"
