// C ABI of the 8-bit linear layer (include/muon_linear8.h): validation, the
// choice of kernel, tile and split, and the launch sequence.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <iterator>

#include "linear8.h"
#include "muon_linear8.h"

using namespace muon::l8;

namespace {

constexpr int64_t kMaxDim = 1ll << 24;
constexpr int64_t kMaxK8 = 131071;  // 128 * 128 * k stays below 2^31

bool known(muon_dtype t) { return t == MUON_F32 || t == MUON_BF16; }
int64_t size_of(muon_dtype t) { return t == MUON_BF16 ? 2 : 4; }
bool aligned(const void* p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
muon_status hip(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }

// A matrix argument: present, aligned to its elements, rows that do not
// overlap.
bool matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t size) {
  return p && aligned(p, size) && (rows <= 1 || ld >= cols);
}

muon_status row_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 1) return MUON_ERR_INVALID_ARGUMENT;
  if (rows > 0x7fffffff || cols > kMaxCols) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

// How a product runs.  `few`: the kernel for few rows of x.
struct Choice {
  bool few = false;
  bool unaligned = false;          // read through registers (tiles 128 and 64)
  bool pack_q = false, pack_p = false;
  int64_t ldq = 0, ldp = 0;        // bytes, as the tile kernel reads them
  int padq = 0, padp = 0;          // readable after the last row
  int64_t at_q = 0, at_p = 0, at_part = 0;
  int tile = 128, groups = 1, splits = 1, direct = 0;
  int np = 0, nq = 0, kd = 0;
  int64_t bytes = 0;
};

Choice choose(muon_q8_product kind, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t t,
              int64_t n, int64_t k) {
  Choice c;
  const bool i8 = kind == MUON_Q8_MATMUL;
  if (i8 && few_rows(t, n, k)) {
    c.few = true;
    return c;
  }
  // a is Q, b is P; their stored shapes
  const int64_t sa = i8 ? 1 : 2;
  const int64_t a_rows = t, a_cols = i8 ? k : n;
  const int64_t b_rows = kind == MUON_Q8_GRAD_WEIGHT ? t : n, b_cols = k;
  c.np = (int)(i8 ? n : k);
  c.nq = (int)(kind == MUON_Q8_GRAD_WEIGHT ? n : t);
  c.kd = (int)(i8 ? k : kind == MUON_Q8_GRAD_INPUT ? n : t);
  c.ldq = a_rows <= 1 ? a_cols * sa : lda * sa;
  c.ldp = b_rows <= 1 ? b_cols : ldb;
  // what the DMA reads: Q, and P of the integer product
  const bool off_q = !aligned(a, 16) || c.ldq % 16 || a_cols * sa % 16;
  const bool off_p = i8 && (!aligned(b, 16) || c.ldp % 16 || b_cols % 16);
  auto tiles = [&](int64_t T) { return (int64_t)((c.np + T - 1) / T) * ((c.nq + T - 1) / T); };
  const int64_t stages = (c.kd + (i8 ? 63 : 31)) / (i8 ? 64 : 32);
  // A way to run it, and its time.  Workgroups that run at once (slots: one
  // per compute unit, two of 128-wide tiles with one group) take a tile each in
  // whole rounds; the tiles left over may be split along K over one more round.
  // Measured: a stage takes 0.3 us in 64-wide integer tiles (0.5 unaligned),
  // 0.55 in the gradients', 0.55 (0.8) and 0.6 in 128-wide ones, 0.75 and 0.85
  // in 256-wide ones; what is ahead of and behind a tile's sum 4, 5.3 (7.5) and
  // 10.5 us; a split costs a second launch (4 us) and its partial sums' way to
  // memory and back (at 4 TB/s), an operand that is packed first a launch behind
  // others (2.5 us) and as much.
  struct Way {
    int tile, groups, splits, direct;
    double us;
  };
  auto way = [&](int tile, int groups) {
    const int64_t all = tiles(tile), slots = tile == 128 && groups == 1 ? 512 : 256, rest = all % slots;
    const int64_t each = (stages + groups - 1) / groups;  // a group's stages
    const bool off = i8 && (off_q || off_p);
    const double stage_us = tile == 256   ? (i8 ? 0.75 : 0.85)
                            : tile == 128 ? (off ? 0.8 : i8 ? 0.55 : 0.6)
                                          : (off ? 0.5 : i8 ? 0.3 : 0.55);
    const double ends_us = tile == 256 ? 10.5 : tile == 128 ? (off ? 7.5 : 5.3) : 4.0;
    const double whole = (double)(all / slots) * (stage_us * (double)each + ends_us);
    Way w = {tile, groups, 1, (int)all, whole + (rest > 0 ? stage_us * (double)each + ends_us : 0.0)};
    const double tile_us = (double)tile * tile * 8 / 4e6;  // written and read
    const int64_t most = rest > 0 ? std::min<int64_t>({slots / rest, each / 4, 32}) : 1;
    for (int64_t n = 2; n <= most; ++n) {
      const double us = whole + stage_us * (double)((each + n - 1) / n) + ends_us + 4.0 + tile_us * (double)(rest * n);
      if (us < w.us) {
        w.us = us;
        w.splits = (int)n;
        w.direct = (int)(all - rest);
      }
    }
    if (tile == 256)
      w.us += (off_q ? 2.5 + (double)(a_rows * a_cols * sa) * 2 / 4e6 : 0.0) +
              (off_p ? 2.5 + (double)(b_rows * b_cols) * 2 / 4e6 : 0.0);
    return w;
  };
  // (wave groups that share K need a compute unit of their own: as many tiles
  // at most)
  Way w = way(128, tiles(128) <= 256 ? 2 : 1);
  const Way large = way(256, 1);
  if (large.us < w.us) w = large;
  if (tiles(64) <= 256) {
    const Way small = way(64, 4);
    if (small.us < w.us) w = small;
  }
  c.tile = w.tile;
  c.groups = w.groups;
  c.splits = w.splits;
  c.direct = w.direct;
  if (c.tile == 256) {
    c.pack_q = off_q;
    c.pack_p = off_p;
  } else {
    // through registers, from matrices of at least 16 bytes
    c.unaligned = off_q || off_p;
    c.pack_q = c.unaligned && (a_rows - 1) * c.ldq + a_cols * sa < 16;
    c.pack_p = (c.unaligned || !i8) && (b_rows - 1) * c.ldp + b_cols < 16;
  }
  if (c.kd == 0) c.pack_q = c.pack_p = false;
  if (c.pack_q) {
    c.ldq = up(a_cols * sa, 16);
    c.padq = (int)(c.ldq - a_cols * sa);
    c.at_q = c.bytes;
    c.bytes += up(a_rows * c.ldq, 256);
  }
  if (c.pack_p) {
    c.ldp = up(b_cols, 16);
    c.padp = (int)(c.ldp - b_cols);
    c.at_p = c.bytes;
    c.bytes += up(b_rows * c.ldp, 256);
  }
  if (c.splits > 1) {
    c.at_part = c.bytes;
    c.bytes += (tiles(c.tile) - c.direct) * c.splits * c.tile * c.tile * 4;
  }
  return c;
}

muon_status product_sizes(muon_q8_product kind, int64_t t, int64_t n, int64_t k) {
  if (t < 0 || n < 0 || k < 0) return MUON_ERR_INVALID_ARGUMENT;
  if (t > kMaxDim || n > kMaxDim || k > kMaxDim) return MUON_ERR_UNSUPPORTED;
  if (kind == MUON_Q8_MATMUL && k > kMaxK8) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

// Lays the operands out, runs the tiles and joins the splits.
muon_status run_product(muon_q8_product kind, const void* a, int64_t lda, const float* a_scale,
                        const int8_t* b, int64_t ldb, const float* b_scale, int64_t t, int64_t n,
                        int64_t k, void* out, int64_t ldo, muon_dtype dtype, bool accumulate,
                        void* workspace, size_t workspace_bytes, hipStream_t s) {
  const muon_status bad = product_sizes(kind, t, n, k);
  if (bad != MUON_OK) return bad;
  if (!known(dtype)) return MUON_ERR_INVALID_ARGUMENT;
  const bool i8 = kind == MUON_Q8_MATMUL;
  const int64_t a_cols = i8 ? k : n;
  const int64_t b_rows = kind == MUON_Q8_GRAD_WEIGHT ? t : n;
  const int64_t o_rows = kind == MUON_Q8_GRAD_WEIGHT ? n : t, o_cols = i8 ? n : k;
  if (o_rows == 0 || o_cols == 0) return MUON_OK;
  if (!matrix(out, ldo, o_rows, o_cols, size_of(dtype))) return MUON_ERR_INVALID_ARGUMENT;
  if (t * a_cols > 0 && !matrix(a, lda, t, a_cols, i8 ? 1 : 2)) return MUON_ERR_INVALID_ARGUMENT;
  if (b_rows * k > 0 && !matrix(b, ldb, b_rows, k, 1)) return MUON_ERR_INVALID_ARGUMENT;
  if ((i8 && !a_scale) || (b_rows > 0 && !b_scale) || !aligned(a_scale, 4) || !aligned(b_scale, 4))
    return MUON_ERR_INVALID_ARGUMENT;
  const Choice c = choose(kind, a, lda, b, ldb, t, n, k);
  if (c.bytes > 0) {
    if (workspace_bytes < (size_t)c.bytes) return MUON_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return MUON_ERR_INVALID_ARGUMENT;
  }
  if (c.few)
    return hip(launch_few((const int8_t*)a, lda, a_scale, b, ldb, b_scale, out, ldo, dtype == MUON_BF16,
                          (int)t, (int)n, (int)k, s));
  char* w = (char*)workspace;
  MmParams p = {};
  p.Q = c.pack_q ? w + c.at_q : (const char*)a;
  p.P = c.pack_p ? w + c.at_p : (const char*)b;
  p.ldq = c.ldq;
  p.ldp = c.ldp;
  p.padq = c.padq;
  p.padp = c.padp;
  p.np = c.np;
  p.nq = c.nq;
  p.kd = c.kd;
  p.tile = c.tile;
  p.groups = c.groups;
  p.unaligned = c.unaligned;
  p.direct = c.direct;
  p.splits = c.splits;
  p.sq = a_scale;
  p.sp = b_scale;
  p.out = out;
  p.ldo = ldo;
  p.obf16 = dtype == MUON_BF16;
  p.accumulate = accumulate;
  p.part = c.splits > 1 ? (float*)(w + c.at_part) : nullptr;
  hipError_t e = hipSuccess;
  if (c.pack_q) {
    const int64_t sa = i8 ? 1 : 2;
    e = launch_pack(a, t > 1 ? lda * sa : 0, a_cols * sa, w + c.at_q, c.ldq, t, s);
  }
  if (e == hipSuccess && c.pack_p) e = launch_pack(b, ldb, k, w + c.at_p, c.ldp, b_rows, s);
  if (e == hipSuccess)
    e = launch_mm(p, i8 ? KIND_I8 : kind == MUON_Q8_GRAD_INPUT ? KIND_DX : KIND_DW, s);
  return hip(e);
}

}  // namespace

extern "C" {

muon_status muon_rmsnorm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                 const float* weight, muon_dtype dtype, int64_t rows, int64_t cols,
                                 float eps, void* h, int64_t ldh, void* y, int64_t ldy, int8_t* q,
                                 int64_t ldq, float* scale, float* rstd, hipStream_t stream) {
  const muon_status bad = row_sizes(rows, cols);
  if (bad != MUON_OK) return bad;
  if (!known(dtype) || !(eps >= 0.0f) || std::isinf(eps)) return MUON_ERR_INVALID_ARGUMENT;
  if ((y != nullptr) == (q != nullptr) && rows > 0) return MUON_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MUON_OK;
  const int64_t sz = size_of(dtype);
  if (!matrix(x, ldx, rows, cols, sz) || !matrix(weight, cols, 1, cols, 4) || !matrix(rstd, 1, 1, rows, 4))
    return MUON_ERR_INVALID_ARGUMENT;
  if (residual && (!matrix(residual, ldr, rows, cols, sz) || !matrix(h, ldh, rows, cols, sz)))
    return MUON_ERR_INVALID_ARGUMENT;
  if (y && !matrix(y, ldy, rows, cols, sz)) return MUON_ERR_INVALID_ARGUMENT;
  if (q && (!matrix(q, ldq, rows, cols, 1) || !matrix(scale, 1, 1, rows, 4))) return MUON_ERR_INVALID_ARGUMENT;
  NormParams p = {};
  p.x = x;
  p.res = residual;
  p.w = weight;
  p.h = h;
  p.y = y;
  p.q = q;
  p.scale = scale;
  p.rstd = rstd;
  p.rows = rows;
  p.cols = cols;
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldh = ldh;
  p.ldy = ldy;
  p.ldq = ldq;
  p.eps = (double)eps;
  return hip(launch_norm(p, dtype == MUON_BF16, stream));
}

muon_status muon_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t* workspace_bytes) {
  const muon_status bad = row_sizes(rows, cols);
  if (bad != MUON_OK) return bad;
  if (!workspace_bytes) return MUON_ERR_INVALID_ARGUMENT;
  const int groups = norm_back_groups(rows, cols, true);
  *workspace_bytes = groups > 1 ? (size_t)groups * (size_t)cols * 4 : 0;
  return MUON_OK;
}

muon_status muon_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                                  const float* h_scale, const float* rstd, const float* weight,
                                  const void* dh, int64_t lddh, muon_dtype dtype, int64_t rows,
                                  int64_t cols, void* dx, int64_t lddx, float* dweight, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  const muon_status bad = muon_rmsnorm_backward_workspace(rows, cols, &need);
  if (bad != MUON_OK) return bad;
  if (!known(dtype) || !matrix(dweight, cols, 1, cols, 4)) return MUON_ERR_INVALID_ARGUMENT;
  if (rows == 0) return hip(launch_norm_back_sum(nullptr, dweight, 0, cols, stream));  // an empty sum
  const int64_t sz = size_of(dtype);
  if (!matrix(dy, lddy, rows, cols, sz) || !matrix(h, ldh, rows, cols, h_scale ? 1 : sz) ||
      !matrix(dx, lddx, rows, cols, sz) || !matrix(weight, cols, 1, cols, 4) || !matrix(rstd, 1, 1, rows, 4) ||
      (h_scale && !aligned(h_scale, 4)) || (dh && !matrix(dh, lddh, rows, cols, sz)))
    return MUON_ERR_INVALID_ARGUMENT;
  if (need > 0) {
    if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
    if (!workspace || !aligned(workspace, 256)) return MUON_ERR_INVALID_ARGUMENT;
  }
  NormBackParams p = {};
  p.dy = dy;
  p.h = h;
  p.hscale = h_scale;
  p.rstd = rstd;
  p.w = weight;
  p.dh = dh;
  p.dx = dx;
  p.rows = rows;
  p.cols = cols;
  p.lddy = lddy;
  p.ldh = ldh;
  p.lddh = lddh;
  p.lddx = lddx;
  p.groups = norm_back_groups(rows, cols, dtype == MUON_BF16);
  p.part = p.groups > 1 ? (float*)workspace : dweight;
  hipError_t e = launch_norm_back(p, dtype == MUON_BF16, stream);
  if (e == hipSuccess && p.groups > 1) e = launch_norm_back_sum(p.part, dweight, p.groups, cols, stream);
  return hip(e);
}

muon_status muon_q8_quantize(const void* x, int64_t ldx, muon_dtype dtype, int64_t rows, int64_t cols,
                             int8_t* q, int64_t ldq, float* scale, hipStream_t stream) {
  const muon_status bad = row_sizes(rows, cols);
  if (bad != MUON_OK) return bad;
  if (!known(dtype)) return MUON_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MUON_OK;
  if (!matrix(x, ldx, rows, cols, size_of(dtype)) || !matrix(q, ldq, rows, cols, 1) ||
      !matrix(scale, 1, 1, rows, 4))
    return MUON_ERR_INVALID_ARGUMENT;
  return hip(launch_quantize(x, ldx, q, ldq, scale, rows, cols, dtype == MUON_BF16, stream));
}

muon_status muon_q8_dequantize(const int8_t* q, int64_t ldq, const float* scale, int64_t rows,
                               int64_t cols, void* x, int64_t ldx, muon_dtype dtype,
                               hipStream_t stream) {
  const muon_status bad = row_sizes(rows, cols);
  if (bad != MUON_OK) return bad;
  if (!known(dtype)) return MUON_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MUON_OK;
  if (!matrix(x, ldx, rows, cols, size_of(dtype)) || !matrix(q, ldq, rows, cols, 1) ||
      !matrix(scale, 1, 1, rows, 4))
    return MUON_ERR_INVALID_ARGUMENT;
  return hip(launch_dequantize(q, ldq, scale, x, ldx, rows, cols, dtype == MUON_BF16, stream));
}

muon_status muon_q8_workspace(muon_q8_product product, const void* a, int64_t lda, const void* b,
                              int64_t ldb, int64_t t, int64_t n, int64_t k, size_t* workspace_bytes) {
  if (product < MUON_Q8_MATMUL || product > MUON_Q8_GRAD_WEIGHT || !workspace_bytes)
    return MUON_ERR_INVALID_ARGUMENT;
  const muon_status bad = product_sizes(product, t, n, k);
  if (bad != MUON_OK) return bad;
  *workspace_bytes = (size_t)choose(product, a, lda, b, ldb, t, n, k).bytes;
  return MUON_OK;
}

// (linear8.h)
void muon_l8_choice(int product, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t t, int64_t n,
                    int64_t k, int64_t* out) {
  const Choice c = choose((muon_q8_product)product, a, lda, b, ldb, t, n, k);
  const int64_t T = c.tile, stages = (c.kd + (product == MUON_Q8_MATMUL ? 63 : 31)) / (product == MUON_Q8_MATMUL ? 64 : 32);
  const int64_t tiles = c.few ? 0 : (c.np + T - 1) / T * ((c.nq + T - 1) / T);
  const int64_t v[] = {c.few, T, c.groups, c.unaligned, c.pack_q, c.pack_p, c.direct, tiles - c.direct, c.splits, stages};
  std::copy(std::begin(v), std::end(v), out);
}

muon_status muon_q8_matmul(const int8_t* xq, int64_t ldx, const float* x_scale, const int8_t* wq,
                           int64_t ldw, const float* w_scale, int64_t t, int64_t n, int64_t k, void* y,
                           int64_t ldy, muon_dtype dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream) {
  return run_product(MUON_Q8_MATMUL, xq, ldx, x_scale, wq, ldw, w_scale, t, n, k, y, ldy, dtype, false,
                     workspace, workspace_bytes, stream);
}

muon_status muon_q8_grad_input(const void* dy, int64_t lddy, const int8_t* wq, int64_t ldw,
                               const float* w_scale, int64_t t, int64_t n, int64_t k, void* dx,
                               int64_t lddx, muon_dtype dtype, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  return run_product(MUON_Q8_GRAD_INPUT, dy, lddy, nullptr, wq, ldw, w_scale, t, n, k, dx, lddx, dtype,
                     false, workspace, workspace_bytes, stream);
}

muon_status muon_q8_grad_weight(const void* dy, int64_t lddy, const int8_t* xq, int64_t ldx,
                                const float* x_scale, int64_t t, int64_t n, int64_t k, void* dw,
                                int64_t lddw, muon_dtype dtype, int accumulate, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  return run_product(MUON_Q8_GRAD_WEIGHT, dy, lddy, nullptr, xq, ldx, x_scale, t, n, k, dw, lddw, dtype,
                     accumulate != 0, workspace, workspace_bytes, stream);
}

}  // extern "C"
