// Internal launch interface of the 8-bit linear layer's kernels
// (include/muon_linear8.h): linear8_rows.hip holds the row-wise ones,
// linear8_gemm.hip the products, linear8_api.cpp validates and dispatches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {
namespace l8 {

// Widest row the row-wise kernels hold in registers (16 waves of 64 lanes,
// 4 chunks of 8 columns each).
constexpr int64_t kMaxCols = 32768;

struct NormParams {
  const void* x;
  const void* res;     // nullptr: no residual
  const float* w;
  void* h;             // x + res, written only with a residual
  void* y;             // normalised rows, or nullptr with q
  int8_t* q;
  float* scale;
  float* rstd;
  int64_t rows, cols;
  int64_t row0;        // the launch's first row (set at the launch)
  int64_t ldx, ldr, ldh, ldy, ldq;
  double eps;
};

struct NormBackParams {
  const void* dy;
  const void* h;       // rows of the planned type, or int8 with hscale
  const float* hscale;
  const float* rstd;
  const float* w;
  const void* dh;      // nullable
  void* dx;
  float* part;         // [groups][cols] sums of dw, or dw itself (1 group)
  int64_t rows, cols;
  int64_t lddy, ldh, lddh, lddx;
  int groups;
};

// bf16 selects the 16-bit type of every typed row, else fp32.
hipError_t launch_norm(const NormParams& p, bool bf16, hipStream_t s);
hipError_t launch_norm_back(const NormBackParams& p, bool bf16, hipStream_t s);
hipError_t launch_norm_back_sum(const float* part, float* dw, int groups, int64_t cols, hipStream_t s);
int norm_back_groups(int64_t rows, int64_t cols, bool bf16);  // never more for fp32
hipError_t launch_quantize(const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale,
                           int64_t rows, int64_t cols, bool bf16, hipStream_t s);
hipError_t launch_dequantize(const int8_t* q, int64_t ldq, const float* scale, void* x, int64_t ldx,
                             int64_t rows, int64_t cols, bool bf16, hipStream_t s);

// Products: C[q][p] = sum_k P(p, k) Q(q, k), C row-major with the P index
// contiguous.  An operand is K-contiguous (its rows are p or q) or K-major
// (its rows are k).
enum ProductKind {
  KIND_I8 = 0,      // int8 x int8 -> int32, both K-contiguous
  KIND_DX = 1,      // P int8 K-major, Q bf16 K-contiguous (input gradient)
  KIND_DW = 2       // P int8 K-major, Q bf16 K-major (weight gradient)
};

struct MmParams {
  const char* P;
  const char* Q;
  int64_t ldp, ldq;         // bytes
  int padp, padq;           // bytes that may be read after the last row
  int np, nq, kd;           // output columns, output rows, contraction
  int tile;                 // 256, 128 or 64
  int groups;               // wave groups that share a tile's K: 1 or 2 (tile 128), 4 (tile 64)
  bool unaligned;           // an operand that the DMA would read has rows off 16 bytes (not tile 256)
  int direct;               // tiles of one workgroup; the others are split
  int splits;               // contraction ranges of a split tile
  const float* sp;          // KIND_I8: per output column; else per row of P
  const float* sq;          // KIND_I8: per output row
  void* out;                // bf16 or fp32
  int64_t ldo;              // elements
  bool obf16, accumulate;
  float* part;              // [split tiles][splits][tile][tile], int32 bits for KIND_I8
};

hipError_t launch_mm(const MmParams& p, ProductKind kind, hipStream_t s);

// The product for few rows of x (generated tokens, short batches): no tiles,
// no alignment, reads the weights once.  Against tiles that share K, weights
// from memory, in us: one row, 18944 x 3584 13.8 and 23.0, 18944 x 16384 65 and
// 80, 1024 x 8192 11.0 and 9.9 (6.9 and 9.0 where the last-level cache holds
// them), but 1024 x 65536 68 and 22 (few workgroups, long sums); up to 32 rows
// the reads of x count as well: 32 rows, 2048 x 4096 8.4 and 13.7, 2048 x 8192
// 13.6 and 11.9, 18944 x 3584 31 and 25.
inline bool few_rows(int64_t t, int64_t n, int64_t k) {
  return t <= 16 ? k <= 8192 || n >= 16384 : t <= 32 && k <= 4096 && n * k <= 1 << 24;
}
hipError_t launch_few(const int8_t* xq, int64_t ldx, const float* xs, const int8_t* wq, int64_t ldw,
                      const float* ws, void* y, int64_t ldy, bool bf16, int t, int n, int k, hipStream_t s);

// dst[r][0 .. ld) = src[r][0 .. bytes), zeros beyond; ld a multiple of 16,
// dst 16-byte aligned, src at any address.
hipError_t launch_pack(const void* src, int64_t lds, int64_t bytes, void* dst, int64_t ld, int64_t rows,
                       hipStream_t s);

}  // namespace l8
}  // namespace muon

// How a product of these arguments runs (muon_q8_product), so that tests can
// see which kernels their sizes reach; not part of the ABI.  out: few rows'
// kernel, tile, wave groups, unaligned, operands a and b laid out again, tiles
// of one workgroup, tiles that are split, their splits, stages of the whole sum.
extern "C" void muon_l8_choice(int product, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t t,
                               int64_t n, int64_t k, int64_t* out);
