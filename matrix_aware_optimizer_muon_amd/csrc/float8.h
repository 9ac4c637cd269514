// Internal launch interface of the 8-bit floating-point layer's kernels
// (include/muon_float8.h): float8_rows.hip holds the 8-bit form and back,
// float8_forward.hip and float8_grads.hip the products, float8_api.cpp validates and dispatches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {
namespace f8 {

constexpr int kBlock = 128;        // values that share a scale
constexpr int kMaxExperts = 1024;

// `count` matrices of rows x cols; a scale per 128 values of a row
// (block_rows 1) or per 128 x 128 (block_rows 128).
struct FormParams {
  void* x;                 // read by quantize, written by dequantize
  uint8_t* q;
  uint8_t* scale;
  int64_t count, rows, cols;
  int64_t ldx, sx, ldq, sq;  // row and matrix distances, elements
  int block_rows;
};
hipError_t launch_quantize(const FormParams& p, bool bf16, hipStream_t s);
hipError_t launch_dequantize(const FormParams& p, bool bf16, hipStream_t s);

// Products: C[q][p] = sum_k P(p, k) Q(q, k), C row-major with the P index
// contiguous.  An operand is K-contiguous (its rows are p or q) or K-major
// (its rows are k).
enum Kind {
  FWD = 0,    // P, Q e4m3, both K-contiguous, on the 8-bit matrix cores
  FWD32 = 1,  // the same widened to bf16 on the way from LDS (fp32 sums)
  DX = 2,     // P e4m3 weights K-major, Q bf16 K-contiguous (input gradient)
  DW = 3      // P e4m3 rows K-major, Q bf16 K-major (weight gradient)
};

struct MmParams {
  const char* P;
  const char* Q;
  const uint8_t* sp;        // scales of P: weights' (FWD, DX) or rows' (DW)
  const uint8_t* sq;        // scales of Q (FWD)
  const int* ends;          // grouped: each expert's end, else nullptr
  int64_t ldp, ldq;         // bytes
  int64_t stride_p;         // bytes from one expert's weights to the next's
  int64_t stride_sp;        // and of their scales
  int64_t stride_o;         // elements from one expert's weight gradient to the next's
  int ldsp, ldsq;           // bytes of a row of scales
  int experts;
  int np, nq, kd;           // output columns, output rows, contraction (grouped: of all experts)
  int tile;                 // 256, 128 or 64
  int groups;               // wave groups that share a tile's K: 1 or 2 (tile 128), 4 (tile 64)
  int direct;               // tiles of one workgroup; the others are split (not grouped)
  int splits;               // contraction ranges of a split tile
  void* out;                // bf16 or fp32
  int64_t ldo;              // elements
  bool obf16, accumulate;
  float* part;              // [split tiles][splits][tile][tile]
};
hipError_t launch_forward(const MmParams& p, Kind kind, hipStream_t s);
hipError_t launch_grads(const MmParams& p, Kind kind, hipStream_t s);
// The split tiles' partial sums added (called by the two).
hipError_t launch_sums(const MmParams& p, hipStream_t s);

// Row tiles of T that t rows need at most, however they fall on the experts (a
// partly filled one each), and one for rows of no expert.
inline int64_t row_tiles(int64_t t, int64_t T, int64_t experts) { return t / T + (experts < t ? experts : t) + 1; }

// The forward product for few rows of x (of each expert): `rows` (16, or 32 of
// one matrix) at a time against 16 rows of w, which is read straight from memory.
hipError_t launch_few(const MmParams& p, int rows, hipStream_t s);

}  // namespace f8
}  // namespace muon

// How a product of these arguments runs (muon_f8_product), so that tests can
// see which kernels their sizes reach; not part of the ABI.  out: kind, rows
// of the few rows' kernel (0: tiles), tile, wave groups, a laid out again,
// tiles of one workgroup, tiles that are split, their splits.
extern "C" void muon_f8_choice(int product, const void* a, int64_t lda, int grouped, int64_t experts, int64_t t,
                               int64_t n, int64_t k, int bf16, int64_t* out);
