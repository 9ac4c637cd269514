// Host code of the 8-bit linear layer's C ABI (linear8_api.cpp) under
// AddressSanitizer (tests/test_asan_linear8.py), with the launches replaced by
// functions that look at what they are given: every buffer that a kernel would
// write in the workspace is touched at its first and last byte, in an
// allocation of exactly the size that the ABI asked for.  Random sizes, row
// distances and alignments, and the refusals.  No GPU is used.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "linear8.h"
#include "muon_linear8.h"

using namespace muon::l8;

static int failures = 0;
static int launches[8];
#define CHECK(cond)                                                    \
  do {                                                                 \
    if (!(cond)) {                                                     \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #cond);          \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

static void touch(const void* p, int64_t bytes) {
  volatile char* c = (volatile char*)p;
  c[0] = 1;
  c[bytes - 1] = 1;
}

// the workspace of the call that is running, and whether an address is in it
static const char* g_ws = nullptr;
static int64_t g_bytes = 0;
static bool in_ws(const void* p) { return (const char*)p >= g_ws && (const char*)p < g_ws + g_bytes; }

namespace muon {
namespace l8 {
hipError_t launch_norm(const NormParams& p, bool, hipStream_t) {
  ++launches[0];
  CHECK(p.rows > 0 && p.cols >= 1 && p.cols <= kMaxCols && (p.y != nullptr) != (p.q != nullptr));
  return hipSuccess;
}
int norm_back_groups(int64_t rows, int64_t, bool) { return (int)(rows < 512 ? rows : 512); }
hipError_t launch_norm_back(const NormBackParams& p, bool, hipStream_t) {
  ++launches[1];
  if (p.groups > 1) touch(p.part, (int64_t)p.groups * p.cols * 4);
  return hipSuccess;
}
hipError_t launch_norm_back_sum(const float* part, float*, int groups, int64_t cols, hipStream_t) {
  ++launches[2];
  if (groups > 0) touch(part, groups * cols * 4);
  return hipSuccess;
}
hipError_t launch_quantize(const void*, int64_t, int8_t*, int64_t, float*, int64_t, int64_t, bool, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_dequantize(const int8_t*, int64_t, const float*, void*, int64_t, int64_t, int64_t, bool,
                             hipStream_t) {
  return hipSuccess;
}
hipError_t launch_pack(const void* src, int64_t, int64_t bytes, void* dst, int64_t ld, int64_t rows, hipStream_t) {
  ++launches[3];
  CHECK(src && in_ws(dst) && rows > 0 && ld % 16 == 0 && ld >= bytes && ld - bytes < 16 && (uintptr_t)dst % 16 == 0);
  touch(dst, rows * ld);
  return hipSuccess;
}
hipError_t launch_few(const int8_t*, int64_t, const float*, const int8_t*, int64_t, const float*, void*, int64_t, bool,
                      int t, int n, int k, hipStream_t) {
  ++launches[4];
  CHECK(t >= 1 && t <= 32 && n >= 1 && k >= 0);
  return hipSuccess;
}
hipError_t launch_mm(const MmParams& p, ProductKind kind, hipStream_t) {
  ++launches[5];
  const int64_t T = p.tile, tiles = (p.np + T - 1) / T * ((p.nq + T - 1) / T);
  CHECK((T == 256 && p.groups == 1 && !p.unaligned) || (T == 128 && (p.groups == 1 || p.groups == 2)) ||
        (T == 64 && p.groups == 4));
  CHECK(p.direct >= 0 && p.direct <= tiles && p.splits >= 1 && (p.splits > 1) == (p.direct < tiles));
  if (p.splits > 1) {
    const int64_t stages = (p.kd + (kind == KIND_I8 ? 63 : 31)) / (kind == KIND_I8 ? 64 : 32);
    CHECK(stages >= p.splits && in_ws(p.part) && (uintptr_t)p.part % 256 == 0);
    touch(p.part, (tiles - p.direct) * p.splits * T * T * 4);
  }
  if (p.kd > 0) {
    // what reads by DMA reads whole 16 bytes: rows 16-byte aligned, and as wide
    const bool q_dma = !p.unaligned, p_dma = kind == KIND_I8 && !p.unaligned;
    const int64_t qc = kind == KIND_I8 ? p.kd : kind == KIND_DX ? 2ll * p.kd : 2ll * p.nq;
    const int64_t pc = kind == KIND_I8 ? p.kd : p.np, qr = kind == KIND_DW ? p.kd : p.nq,
                  pr = kind == KIND_I8 ? p.np : p.kd;
    if (q_dma) CHECK((uintptr_t)p.Q % 16 == 0 && (qr <= 1 || p.ldq % 16 == 0) && (qc + p.padq) % 16 == 0);
    if (p_dma) CHECK((uintptr_t)p.P % 16 == 0 && (pr <= 1 || p.ldp % 16 == 0) && (pc + p.padp) % 16 == 0);
    // what reads through registers has at least 16 bytes
    if (!q_dma) CHECK((qr - 1) * p.ldq + qc + p.padq >= 16);
    if (!p_dma) CHECK((pr - 1) * p.ldp + pc + p.padp >= 16);
  }
  return hipSuccess;
}
}  // namespace l8
}  // namespace muon

static std::mt19937_64 rng(7);
static int64_t below(int64_t n) { return (int64_t)(rng() % (uint64_t)n); }
static int64_t size(int bits) {
  const int64_t v = 1 + below(1ll << (1 + below(bits)));
  return below(2) ? v : (v + 15) / 16 * 16;
}

static char* make(size_t bytes) {
  void* p = nullptr;
  return bytes && posix_memalign(&p, 256, bytes) == 0 ? (char*)p : nullptr;
}

int main() {
  const char* const base = (const char*)(uintptr_t)(1 << 20);  // no memory: host code reads no operand
  for (int i = 0; i < 8000; ++i) {
    const int kind = (int)below(3);
    const int64_t t = below(40) ? size(14) : 0, n = below(40) ? size(14) : 0, k = below(40) ? size(14) : 0;
    const int64_t ac = kind == 0 ? k : n, pad = below(3) == 0 ? below(40) : 0, sa = kind == 0 ? 1 : 2;
    const void* a = base + (below(3) ? 0 : sa * below(32));
    const void* b = base + (below(3) ? 0 : below(32));
    const int64_t lda = ac + pad, ldb = k + (below(3) ? 0 : below(40));
    const float* sc = (const float*)base;
    size_t need = 0;
    CHECK(muon_q8_workspace((muon_q8_product)kind, a, lda, b, ldb, t, n, k, &need) == MUON_OK);
    char* ws = make(need);
    g_ws = ws;
    g_bytes = (int64_t)need;
    void* out = (void*)base;
    auto call = [&](size_t bytes) {
      if (kind == 0) return muon_q8_matmul((const int8_t*)a, lda, sc, (const int8_t*)b, ldb, sc, t, n, k, out, n,
                                           MUON_F32, ws, bytes, nullptr);
      if (kind == 1) return muon_q8_grad_input(a, lda, (const int8_t*)b, ldb, sc, t, n, k, out, k, MUON_BF16, ws,
                                               bytes, nullptr);
      return muon_q8_grad_weight(a, lda, (const int8_t*)b, ldb, sc, t, n, k, out, k, MUON_F32, 1, ws, bytes, nullptr);
    };
    const int64_t outputs = kind == 0 ? t * n : kind == 1 ? t * k : n * k;
    CHECK(call(need) == MUON_OK);
    if (need && outputs) CHECK(call(need - 1) == MUON_ERR_WORKSPACE_TOO_SMALL);
    std::free(ws);
    int64_t v[10];
    muon_l8_choice(kind, a, lda, b, ldb, t, n, k, v);
    CHECK((v[0] == 0 || kind == 0) && v[8] >= 1);

    const int64_t rows = below(20) ? size(20) : 0, cols = 1 + below(kMaxCols);
    size_t part = 0;
    CHECK(muon_rmsnorm_backward_workspace(rows, cols, &part) == MUON_OK);
    ws = make(part);
    CHECK(muon_rmsnorm_backward(base, cols, base, cols, nullptr, sc, sc, nullptr, 0, MUON_BF16, rows, cols, out, cols,
                                (float*)out, ws, part, nullptr) == MUON_OK);
    if (part) CHECK(muon_rmsnorm_backward(base, cols, base, cols, sc, sc, sc, base, cols, MUON_F32, rows, cols, out,
                                          cols, (float*)out, ws, part - 1, nullptr) == MUON_ERR_WORKSPACE_TOO_SMALL);
    std::free(ws);
    CHECK(muon_rmsnorm_forward(base, cols, i % 2 ? base : nullptr, cols, sc, MUON_F32, rows, cols, 1e-6f, out, cols,
                               i % 3 ? out : nullptr, cols, i % 3 ? nullptr : (int8_t*)out, cols, (float*)out,
                               (float*)out, nullptr) == MUON_OK);
  }
  // refusals: sizes, null and misaligned pointers, types
  const void* p = base;
  const float* s = (const float*)base;
  void* o = (void*)base;
  size_t z;
  CHECK(muon_q8_workspace((muon_q8_product)3, p, 1, p, 1, 1, 1, 1, &z) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_workspace(MUON_Q8_MATMUL, p, 1, p, 1, 1, 1, 1, nullptr) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_workspace(MUON_Q8_MATMUL, p, 1, p, 1, -1, 1, 1, &z) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_workspace(MUON_Q8_MATMUL, p, 1, p, 1, 1, 1, 131072, &z) == MUON_ERR_UNSUPPORTED);
  CHECK(muon_q8_matmul(nullptr, 8, s, (const int8_t*)p, 8, s, 4, 4, 8, o, 4, MUON_F32, nullptr, 0, nullptr) ==
        MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_grad_input((const char*)p + 1, 8, (const int8_t*)p, 8, s, 4, 8, 8, o, 8, MUON_F32, nullptr, 0,
                           nullptr) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_grad_weight(p, 8, (const int8_t*)p, 8, s, 4, 8, 8, o, 8, (muon_dtype)2, 0, nullptr, 0, nullptr) ==
        MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_rmsnorm_backward_workspace(4, 0, &z) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_rmsnorm_backward_workspace(4, 8, nullptr) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_rmsnorm_backward_workspace(4, kMaxCols + 1, &z) == MUON_ERR_UNSUPPORTED);
  CHECK(muon_q8_quantize(p, 8, MUON_F32, 4, 8, nullptr, 8, (float*)o, nullptr) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_quantize(p, 8, MUON_F32, 4, 8, (int8_t*)o, 8, (float*)o, nullptr) == MUON_OK);
  CHECK(muon_q8_dequantize((const int8_t*)p, 8, nullptr, 4, 8, o, 8, MUON_F32, nullptr) == MUON_ERR_INVALID_ARGUMENT);
  CHECK(muon_q8_dequantize((const int8_t*)p, 8, s, 4, 8, o, 8, MUON_F32, nullptr) == MUON_OK);
  for (int i = 0; i < 6; ++i) CHECK(launches[i] > 0);
  std::printf("%d failures\n", failures);
  return failures != 0;
}
