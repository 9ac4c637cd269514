// Host code of the 8-bit floating-point layer's and of gradient clipping's C
// ABI (float8_api.cpp, clip_api.cpp) under AddressSanitizer
// (tests/test_asan_float8.py), with the launches replaced by functions that look
// at what they are given: every buffer that a kernel would write in the
// workspace is touched at its first and last byte, in an allocation of exactly
// the size that the ABI asked for.  Random sizes, row distances and alignments.
// No GPU is used.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "clip.h"
#include "float8.h"
#include "linear8.h"
#include "muon_clip.h"
#include "muon_float8.h"

static int failures = 0;
static int launches[9];
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
hipError_t launch_pack(const void* src, int64_t, int64_t bytes, void* dst, int64_t ld, int64_t rows, hipStream_t) {
  ++launches[0];
  CHECK(src && in_ws(dst) && rows > 0 && ld % 16 == 0 && ld >= bytes && ld - bytes < 16 && (uintptr_t)dst % 16 == 0);
  touch(dst, rows * ld);
  return hipSuccess;
}
}  // namespace l8
namespace f8 {
static void rows_in_place(const void* p, int64_t ld) { CHECK((uintptr_t)p % 16 == 0 && ld % 16 == 0); }
static void product(const MmParams& p, bool fwd, bool dw) {
  const int64_t T = p.tile, tiles = (p.np + T - 1) / T * ((p.nq + T - 1) / T);
  CHECK((T == 256 && p.groups == 1) || (T == 128 && (p.groups == 1 || p.groups == 2)) || (T == 64 && p.groups == 4));
  CHECK(p.np > 0 && p.nq > 0 && p.splits >= 1 && p.out && p.experts >= 1);
  if (p.ends) {
    CHECK(p.groups == 1 && p.splits == 1 && !p.part);
  } else {
    CHECK(p.direct >= 0 && p.direct <= tiles && (p.splits > 1) == (p.direct < tiles));
  }
  if (p.splits > 1) {
    // (no range of the sum is empty)
    const int64_t stages = fwd ? (p.kd + 127) / 128 : (p.kd + 31) / 32;
    CHECK(stages >= p.splits && in_ws(p.part) && (uintptr_t)p.part % 256 == 0);
    touch(p.part, (tiles - p.direct) * p.splits * T * T * 4);
  }
  if (p.kd == 0) return;
  // what reads 16 bytes at a time: rows 16-byte aligned, and read no further
  // than the next multiple of 16
  rows_in_place(p.P, p.ldp);
  rows_in_place(p.Q, p.ldq);
  const int64_t row = fwd ? p.kd : dw ? 2ll * p.nq : 2ll * p.kd;
  CHECK(p.ldq >= row && (fwd || row % 16 == 0 || in_ws(p.Q)));
}
hipError_t launch_quantize(const FormParams& p, bool, hipStream_t) {
  ++launches[1];
  CHECK(p.count > 0 && p.rows > 0 && p.cols > 0 && p.x && p.q && p.scale);
  return hipSuccess;
}
hipError_t launch_dequantize(const FormParams& p, bool, hipStream_t) {
  ++launches[2];
  CHECK(p.count > 0 && p.rows > 0 && p.cols > 0 && p.x && p.q && p.scale);
  return hipSuccess;
}
hipError_t launch_forward(const MmParams& p, Kind kind, hipStream_t) {
  ++launches[3];
  CHECK(kind == (p.obf16 ? FWD : FWD32) && (kind == FWD || p.tile < 256));
  product(p, true, false);
  return hipSuccess;
}
hipError_t launch_grads(const MmParams& p, Kind kind, hipStream_t) {
  ++launches[4];
  CHECK(kind == DX || kind == DW);
  product(p, false, kind == DW);
  return hipSuccess;
}
hipError_t launch_few(const MmParams& p, int rows, hipStream_t) {
  ++launches[5];
  const int64_t y = p.ends ? row_tiles(p.nq, rows, p.experts) : (p.nq + rows - 1) / rows;
  CHECK((rows == 16 || (rows == 32 && !p.ends)) && y <= 65535 && (p.ends || y == 1));
  if (p.kd > 0) {
    rows_in_place(p.P, p.ldp);
    rows_in_place(p.Q, p.ldq);
  }
  return hipSuccess;
}
}  // namespace f8
namespace clip {
static int64_t g_count, g_scaled;
static int64_t groups(const Table& t, int64_t chunk) {
  int64_t g = 0;
  CHECK(t.num >= 1 && t.num <= kTensors);
  for (int i = 0; i < t.num; ++i) {
    CHECK(t.t[i].n > 0 && t.t[i].first == g);
    g += (t.t[i].n + chunk - 1) / chunk;
  }
  CHECK(g == (int64_t)t.groups && t.chunk == chunk);
  return g;
}
hipError_t launch_small(const Table& t, bool, float, float* norm, hipStream_t) {
  ++launches[6];
  CHECK(norm && groups(t, kSmallChunk) <= kSmallGroups);
  return hipSuccess;
}
hipError_t launch_squares(const Table& t, double* part, int64_t from, hipStream_t) {
  ++launches[7];
  CHECK(from == g_count && in_ws(part));
  g_count += groups(t, t.chunk);
  touch(part + from, groups(t, t.chunk) * 8);
  return hipSuccess;
}
hipError_t launch_norm(const double* part, int64_t count, float* norm, hipStream_t) {
  CHECK(count == g_count && norm && (count == 0 || in_ws(part)));
  return hipSuccess;
}
hipError_t launch_scale(const Table& t, const double* part, int64_t count, float, float* norm, bool first, hipStream_t) {
  ++launches[8];
  CHECK(count == g_count && in_ws(part) && first == (g_scaled == 0) && norm);
  g_scaled += groups(t, t.chunk);
  return hipSuccess;
}
}  // namespace clip
}  // namespace muon

static std::mt19937_64 rng(11);
static int64_t below(int64_t n) { return (int64_t)(rng() % (uint64_t)n); }
static int64_t size(int bits) {
  const int64_t v = 1 + below(1ll << (1 + below(bits)));
  return below(2) ? v : (v + 15) / 16 * 16;
}
static int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

static char* make(size_t bytes) {
  void* p = nullptr;
  g_ws = bytes && posix_memalign(&p, 256, bytes) == 0 ? (char*)p : nullptr;
  g_bytes = (int64_t)bytes;
  return (char*)g_ws;
}

static void products() {
  char* const base = (char*)(uintptr_t)(1 << 20);  // no memory: host code reads no operand
  for (int i = 0; i < 8000; ++i) {
    const muon_f8_product kind = (muon_f8_product)below(3);
    const bool fwd = kind == MUON_F8_MATMUL;
    const int64_t t = below(40) ? size(14) : 0, n = below(40) ? size(14) : 0, k = below(40) ? size(14) : 0;
    const bool grouped = below(2);
    const int64_t experts = grouped ? size(9) : 1;
    const void* a = base + (fwd ? 0 : below(3) ? 0 : 2 * below(32));
    const int64_t lda = fwd ? up16(k) + 16 * below(3) : n + (below(3) ? 0 : below(40)), ldb = up16(k) + 16 * below(3);
    const muon_dtype dtype = below(2) ? MUON_BF16 : MUON_F32;
    const int32_t* ends = grouped ? (const int32_t*)base : nullptr;
    const uint8_t *b = (const uint8_t*)base, *sc = (const uint8_t*)base;
    size_t need = 0;
    CHECK(muon_f8_workspace(kind, a, lda, grouped, experts, t, n, k, dtype, &need) == MUON_OK);
    char* const ws = make(need);
    auto call = [&](size_t bytes) {
      if (fwd) return muon_f8_matmul((const uint8_t*)a, lda, sc, b, ldb, n * ldb, sc, ends, experts, t, n, k, base, n,
                                     dtype, ws, bytes, nullptr);
      if (kind == MUON_F8_GRAD_INPUT) return muon_f8_grad_input(a, lda, b, ldb, n * ldb, sc, ends, experts, t, n, k, base,
                                                                k, dtype, ws, bytes, nullptr);
      return muon_f8_grad_weight(a, lda, b, ldb, sc, ends, experts, t, n, k, base, k, n * k, dtype, 1, ws, bytes, nullptr);
    };
    const int64_t outputs = fwd ? t * n : kind == MUON_F8_GRAD_INPUT ? t * k : n * k;
    CHECK(call(need) == MUON_OK);
    if (need && outputs) CHECK(call(need - 1) == MUON_ERR_WORKSPACE_TOO_SMALL);
    std::free(ws);

    const int64_t count = below(20) ? size(6) : 0, rows = below(20) ? size(16) : 0, cols = below(20) ? size(12) : 0;
    const int64_t ldq = up16(cols);
    CHECK(muon_f8_quantize(base, cols, rows * cols, dtype, count, rows, cols, i % 2 ? 1 : 128, (uint8_t*)base, ldq,
                           rows * ldq, (uint8_t*)base, nullptr) == MUON_OK);
    CHECK(muon_f8_dequantize(b, ldq, rows * ldq, sc, count, rows, cols, i % 2 ? 1 : 128, base, cols, rows * cols, dtype,
                             nullptr) == MUON_OK);
  }
}

static void clips() {
  for (int i = 0; i < 3000; ++i) {
    const int num = (int)(below(4) ? below(6) : below(400));
    std::vector<int64_t> numel(num);
    std::vector<muon_dtype> types(num), otypes(num);
    std::vector<const void*> g(num);
    std::vector<void*> out(num);
    char* at = (char*)(uintptr_t)(1 << 20);
    char* const norm = at - 4;
    for (int j = 0; j < num; ++j) {
      numel[j] = below(10) ? size(below(4) ? 11 : 30) : 0;
      types[j] = below(2) ? MUON_BF16 : MUON_F32;
      otypes[j] = below(2) ? types[j] : MUON_F32;
      g[j] = at;
      at += numel[j] * 4;
      out[j] = otypes[j] == types[j] && below(2) ? (void*)g[j] : at;
      at += numel[j] * 4;
    }
    size_t need = 0;
    CHECK(muon_clip_workspace(num, numel.data(), types.data(), &need) == MUON_OK);
    char* const ws = make(need);
    auto norm_call = [&](size_t bytes) {
      muon::clip::g_count = muon::clip::g_scaled = 0;
      return muon_grad_norm(num, g.data(), numel.data(), types.data(), (float*)norm, ws, bytes, nullptr);
    };
    auto clip_call = [&](size_t bytes, char* n) {
      muon::clip::g_count = muon::clip::g_scaled = 0;
      return muon_clip_grads(num, g.data(), numel.data(), types.data(), out.data(), otypes.data(), 1.0f, (float*)n, ws,
                             bytes, nullptr);
    };
    CHECK(norm_call(need) == MUON_OK);
    CHECK(clip_call(need, norm) == MUON_OK);
    CHECK(muon::clip::g_scaled == muon::clip::g_count);
    if (need) {
      CHECK(norm_call(need - 1) == MUON_ERR_WORKSPACE_TOO_SMALL);
      CHECK(clip_call(need - 1, norm) == MUON_ERR_WORKSPACE_TOO_SMALL);
      for (int j = 0; j < num; ++j)
        if (numel[j] > 0) {
          CHECK(clip_call(need, (char*)out[j]) == MUON_ERR_INVALID_ARGUMENT);
          break;
        }
    }
    std::free(ws);
  }
}

int main() {
  products();
  clips();
  for (const int n : launches) CHECK(n > 0);
  std::printf("%d failures\n", failures);
  return failures != 0;
}
