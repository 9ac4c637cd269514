// C ABI of gradient clipping (include/muon_clip.h): validation, the layout of
// the chunks, and the launch sequence.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "clip.h"
#include "muon_clip.h"

using namespace muon::clip;

namespace {

bool known(muon_dtype t) { return t == MUON_F32 || t == MUON_BF16; }
int64_t size_of(muon_dtype t) { return t == MUON_BF16 ? 2 : 4; }
bool aligned(const void* p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }
muon_status hip(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_ERR_HIP; }

constexpr int64_t kMaxElements = 1ll << 40;

muon_status sizes(int num, const int64_t* numel, const muon_dtype* dtypes, int64_t* total) {
  if (num < 0 || (num > 0 && (!numel || !dtypes))) return MUON_ERR_INVALID_ARGUMENT;
  int64_t& n = *total;
  n = 0;
  for (int i = 0; i < num; ++i) {
    if (numel[i] < 0 || !known(dtypes[i])) return MUON_ERR_INVALID_ARGUMENT;
    if (numel[i] > kMaxElements || (n += numel[i]) > kMaxElements) return MUON_ERR_UNSUPPORTED;
  }
  return MUON_OK;
}

// Elements that a workgroup takes: some 4096 workgroups, two rounds of eight per
// compute unit (932 M fp32 elements: 602 and 1377 us for the two passes, with
// one round 629 and 1450), none with less than 2048.
int64_t chunk_of(int64_t total) { return std::max<int64_t>(1, (total + 4096 * 2048 - 1) / (4096 * 2048)) * 2048; }

int64_t groups_of(int num, const int64_t* numel, int64_t chunk) {
  int64_t g = 0;
  for (int i = 0; i < num; ++i) g += (numel[i] + chunk - 1) / chunk;
  return g;
}

// The launches' tables, tensors without elements left out.
template <typename L>
hipError_t tables(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes, void* const* out,
                  const muon_dtype* out_dtypes, int64_t chunk, L launch) {
  Table t;
  t.chunk = chunk;
  t.num = 0;
  t.groups = 0;
  int64_t from = 0;
  for (int i = 0; i <= num; ++i) {
    if (t.num > 0 && (i == num || t.num == kTensors)) {
      const hipError_t e = launch(t, from);
      if (e != hipSuccess) return e;
      from += t.groups;
      t.num = 0;
      t.groups = 0;
    }
    if (i == num || numel[i] == 0) continue;
    t.t[t.num++] = {g[i], out ? out[i] : nullptr, numel[i], t.groups, (uint16_t)(dtypes[i] == MUON_BF16),
                    (uint16_t)(out && out_dtypes[i] == MUON_BF16)};
    t.groups += (uint32_t)((numel[i] + chunk - 1) / chunk);
  }
  return hipSuccess;
}

// Whether one launch does (a workgroup that goes through more, or through many
// small tensors, takes longer than two launches).
bool small(int num, const int64_t* numel) {
  int64_t groups = 0;
  for (int i = 0; i < num && groups <= kSmallGroups; ++i) groups += (numel[i] + kSmallChunk - 1) / kSmallChunk;
  return groups > 0 && groups <= kSmallGroups;
}

muon_status check(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes, float* norm,
                  void* workspace, size_t workspace_bytes, int64_t* chunk, int64_t* groups) {
  int64_t total;
  const muon_status bad = sizes(num, numel, dtypes, &total);
  if (bad != MUON_OK) return bad;
  if (!norm || !aligned(norm, 4) || (num > 0 && !g)) return MUON_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < num; ++i)
    if (numel[i] > 0 && (!g[i] || !aligned(g[i], size_of(dtypes[i])))) return MUON_ERR_INVALID_ARGUMENT;
  *chunk = chunk_of(total);
  *groups = groups_of(num, numel, *chunk);
  // (a launch has fewer than 2^32 threads)
  if (*groups >= 1 << 24) return MUON_ERR_UNSUPPORTED;
  if (workspace_bytes < (size_t)*groups * 8) return MUON_ERR_WORKSPACE_TOO_SMALL;
  if (*groups > 0 && (!workspace || !aligned(workspace, 256))) return MUON_ERR_INVALID_ARGUMENT;
  return MUON_OK;
}

// Whether something that is written overlaps anything else.
bool overlaps(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes, void* const* out,
              const muon_dtype* out_dtypes, const float* norm) {
  struct Range {
    uintptr_t from, to;
    bool written;
  };
  std::vector<Range> r;
  r.reserve(2 * (size_t)num + 1);
  r.push_back({(uintptr_t)norm, (uintptr_t)norm + 4, true});
  for (int i = 0; i < num; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t a = (uintptr_t)g[i], b = (uintptr_t)out[i];
    r.push_back({b, b + (uintptr_t)(numel[i] * size_of(out_dtypes[i])), true});
    if (a != b) r.push_back({a, a + (uintptr_t)(numel[i] * size_of(dtypes[i])), false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
  uintptr_t any = 0, written = 0;  // ends so far
  for (const Range& v : r) {
    if (v.from < (v.written ? any : written)) return true;
    any = std::max(any, v.to);
    if (v.written) written = std::max(written, v.to);
  }
  return false;
}

}  // namespace

extern "C" {

muon_status muon_clip_workspace(int num, const int64_t* numel, const muon_dtype* dtypes, size_t* workspace_bytes) {
  if (!workspace_bytes) return MUON_ERR_INVALID_ARGUMENT;
  int64_t total;
  const muon_status bad = sizes(num, numel, dtypes, &total);
  if (bad != MUON_OK) return bad;
  *workspace_bytes = (size_t)groups_of(num, numel, chunk_of(total)) * 8;
  return MUON_OK;
}

muon_status muon_grad_norm(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes, float* norm,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int64_t chunk, groups;
  const muon_status bad = check(num, g, numel, dtypes, norm, workspace, workspace_bytes, &chunk, &groups);
  if (bad != MUON_OK) return bad;
  if (small(num, numel))
    return hip(tables(num, g, numel, dtypes, nullptr, nullptr, kSmallChunk,
                      [&](const Table& t, int64_t) { return launch_small(t, false, 0.0f, norm, stream); }));
  double* const part = (double*)workspace;
  hipError_t e = tables(num, g, numel, dtypes, nullptr, nullptr, chunk,
                        [&](const Table& t, int64_t from) { return launch_squares(t, part, from, stream); });
  if (e == hipSuccess) e = launch_norm(part, groups, norm, stream);
  return hip(e);
}

muon_status muon_clip_grads(int num, const void* const* g, const int64_t* numel, const muon_dtype* dtypes,
                            void* const* out, const muon_dtype* out_dtypes, float max_norm, float* norm,
                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int64_t chunk, groups;
  const muon_status bad = check(num, g, numel, dtypes, norm, workspace, workspace_bytes, &chunk, &groups);
  if (bad != MUON_OK) return bad;
  if (!(max_norm >= 0.0f) || (num > 0 && (!out || !out_dtypes))) return MUON_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < num; ++i) {
    if (!known(out_dtypes[i])) return MUON_ERR_INVALID_ARGUMENT;
    if (numel[i] == 0) continue;
    if (!out[i] || !aligned(out[i], size_of(out_dtypes[i]))) return MUON_ERR_INVALID_ARGUMENT;
    if (out[i] == g[i] && out_dtypes[i] != dtypes[i]) return MUON_ERR_INVALID_ARGUMENT;
  }
  try {
    if (overlaps(num, g, numel, dtypes, out, out_dtypes, norm)) return MUON_ERR_INVALID_ARGUMENT;
  } catch (const std::bad_alloc&) {
    return MUON_ERR_UNSUPPORTED;
  }
  if (small(num, numel))
    return hip(tables(num, g, numel, dtypes, out, out_dtypes, kSmallChunk,
                      [&](const Table& t, int64_t) { return launch_small(t, true, max_norm, norm, stream); }));
  double* const part = (double*)workspace;
  hipError_t e = tables(num, g, numel, dtypes, nullptr, nullptr, chunk,
                        [&](const Table& t, int64_t from) { return launch_squares(t, part, from, stream); });
  if (e == hipSuccess && groups == 0) e = launch_norm(part, 0, norm, stream);
  if (e == hipSuccess)
    e = tables(num, g, numel, dtypes, out, out_dtypes, chunk, [&](const Table& t, int64_t from) {
      return launch_scale(t, part, groups, max_norm, norm, from == 0, stream);
    });
  return hip(e);
}

}  // extern "C"
