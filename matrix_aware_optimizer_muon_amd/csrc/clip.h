// Internal launch interface of gradient clipping (include/muon_clip.h):
// clip.hip holds the kernels, clip_api.cpp validates and lays the work out.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {
namespace clip {

// A tensor of a launch: a workgroup for each `chunk` of its elements, the first
// of which is the launch's workgroup `first`.
struct Tensor {
  const void* g;
  void* out;
  int64_t n;
  uint32_t first;
  uint16_t gbf16, obf16;
};
// Tensors per launch: what kernel arguments hold (4 KB).
constexpr int kTensors = 124;
struct Table {
  Tensor t[kTensors];
  int num;
  uint32_t groups;    // workgroups of the launch
  int64_t chunk;      // elements, a multiple of 2048
};
static_assert(sizeof(Table) + 64 <= 4096, "kernel arguments");

// All of it for few elements, in one launch: at most kSmallGroups workgroups'
// shares at a chunk of kSmallChunk.
constexpr int64_t kSmallChunk = 2048, kSmallGroups = 16;
hipError_t launch_small(const Table& t, bool scaled, float max_norm, float* norm, hipStream_t s);

// part[from + workgroup] = the sum of its squares.
hipError_t launch_squares(const Table& t, double* part, int64_t from, hipStream_t s);
// norm[0] from `count` partial sums (one workgroup).
hipError_t launch_norm(const double* part, int64_t count, float* norm, hipStream_t s);
// out = g * factor, the factor from all partial sums; the first launch writes
// the norm.
hipError_t launch_scale(const Table& t, const double* part, int64_t count, float max_norm, float* norm, bool first,
                        hipStream_t s);

}  // namespace clip
}  // namespace muon
