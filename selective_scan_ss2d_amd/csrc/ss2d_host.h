// Host-side helpers shared by the C entry points: the failure record, stream-ordered scratch
// from the library's pool (both in ss2d_abi.hip), and checked sizes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace ss2d {

// Records a failed HIP call for ss2d_last_hip_error and returns SS2D_ERR_HIP.
int host_hip_fail(hipError_t e);
// Stream-ordered scratch on the current device; release it with hipFreeAsync on `st`.
int host_scratch_alloc(char** ws, size_t bytes, hipStream_t st);

// The same for callers that can bring scratch of their own: SS2D_ERR_SCRATCH while `st` is being
// captured, where the allocation would become a node of the graph.
int host_scratch_outside_graphs(char** ws, size_t bytes, hipStream_t st);

constexpr int64_t kHostMaxElems = int64_t(1) << 62;

inline bool host_mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a == 0 || b == 0) { *out = 0; return true; }
  if (a > kHostMaxElems / b) return false;
  *out = a * b;
  return true;
}

inline bool host_overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const auto pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return a && b && pa < pb + static_cast<uintptr_t>(bbytes) &&
         pb < pa + static_cast<uintptr_t>(abytes);
}

inline size_t host_align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace ss2d
