// Arguments and shared pieces of the block norm's kernels: the norms before and after a block
// with its gate, residual scale and residual connection.
//   p = Norm(h; w_post, b_post) (h without w_post),  p <- p SiLU(z),
//   y = residual + res_scale p,  n = Norm(y; w_pre, b_pre).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ss2d_device.h"
#include "ss2d_lanes.h"

namespace ss2d {
namespace norm {

struct Args {
  const void *h, *z, *residual;             // data type; residual: y's type
  const float *scale;                       // (G, D)
  const float *w_post, *b_post, *w_pre, *b_pre;
  void *y, *n;
  // backward
  const void *dy, *dn;                      // dy: y's type
  void *dh, *dz, *dres;
  float *dscale, *dw_post, *db_post, *dw_pre, *db_pre;
  float* parts;                             // partial sums, (blocks, kSums, D)
  float* scale_parts;                       // (G, parts of a group, D)
  int64_t B, L;                             // channels first: (B, D, L); else B * L rows of D
  int D;
  int64_t G;                                // groups of res_scale (1 without one)
  int64_t group;                            // rows (channels first: images) of a group
  int64_t groups_per_block, blocks_per_group;
  int layer;
  float eps;
};

constexpr int kMaxD = 8192;        // channels last: 8 values a thread, 1024 threads
constexpr int kMaxDFirst = 1024;   // channels first
constexpr int64_t kMaxLFirst = int64_t(1) << 24;  // 64 planes of fp32 within 32-bit offsets
constexpr int kSums = 4;           // dw_post, db_post, dw_pre, db_pre

// SiLU and its derivative sigmoid(z) (1 + z (1 - sigmoid(z))).
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_hw(-v * kLog2e));
}
// z sigmoid(z) with SiLU(-inf) = -0 rather than NaN.
__device__ __forceinline__ float gate_value(float z, float sg) { return sg == 0.0f ? -0.0f : z * sg; }
__device__ __forceinline__ float gate_slope(float z, float sg) {
  return sg == 0.0f ? 0.0f : (sg == 1.0f ? 1.0f : sg * fmaf(z, 1.0f - sg, 1.0f));
}

// kind: bit 0, fp32 y (with bfloat16 data); types (data, y).
int launch_norm(const Args& a, int dtype, int ytype, bool first, bool vec, hipStream_t st);
int launch_norm_bwd(const Args& a, int dtype, int ytype, bool first, bool vec, hipStream_t st);
int launch_norm_sums(const Args& a, int64_t blocks, hipStream_t st);
// Blocks of the backward's launch; fills groups_per_block and blocks_per_group.
int64_t plan_norm_bwd(Args* a, bool first);

}  // namespace norm
}  // namespace ss2d
