// Arguments of the group norm's kernels, channels last:
//   y = act((x - mean) r w + b),  r = 1 / sqrt(var + eps),
// mean and var over the L positions and the C / G channels of a group, act = SiLU or nothing.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ss2d_device.h"
#include "ss2d_lanes.h"

namespace ss2d {
namespace group {

struct Args {
  const void* x;                // (B, L, C)
  const float *w, *b;           // (C) or NULL
  void* y;
  float* stats;                 // (B, G, 2): mean, r
  int64_t B, L;
  int C, G, cg;                 // cg = C / G
  int silu;
  float eps;
  // backward
  const void* dy;
  void* dx;
  float *dw, *db;
  int given;                    // stats hold the forward's
  float* parts;                 // (B, chunks, 2, C): a channel's mean and sum of squares about it,
                                // or its sums of the gradient and of gradient times unit value
  float* sums;                  // (B, G, 2): the groups' sums of the backward
  // one block for a set of whole groups of an image
  int set, sets;                // channels of a set; sets of C
  // or chunks of positions
  int64_t chunk, chunks;        // positions of a chunk; chunks of L
};

// How a call is cut: rows held in registers by one block per set of groups (rows, threads), or in
// chunks (rows 0).
struct Plan {
  int width, rows, threads, set;
};
Plan plan(int64_t B, int64_t L, int64_t C, int64_t G, int dtype, bool vec, bool backward);
int64_t chunk_positions(int64_t B, int64_t L, int64_t C, int dtype);

int launch_group(const Args& a, const Plan& p, int dtype, hipStream_t st);
int launch_group_bwd(const Args& a, const Plan& p, int dtype, hipStream_t st);

}  // namespace group
}  // namespace ss2d
