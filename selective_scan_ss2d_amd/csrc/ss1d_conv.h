// Arguments of the short causal convolution's kernels, per channel and channels last:
//   y_t = act(b + sum_{j < KW} w_j x_{t - KW + 1 + j}),   act = SiLU or nothing,
// where the KW - 1 inputs before a sequence are its initial state, or zero.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ss1d_sequences.h"
#include "ss2d_device.h"

namespace ss2d {
namespace conv {

constexpr int kMaxKW = 8;
constexpr int kRun = 32;      // tokens of a unit (at least kMaxKW - 1, so that only a sequence's
                              // first unit reads its initial state)
constexpr int kThreads = 256;

struct Args {
  const void* x;       // (B, L, D), rows apart by sx
  const float *w, *b;  // (D, KW), (D) or NULL
  const void* h0;      // (S, KW - 1, D) or NULL
  void *y, *ht;        // (B, L, D); (S, KW - 1, D) or NULL
  RowStrides sx;
  Sequences q;
  int64_t units;
  int D, KW, silu;
  // backward
  const void *dy, *dht;
  void *dx, *dh0;
  float *dw, *db;
  float* parts;        // (unit blocks, KW + 1, D)
  // step
  void* state;         // (S, KW - 1, D)
  const int32_t* slots;
};

// Threads that share a row of D channels of a block, in pieces of `width` channels.
int lanes_of(int64_t D, int width);
// Blocks along the units of the backward.
int64_t unit_blocks(const Args& a, int width);
// Channels of a thread: one 16-byte piece (vec) or one.
inline int width_of(int dtype, bool vec) { return vec ? (dtype == 0 ? 4 : 8) : 1; }

int launch_conv(const Args& a, int dtype, bool vec, hipStream_t st);
int launch_conv_bwd(const Args& a, int dtype, bool vec, hipStream_t st);
int launch_conv_sums(const Args& a, int64_t blocks, hipStream_t st);
int launch_conv_step(const Args& a, int dtype, bool vec, hipStream_t st);

}  // namespace conv
}  // namespace ss2d
