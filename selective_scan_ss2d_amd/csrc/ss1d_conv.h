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
constexpr int kThreads = 256;

struct Args {
  const void* x;       // (B, L, D), rows apart by sx
  const float *w, *b;  // (D, KW), (D) or NULL
  const void* h0;      // (S, KW - 1, D) or NULL
  void *y, *ht;        // (B, L, D); (S, KW - 1, D) or NULL
  RowStrides sx;
  Sequences q;
  int64_t units;
  int run;             // tokens of a unit: at least kMaxKW - 1, so that only a sequence's first unit
                       // reads its initial state
  int D, KW, silu;
  // backward
  const void *dy, *dht;
  void *dx, *dh0;
  float *dw, *db;
  float* parts;        // (unit blocks, KW + 1, D)
  // step
  void* state;         // (S, KW - 1, D)
  Slots slots;
};

// Threads that share a row of D channels of a block, in pieces of `width` channels.
int lanes_of(int64_t D, int width);
// Tokens of a unit, of B rows (`rows`, 0: of packed sequences, S of them).
int run_of(int64_t rows, int64_t tokens, int64_t S, int64_t D, int KW, int dtype, bool backward);
// Blocks along the units of the backward.
int64_t unit_blocks(const Args& a, int width);
// Channels of a thread: four (vec), or one.  Eight bfloat16 values, 16 bytes, take too many registers:
// forward 150 against 96, 48.6 against 44.6 us (12007 tokens x 4096); backward 246 against 144, 55.7
// against 44.0 us (128 x 197 tokens x 768).
inline int width_of(bool vec) { return vec ? 4 : 1; }

int launch_conv(const Args& a, int dtype, bool vec, hipStream_t st);
int launch_conv_bwd(const Args& a, int dtype, bool vec, hipStream_t st);
int launch_conv_sums(const Args& a, int64_t blocks, hipStream_t st);
int launch_conv_step(const Args& a, int dtype, bool vec, hipStream_t st);

}  // namespace conv
}  // namespace ss2d
