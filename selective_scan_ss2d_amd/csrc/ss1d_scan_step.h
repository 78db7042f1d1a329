// Arguments of the token-order scan's single-token kernel.
#pragma once

#include "ss1d_sequences.h"
#include "ss2d_device.h"

namespace ss2d {
namespace sscan {

struct StepArgs {
  const void *u, *dt, *z, *Bs, *Cs;   // (B, T, D), z NULL for none; (B, T, G, N)
  const float *A_log, *Ds, *bias;
  const int32_t* slots;               // (B) or NULL (row b's state is state[b])
  float* state;                       // (S, D, N)
  void* y;                            // (B, T, D)
  RowStrides su, sd, sz, sb, sc;
  int64_t sbg, scg;
  int64_t B, T, S;
  int D, G, N;
  bool vec;                           // state and A_log in pieces of 16 bytes
};

int launch_scan_step(const StepArgs& a, int dtype, hipStream_t st);

}  // namespace sscan
}  // namespace ss2d
