// Arguments of the token-order scan's single-token kernel.
#pragma once

#include "ss1d_sequences.h"
#include "ss2d_device.h"

namespace ss2d {
namespace sscan {

constexpr int kStepCh = 64;  // channels of a block, four lanes each

struct StepArgs {
  const void *u, *dt, *z, *Bs, *Cs;   // (B, T, D), z NULL for none; (B, T, G, N)
  const float *A_log, *Ds, *bias;
  Slots slots;                        // of the B rows, into state
  float* state;                       // (S, D, N)
  void* y;                            // (B, T, D)
  RowStrides su, sd, sz, sb, sc;
  int64_t sbg, scg;
  int T, D, G, N;
  bool whole;                         // N is 16 or 32, and its rows lie on four values
  int rows;                           // rows of a block
};

int launch_scan_step(const StepArgs& a, int dtype, hipStream_t st);

}  // namespace sscan
}  // namespace ss2d
