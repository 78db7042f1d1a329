// Arguments of the gated delta rule's single-token kernel.
#pragma once

#include "ss1d_delta.h"

namespace ss2d {
namespace delta {

struct StepArgs {
  const void *q, *k, *v;   // (B, T, HK, DK), (B, T, HK, DK), (B, T, H, DV)
  const float *g, *beta;   // (B, T, H)
  const int32_t* slots;    // (B) or NULL (row b's state is state[b])
  float* state;            // (S, H, DK, DV)
  void* o;                 // (B, T, H, DV)
  Strides sq, sk, sv;
  int64_t B, T, S;
  int H, HK, rep, DK, DV;
  float scale;
};

// vec: the state's rows are a multiple of 4 values and start on 16 bytes.
int launch_step(const StepArgs& a, int dtype, bool vec, hipStream_t st);

}  // namespace delta
}  // namespace ss2d
