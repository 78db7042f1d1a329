// Arguments and shared pieces of the token-order selective scan's kernels.
//   delta = softplus(dt_raw + dt_bias),  h_n <- exp(A_n delta) h_n + delta B_n u,  A = -exp(A_log),
//   y = (sum_n C_n h_n + Ds u) SiLU(z),
// channels last: u, dt_raw, z, y (B, L, D), B and C (B, L, G, N), group g for D / G channels.
//
// Four lanes (a quad) share a channel, each with kNS adjacent ones of its states; a wave covers 16
// channels, lane / 4 counting them, and a block of 4 waves 64 channels of one group.  Time advances
// in tiles of kTile steps: B and C of a tile lie in LDS as fp32, double buffered; lane s of a quad
// owns steps s, s + 4, ... of the tile, loads their u, dt_raw and z (a tile ahead), and shares
// delta and delta u with the quad through DPP.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "ss1d_sequences.h"
#include "ss2d_device.h"
#include "ss2d_lanes.h"

namespace ss2d {
namespace sscan {

constexpr int kMaxN = 32;
constexpr int kBlockCh = 64;    // channels of a block
constexpr int kThreads = 256;

// Steps of a tile, by the states of a lane: the adjoint holds a tile's states and decays.
constexpr int tile_of(int ns) { return ns <= 4 ? 16 : 8; }
// States per lane for N: the smallest of 1, 2, 4, 8 that holds N on four lanes.
inline int lane_states(int64_t N) { return N <= 4 ? 1 : (N <= 8 ? 2 : (N <= 16 ? 4 : 8)); }
inline int tile_steps(int64_t N) { return tile_of(lane_states(N)); }

struct Args {
  const void *u, *dt, *z, *Bs, *Cs;
  const float *A_log, *Ds, *bias;
  const float *h0;      // (S, D, N) or NULL
  void* y;              // (B, L, D)
  float* ht;            // (S, D, N) or NULL
  float* marks;         // states before every tile, (tile slots, D, N), or NULL
  // segments: end states from a zero start and sums of delta, then start states
  float *seg_end, *seg_delta, *seg_start;
  RowStrides su, sd, sz, sb, sc;
  int64_t sbg, scg;     // strides from one group of B, of C to the next
  Sequences q;
  int64_t seglen;       // tokens of a segment (a multiple of the tile), 0: whole sequences
  int64_t units;        // segments, or sequences
  int D, G, N;
  int cbg;              // channel blocks (of kBlockCh) of a group
  int lanes;            // of a channel in the forward: 4 or 16
  // backward
  const void* dy;
  const float* dht;
  void *du, *ddt, *dz, *dB, *dC;
  float *dA, *dD, *dbias, *dh0;
  float* bc_parts;      // (cbg, T, G, 2 N)
  float* par_parts;     // (units, D, N + 2): dA, dD, dbias
};

int launch_scan_tokens(const Args& a, int dtype, hipStream_t st);
int launch_scan_segments(const Args& a, int dtype, hipStream_t st);  // seg_end, seg_delta
int launch_scan_join(const Args& a, bool back, hipStream_t st);      // seg_start
int launch_scan_adjoint(const Args& a, int dtype, hipStream_t st);
int launch_scan_adjoint_segments(const Args& a, int dtype, hipStream_t st);
int launch_scan_sums(const Args& a, int dtype, hipStream_t st);

// ---- device pieces -----------------------------------------------------------------------------
// A log2(e) of a state.  Held at the largest fp32 where exp(A_log) passes it: a step of delta 0 (past the
// end of a tile, or of a lane past the channels) then leaves the state alone, and a decay of 0 times the
// rate stays 0 in the gradients, where infinity would make both NaN.  (The comparison keeps a NaN.)
__device__ __forceinline__ float decay_rate(float A_log) {
  const float v = -expf(A_log) * kLog2e;
  return v < -FLT_MAX ? -FLT_MAX : v;
}

// Sums four values over a quad: lane s gets the sum of v_s.
__device__ __forceinline__ float quad_scatter_sum(float v0, float v1, float v2, float v3, bool odd,
                                                  bool high) {
  const float a = (odd ? v1 : v0) + quad_perm<1, 0, 3, 2>(odd ? v0 : v1);
  const float b = (odd ? v3 : v2) + quad_perm<1, 0, 3, 2>(odd ? v2 : v3);
  return (high ? b : a) + quad_perm<2, 3, 0, 1>(high ? a : b);
}

// kNS states of a lane from LDS or memory rows on 16 bytes.
template <int kNS> __device__ __forceinline__ void load_states(const float* p, float* x) {
  if constexpr (kNS % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kNS; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      x[i] = v.x;
      x[i + 1] = v.y;
      x[i + 2] = v.z;
      x[i + 3] = v.w;
    }
  } else if constexpr (kNS == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x;
    x[1] = v.y;
  } else {
    x[0] = *p;
  }
}

template <int I, int N, typename F> __device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<I + 1, N>(f);
  }
}

// The place of a block: its unit, group and first channel.  The channel blocks of a unit follow
// each other on one XCD, whose L2 then holds the lines of u, dt_raw, z, B and C that they share.
struct Place {
  int64_t unit;
  int g, cb, c0;   // group, channel block of it, first channel within the group
};
__device__ __forceinline__ Place place_of(const Args& a, int channels, unsigned lin, unsigned total) {
  const unsigned id = xcd_local_order(lin, total);
  const unsigned cbg = (a.D / a.G + channels - 1) / channels, per = a.G * cbg;
  Place p;
  p.unit = uniform(id / per);
  const unsigned r = id % per;
  p.g = r / cbg;
  p.cb = r % cbg;
  p.c0 = p.cb * channels;
  return p;
}

// B and C of a tile of kTile steps as a block's 256 threads load them: a thread takes one n of one of
// the two, and every kRows-th step.  Element e = thread + 256 m is step e / (2 kNP), B before C.
template <typename T, int kTile, int kNP> struct Operands {
  static constexpr int kRows = kThreads / (2 * kNP), kPer = kTile > kRows ? kTile / kRows : 1;
  const T* p;
  int stride, step;
  bool on;
  T raw[kPer];
  __device__ __forceinline__ void start(const Args& a, int64_t b, int64_t row, int g, bool both, bool b_only) {
    const int tid = threadIdx.x, n = tid % kNP;
    const bool is_c = tid / kNP % 2;
    step = tid / (2 * kNP);
    on = n < a.N && step < kTile && (both || is_c != b_only);
    const RowStrides s = is_c ? a.sc : a.sb;
    p = static_cast<const T*>(is_c ? a.Cs : a.Bs) + b * s.b + (row + step) * s.l + g * (is_c ? a.scg : a.sbg) + n;
    stride = static_cast<int>(s.l);
  }
  // the first `rows` steps of the tile; then on by `moved` steps
  __device__ __forceinline__ void load(int rows, int moved) {
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      raw[m] = T(0);
      if (on && step + m * kRows < rows) raw[m] = element(p, opaque(stride) * uint32_t(m * kRows));
    }
    p += int64_t(moved) * stride;
  }
};

}  // namespace sscan
}  // namespace ss2d
