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

#include <cstdint>

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
  int cbg;              // channel blocks of a group
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
// Sums four values over a quad: lane s gets the sum of v_s.
__device__ __forceinline__ float quad_scatter_sum(float v0, float v1, float v2, float v3, bool odd,
                                                  bool high) {
  const float a = (odd ? v1 : v0) + quad_perm<1, 0, 3, 2>(odd ? v0 : v1);
  const float b = (odd ? v3 : v2) + quad_perm<1, 0, 3, 2>(odd ? v2 : v3);
  return (high ? b : a) + quad_perm<2, 3, 0, 1>(high ? a : b);
}

// The place of a block: its unit, group and first channel.  The channel blocks of a unit follow
// each other on one XCD, whose L2 then holds the lines of u, dt_raw, z, B and C that they share.
struct Place {
  int64_t unit;
  int g, cb, c0;   // group, channel block of it, first channel within the group
};
__device__ __forceinline__ Place place_of(const Args& a, unsigned lin, unsigned total) {
  const unsigned id = xcd_local_order(lin, total);
  const unsigned per = a.G * a.cbg;
  Place p;
  p.unit = id / per;
  const unsigned r = id % per;
  p.g = r / a.cbg;
  p.cb = r % a.cbg;
  p.c0 = p.cb * kBlockCh;
  return p;
}

}  // namespace sscan
}  // namespace ss2d
