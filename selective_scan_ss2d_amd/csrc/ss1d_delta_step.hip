// The gated delta rule for single tokens (serving): one wave holds a tile of columns of one
// sequence and head's state in registers, advances it over the call's few tokens and writes
// it back in place.
//
// Per token, from the state before it: a = S^T k, b = S^T q and q.k are summed in one pass,
//   u = beta (v - e^g a),   o = scale (e^g b + (q.k) u),   S <- e^g S + k u^T,
// so that one reduction across the wave serves both the solution and the output.
//
// Bound by HBM: the fp32 state is read and written once, 2 * 4 * DK * DV bytes per sequence
// and head, against 6 DK DV operations.  256 sequences of 32 heads of 128 x 128: 239 us, 4.5
// TB/s of the 5.0 that a copy reaches; one sequence: 9 us, the latency of its loads.
#include "ss1d_delta_step.h"

namespace ss2d {
namespace delta {
namespace {

template <typename T>
__device__ __forceinline__ float value(const T* p) { return Elem<T>::load(p); }

// kRows rows of the state per lane, kVec columns; kVec lanes' columns are adjacent.  A wave
// covers kLanes * kVec columns and 64 / kLanes groups of kRows rows.
template <typename T, int kRows, int kVec, int kLanes>
__global__ __launch_bounds__(64) void k_delta_step(StepArgs a) {
  constexpr int kGroups = 64 / kLanes;
  const int lane = threadIdx.x;
  const int tiles = (a.DV + kLanes * kVec - 1) / (kLanes * kVec);
  const int64_t unit = blockIdx.x;
  const int tile = static_cast<int>(unit % tiles);
  const int64_t bh = unit / tiles;
  const int hv = static_cast<int>(bh % a.H), hk = hv / a.rep;
  int64_t b = bh / a.H;
  const int r0 = (lane / kLanes) * kRows;
  const int c0 = (tile * kLanes + lane % kLanes) * kVec;
  const bool in = c0 < a.DV;

  int64_t slot = b;
  if (a.slots) {
    slot = a.slots[b];
    if (slot < 0 || slot >= a.S) return;  // a padded row: nothing is read or written
    // Rows that name one slot are further tokens of one sequence, in row order: the first
    // of them does them all, so that no two waves hold the same state.
    bool earlier = false;
    for (int64_t i = lane; i < b; i += 64) earlier |= a.slots[i] == slot;
    if (__any(earlier)) return;
  }
  float* at = a.state + ((slot * a.H + hv) * a.DK + r0) * a.DV + c0;
  float S[kRows][kVec];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if constexpr (kVec == 4) {
      f32x4 x = {0, 0, 0, 0};
      if (in && r0 + i < a.DK) x = *reinterpret_cast<const f32x4*>(at + int64_t(i) * a.DV);
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = x[j];
    } else {
      S[i][0] = in && r0 + i < a.DK ? at[int64_t(i) * a.DV] : 0.0f;
    }
  }
  for (;;) {
    for (int64_t t = 0; t < a.T; ++t) {
      const T* kp = static_cast<const T*>(a.k) + b * a.sk.b + t * a.sk.l + hk * a.sk.h + r0;
      const T* qp = static_cast<const T*>(a.q) + b * a.sq.b + t * a.sq.l + hk * a.sq.h + r0;
      const T* vp = static_cast<const T*>(a.v) + b * a.sv.b + t * a.sv.l + hv * a.sv.h + c0;
      const int64_t row = (b * a.T + t) * a.H + hv;
      const float decay = expf(a.g[row]), beta = a.beta[row];
      float k[kRows], q[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        k[i] = r0 + i < a.DK ? value(kp + i) : 0.0f;
        q[i] = r0 + i < a.DK ? value(qp + i) : 0.0f;
      }
      float sk[kVec] = {}, sq[kVec] = {}, qk = 0.0f;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        qk = fmaf(q[i], k[i], qk);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          sk[j] = fmaf(S[i][j], k[i], sk[j]);
          sq[j] = fmaf(S[i][j], q[i], sq[j]);
        }
      }
      qk = lane_sum<64, kLanes>(qk);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        sk[j] = lane_sum<64, kLanes>(sk[j]);
        sq[j] = lane_sum<64, kLanes>(sq[j]);
      }
      float o[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float v = c0 + j < a.DV ? value(vp + j) : 0.0f;
        const float u = beta * (v - decay * sk[j]);
        o[j] = a.scale * fmaf(qk, u, decay * sq[j]);
#pragma unroll
        for (int i = 0; i < kRows; ++i) S[i][j] = fmaf(k[i], u, decay * S[i][j]);
      }
      if (in && lane < kLanes) {
        T* op = static_cast<T*>(a.o) + row * a.DV + c0;
#pragma unroll
        for (int j = 0; j < kVec; ++j) op[j] = Elem<T>::from_f32(o[j]);
      }
    }
    if (!a.slots) break;
    int64_t next = a.B;  // the next row of the same slot
    for (int64_t base = b + 1; base < a.B && next == a.B; base += 64) {
      const int64_t i = base + lane;
      const uint64_t hit = __ballot(i < a.B && a.slots[i < a.B ? i : b] == slot);
      if (hit) next = base + __ffsll(static_cast<unsigned long long>(hit)) - 1;
    }
    if (next == a.B) break;
    b = next;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!in || r0 + i >= a.DK) continue;
    if constexpr (kVec == 4) {
      f32x4 x;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = S[i][j];
      *reinterpret_cast<f32x4*>(at + int64_t(i) * a.DV) = x;
    } else {
      at[int64_t(i) * a.DV] = S[i][0];
    }
  }
  static_assert(kGroups * kLanes == 64, "a wave is covered once");
}

template <typename T, int kRows4, int kRows1>
int launch_rows(const StepArgs& a, bool vec, hipStream_t st) {
  const int64_t cols = vec ? 32 : 16;
  const int64_t blocks = a.B * a.H * ((a.DV + cols - 1) / cols);
  const dim3 grid(static_cast<unsigned>(blocks)), block(64);
  if (vec) hipLaunchKernelGGL((k_delta_step<T, kRows4, 4, 8>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_step<T, kRows1, 1, 16>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int launch_t(const StepArgs& a, bool vec, hipStream_t st) {
  if (a.DK <= 32) return launch_rows<T, 4, 8>(a, vec, st);
  if (a.DK <= 64) return launch_rows<T, 8, 16>(a, vec, st);
  return launch_rows<T, 16, 32>(a, vec, st);
}

}  // namespace

int launch_step(const StepArgs& a, int dtype, bool vec, hipStream_t st) {
  return dtype == 0 ? launch_t<float>(a, vec, st) : launch_t<uint16_t>(a, vec, st);
}

}  // namespace delta
}  // namespace ss2d
