// The token-order selective scan for single tokens (serving): four lanes hold a channel's states in
// registers, advance them over the call's few tokens and write them back in place.
#include "ss1d_scan_step.h"

namespace ss2d {
namespace sscan {
namespace {

// kNS adjacent states of a lane, vec: on kNS * 4 bytes and none past N.
template <int kNS>
__device__ __forceinline__ void take_states(const float* p, int left, bool vec, float other, float* x) {
  if constexpr (kNS >= 4) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < kNS; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + i);
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kNS; ++i) x[i] = i < left ? p[i] : other;
}

template <typename T, int kNS>
__global__ __launch_bounds__(64) void k_scan_step(StepArgs a) {
  const int lane = threadIdx.x, s = lane & 3;
  const int64_t unit = blockIdx.x;
  const int blocks = (a.D + 15) / 16;
  const int ch = static_cast<int>(unit % blocks) * 16 + (lane >> 2);
  int64_t b = unit / blocks;
  const bool on = ch < a.D;
  const int d = on ? ch : a.D - 1, g = d / (a.D / a.G);
  const int n0 = s * kNS, left = a.N - n0;

  int64_t slot = b;
  if (a.slots) {
    slot = a.slots[b];
    if (slot < 0 || slot >= a.S) return;  // a padded row: nothing is read or written
    // Rows that name one slot are further tokens of one sequence, in row order: the first of
    // them does them all, so that no two waves hold the same state.
    bool earlier = false;
    for (int64_t i = lane; i < b; i += 64) earlier |= a.slots[i] == slot;
    if (__any(earlier)) return;
  }
  float* at = a.state + (slot * a.D + d) * a.N + n0;
  float h[kNS], Ap[kNS];
  take_states<kNS>(at, left, a.vec, 0.0f, h);
  take_states<kNS>(a.A_log + int64_t(d) * a.N + n0, left, a.vec, 0.0f, Ap);
#pragma unroll
  for (int i = 0; i < kNS; ++i) Ap[i] = -expf(Ap[i]) * kLog2e;
  const float bias = a.bias[d], skip = a.Ds[d];
  for (;;) {
    for (int64_t t = 0; t < a.T; ++t) {
      const float u = Elem<T>::load(static_cast<const T*>(a.u) + b * a.su.b + t * a.su.l + d);
      const float raw = Elem<T>::load(static_cast<const T*>(a.dt) + b * a.sd.b + t * a.sd.l + d);
      const float z = a.z ? Elem<T>::load(static_cast<const T*>(a.z) + b * a.sz.b + t * a.sz.l + d) : 0.0f;
      const T* pB = static_cast<const T*>(a.Bs) + b * a.sb.b + t * a.sb.l + g * a.sbg + n0;
      const T* pC = static_cast<const T*>(a.Cs) + b * a.sc.b + t * a.sc.l + g * a.scg + n0;
      T B[kNS], C[kNS];
#pragma unroll
      for (int i = 0; i < kNS; ++i) {
        B[i] = i < left ? pB[i] : T(0);
        C[i] = i < left ? pC[i] : T(0);
      }
      const float delta = softplus_f32(raw + bias), w = delta * u;
      float y = 0.0f;
#pragma unroll
      for (int i = 0; i < kNS; ++i) {
        h[i] = fmaf(exp2_hw(delta * Ap[i]), h[i], w * Elem<T>::to_f32(B[i]));
        y = fmaf(Elem<T>::to_f32(C[i]), h[i], y);
      }
      y = fmaf(skip, u, group_sum<4>(y));
      if (a.z) y *= silu_f32(z);
      if (on && s == 0) static_cast<T*>(a.y)[(b * a.T + t) * a.D + d] = Elem<T>::from_f32(y);
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
  if (!on) return;
  if constexpr (kNS >= 4) {
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < kNS; i += 4)
        *reinterpret_cast<float4*>(at + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kNS; ++i)
    if (i < left) at[i] = h[i];
}

template <typename T>
int launch_t(const StepArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.B * ((a.D + 15) / 16))), block(64);
  if (a.N <= 4) hipLaunchKernelGGL((k_scan_step<T, 1>), grid, block, 0, st, a);
  else if (a.N <= 8) hipLaunchKernelGGL((k_scan_step<T, 2>), grid, block, 0, st, a);
  else if (a.N <= 16) hipLaunchKernelGGL((k_scan_step<T, 4>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_scan_step<T, 8>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_scan_step(const StepArgs& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_t<float>(a, st) : launch_t<uint16_t>(a, st);
}

}  // namespace sscan
}  // namespace ss2d
