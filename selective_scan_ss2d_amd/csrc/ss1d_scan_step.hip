// The token-order selective scan for single tokens (serving): four lanes hold a channel's states in
// registers, advance them over the call's few tokens and write them back in place.
// What bounds it is HBM, the states in and out: 256 rows of 4096 channels of 16 states, 143 MB, in 32 us
// (4.5 TB/s); of one row the latency of its loads, 3.5 us.
#include "ss1d_scan.h"
#include "ss1d_scan_step.h"

namespace ss2d {
namespace sscan {
namespace {

// kNS adjacent values of a lane from memory.  kWhole: N is four lanes' values, and the rows lie on
// the size of four of them; else one by one, none past N.
template <int kNS, bool kWhole, typename T>
__device__ __forceinline__ void take(const T* p, int left, T* x) {
  if constexpr (kWhole) {
    struct alignas(4 * sizeof(T)) Four { T v[4]; };
#pragma unroll
    for (int i = 0; i < kNS; i += 4) {
      const Four f = *reinterpret_cast<const Four*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i + j] = f.v[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNS; ++i) x[i] = i < left ? p[i] : T(0);
  }
}

// A token as it comes from memory; the rows of b and t by uniform pointers, the lane's place in them
// by 32-bit offsets.
template <typename T, int kNS, bool kWhole, bool kGate> struct Token {
  T u, dt, z, B[kNS], C[kNS];
  __device__ __forceinline__ void load(const StepArgs& a, int b, int t, uint32_t d, uint32_t nb, uint32_t nc, int left) {
    u = element(static_cast<const T*>(a.u) + b * a.su.b + t * a.su.l, opaque(d));
    dt = element(static_cast<const T*>(a.dt) + b * a.sd.b + t * a.sd.l, opaque(d));
    z = kGate ? element(static_cast<const T*>(a.z) + b * a.sz.b + t * a.sz.l, opaque(d)) : T(0);
    take<kNS, kWhole>(&element(static_cast<const T*>(a.Bs) + b * a.sb.b + t * a.sb.l, opaque(nb)), left, B);
    take<kNS, kWhole>(&element(static_cast<const T*>(a.Cs) + b * a.sc.b + t * a.sc.l, opaque(nc)), left, C);
  }
};

// A block takes 64 channels, whose rows of u, dt_raw, z and y fill lines, of a.rows rows one after the
// other, each one's state and first token loaded while the one before is computed.  (Blocks of 16
// channels, four times as many: 300 rows of 3000 channels 25.9 us for 24.7, one of 4096 as fast.)
template <typename T, int kNS, bool kWhole, bool kGate>
__global__ __launch_bounds__(4 * kStepCh) void k_scan_step(StepArgs a) {
  __shared__ uint32_t seen[2];
  const int lane = threadIdx.x & 63, s = lane & 3;
  const int blocks = (a.D + kStepCh - 1) / kStepCh;
  const int ch = static_cast<int>(blockIdx.x % blocks) * kStepCh + static_cast<int>(threadIdx.x >> 2);
  const int b0 = static_cast<int>(blockIdx.x / blocks) * a.rows, n = min(a.slots.rows - b0, a.rows);
  const bool on = ch < a.D;
  const uint32_t d = on ? ch : a.D - 1, g = d / (a.D / a.G), n0 = s * kNS;
  const uint32_t nb = g * uint32_t(a.sbg) + n0, nc = g * uint32_t(a.scg) + n0, at = d * a.N + n0;
  const int left = a.N - static_cast<int>(n0);
  const int64_t state_row = int64_t(a.D) * a.N;
  float Ap[kNS];
  take<kNS, kWhole>(a.A_log + at, left, Ap);
  const float bias = a.bias[d], skip = a.Ds[d];
  find_repeats(a.slots, b0, n, seen);
  float h_in[kNS] = {};
  Token<T, kNS, kWhole, kGate> in{};
  int slot_in = slot_of(a.slots, b0, 0, seen);
  auto fetch = [&](int b) {
    if (slot_in < 0) return;
    take<kNS, kWhole>(&element(static_cast<const float*>(a.state) + slot_in * state_row, opaque(at)), left, h_in);
    in.load(a, b, 0, d, nb, nc, left);
  };
  fetch(b0);
#pragma unroll
  for (int i = 0; i < kNS; ++i) Ap[i] = decay_rate(Ap[i]);
  for (int i = 0; i < n; ++i) {
    int b = b0 + i;
    const int slot = slot_in;
    float h[kNS];
    Token<T, kNS, kWhole, kGate> x = in;
#pragma unroll
    for (int k = 0; k < kNS; ++k) h[k] = h_in[k];
    if (i + 1 < n) {
      slot_in = slot_of(a.slots, b0, i + 1, seen);
      fetch(b + 1);
    }
    if (slot < 0) continue;
    const bool more = a.slots.at && (__builtin_amdgcn_readfirstlane(seen[1]) >> i & 1);
    for (;;) {
      for (int t = 0;;) {
        const float u = Elem<T>::to_f32(x.u);
        const float delta = softplus_f32(Elem<T>::to_f32(x.dt) + bias), w = delta * u;
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < kNS; ++k) {
          h[k] = fmaf(exp2_hw(delta * Ap[k]), h[k], w * Elem<T>::to_f32(x.B[k]));
          y = fmaf(Elem<T>::to_f32(x.C[k]), h[k], y);
        }
        y = fmaf(skip, u, group_sum<4>(y));
        if (kGate) y *= silu_f32(Elem<T>::to_f32(x.z));
        if (on && s == 0) element(static_cast<T*>(a.y) + (int64_t(b) * a.T + t) * a.D, opaque(d)) = Elem<T>::from_f32(y);
        if (++t >= a.T) break;
        x.load(a, b, t, d, nb, nc, left);
      }
      if (!more) break;
      b = next_of(a.slots, b, slot);
      if (b >= a.slots.rows) break;
      x.load(a, b, 0, d, nb, nc, left);
    }
    if (!on) continue;
    float* to = &element(a.state + slot * state_row, opaque(at));
    if constexpr (kWhole) {
#pragma unroll
      for (int k = 0; k < kNS; k += 4)
        *reinterpret_cast<float4*>(to + k) = make_float4(h[k], h[k + 1], h[k + 2], h[k + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < kNS; ++k)
        if (k < left) to[k] = h[k];
    }
  }
}

template <typename T, int kNS, bool kWhole>
int launch_gate(const StepArgs& a, hipStream_t st) {
  const int64_t rows = (a.slots.rows + a.rows - 1) / a.rows;
  const dim3 grid(static_cast<unsigned>(rows * ((a.D + kStepCh - 1) / kStepCh))), block(4 * kStepCh);
  if (a.z) hipLaunchKernelGGL((k_scan_step<T, kNS, kWhole, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_scan_step<T, kNS, kWhole, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int launch_t(const StepArgs& a, hipStream_t st) {
  if (a.whole) return a.N == 16 ? launch_gate<T, 4, true>(a, st) : launch_gate<T, 8, true>(a, st);
  if (a.N <= 4) return launch_gate<T, 1, false>(a, st);
  if (a.N <= 8) return launch_gate<T, 2, false>(a, st);
  return a.N <= 16 ? launch_gate<T, 4, false>(a, st) : launch_gate<T, 8, false>(a, st);
}

}  // namespace

int launch_scan_step(const StepArgs& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_t<float>(a, st) : launch_t<uint16_t>(a, st);
}

}  // namespace sscan
}  // namespace ss2d
