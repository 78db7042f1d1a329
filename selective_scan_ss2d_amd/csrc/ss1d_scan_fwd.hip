// The token-order selective scan, forward: whole sequences or segments of them.
#include <algorithm>

#include "ss1d_scan.h"

namespace ss2d {
namespace sscan {
namespace {

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

// kOut: outputs, end states and marks; else a segment's end state from a zero start and its sum
// of delta.
template <typename T, int kNS, bool kOut>
__global__ __launch_bounds__(kThreads) void k_scan_tokens(Args a) {
  constexpr int kTile = tile_of(kNS), kOwn = kTile / 4, kNP = 4 * kNS;
  constexpr int kBC = kTile * 2 * kNP, kPer = (kBC + kThreads - 1) / kThreads;
  __shared__ __align__(16) float sBC[2][kBC];  // rows of a step: B, then C

  const Place p = place_of(a, blockIdx.x, gridDim.x);
  int64_t idx = 0;
  const Sequence q = a.seglen ? sequence_of(a.q, p.unit, a.seglen, &idx) : sequence(a.q, p.unit);
  const int64_t t_begin = idx * a.seglen;
  if (idx > 0 && t_begin >= q.len) return;  // an empty unit
  const int64_t t_end = a.seglen ? min(q.len, t_begin + a.seglen) : q.len;

  const int tid = threadIdx.x, lane = tid & 63, s = lane & 3;
  const int Dg = a.D / a.G, c = p.c0 + (tid >> 2);
  const bool on = c < Dg, wave_on = p.c0 + (tid >> 6) * 16 < Dg;
  const int d = p.g * Dg + (on ? c : Dg - 1);
  const bool odd = s & 1, high = s & 2;

  float Ap[kNS], h[kNS];
#pragma unroll
  for (int i = 0; i < kNS; ++i) {
    const int n = s * kNS + i;
    // states past N decay to nothing; their B and C are zero
    Ap[i] = n < a.N ? -expf(a.A_log[int64_t(d) * a.N + n]) * kLog2e : -1.0f;
    h[i] = 0.0f;
  }
  if constexpr (kOut) {
    const float* start = a.seglen ? a.seg_start : a.h0;
    if (start) {
      start += (p.unit * a.D + d) * a.N;  // without segments a unit is a sequence
#pragma unroll
      for (int i = 0; i < kNS; ++i)
        if (s * kNS + i < a.N) h[i] = start[s * kNS + i];
    }
  }
  const float bias = a.bias[d], skip = a.Ds[d];

  // rows of the next tile: uniform pointers, and the lane's offsets from them
  const int64_t row = q.begin + t_begin;
  const T* pu = static_cast<const T*>(a.u) + q.b * a.su.b + row * a.su.l;
  const T* pd = static_cast<const T*>(a.dt) + q.b * a.sd.b + row * a.sd.l;
  const T* pz = kOut && a.z ? static_cast<const T*>(a.z) + q.b * a.sz.b + row * a.sz.l : nullptr;
  const T* pB = static_cast<const T*>(a.Bs) + q.b * a.sb.b + row * a.sb.l + p.g * a.sbg;
  const T* pC = static_cast<const T*>(a.Cs) + q.b * a.sc.b + row * a.sc.l + p.g * a.scg;
  T* py = kOut ? static_cast<T*>(a.y) + (q.b * a.q.L + row) * a.D : nullptr;
  const uint32_t ul = a.su.l, dl_ = a.sd.l, zl = a.sz.l;

  T ru[kOwn], rd[kOwn], rz[kOwn], rbc[kPer];
  auto fetch = [&](int64_t left) {
    const bool full = left >= kTile;
    const int last = full ? kTile - 1 : static_cast<int>(left) - 1;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const uint32_t r = min(s + 4 * j, last);
      ru[j] = pu[r * ul + d];
      rd[j] = pd[r * dl_ + d];
      if (kOut && pz) rz[j] = pz[r * zl + d];
    }
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const int e = tid + m * kThreads;
      const int n = e % kNP, which = e / kNP % 2, t = e / (2 * kNP);
      rbc[m] = T(0);
      if (e < kBC && n < a.N && t <= last) {
        if (which == 0) rbc[m] = pB[uint32_t(t) * uint32_t(a.sb.l) + n];
        else if (kOut) rbc[m] = pC[uint32_t(t) * uint32_t(a.sc.l) + n];
      }
    }
    pu += kTile * a.su.l;
    pd += kTile * a.sd.l;
    if (kOut && pz) pz += kTile * a.sz.l;
    pB += kTile * a.sb.l;
    pC += kTile * a.sc.l;
  };

  float* mark = nullptr;
  if (kOut && a.marks)
    mark = a.marks + ((first_unit(a.q, q, kTile) + t_begin / kTile) * a.D + d) * a.N + s * kNS;
  float sum_delta = 0.0f;
  int64_t left = t_end - t_begin;
  if (left > 0) fetch(left);
  for (int buf = 0; left > 0; left -= kTile, buf ^= 1) {
#pragma unroll
    for (int m = 0; m < kPer; ++m)
      if (tid + m * kThreads < kBC) sBC[buf][tid + m * kThreads] = Elem<T>::to_f32(rbc[m]);
    float u[kOwn], delta[kOwn], z[kOwn], w[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      u[j] = Elem<T>::to_f32(ru[j]);
      delta[j] = Elem<T>::to_f32(rd[j]);
      z[j] = kOut && pz ? Elem<T>::to_f32(rz[j]) : 0.0f;
    }
    if (left > kTile) fetch(left - kTile);
    __syncthreads();
    if (wave_on) {
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const bool in = s + 4 * j < left;
        delta[j] = in ? softplus_f32(delta[j] + bias) : 0.0f;
        w[j] = in ? delta[j] * u[j] : 0.0f;
        sum_delta += delta[j];
      }
      if (kOut && mark) {
        if (on) {
#pragma unroll
          for (int i = 0; i < kNS; ++i)
            if (s * kNS + i < a.N) mark[i] = h[i];
        }
        mark += int64_t(a.D) * a.N;
      }
      const float* bc = sBC[buf] + s * kNS;
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float dt = from_owner<4>(delta[j], r), wt = from_owner<4>(w[j], r);
          float B[kNS], C[kNS];
          load_states<kNS>(bc + (4 * j + r) * 2 * kNP, B);
          if (kOut) load_states<kNS>(bc + (4 * j + r) * 2 * kNP + kNP, C);
          y[r] = 0.0f;
#pragma unroll
          for (int i = 0; i < kNS; ++i) {
            h[i] = fmaf(exp2_hw(dt * Ap[i]), h[i], wt * B[i]);
            if (kOut) y[r] = fmaf(C[i], h[i], y[r]);
          }
        }
        if constexpr (kOut) {
          float v = quad_scatter_sum(y[0], y[1], y[2], y[3], odd, high);
          v = fmaf(skip, u[j], v);
          if (pz) v *= silu_f32(z[j]);
          if (on && s + 4 * j < left) py[uint32_t(s + 4 * j) * uint32_t(a.D) + d] = Elem<T>::from_f32(v);
        }
      }
    }
    if (kOut) py += int64_t(kTile) * a.D;
  }
  if (!on) return;
  if constexpr (kOut) {
    if (a.ht && t_end == q.len) {
#pragma unroll
      for (int i = 0; i < kNS; ++i)
        if (s * kNS + i < a.N) a.ht[(q.n * a.D + d) * a.N + s * kNS + i] = h[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNS; ++i)
      if (s * kNS + i < a.N) a.seg_end[(p.unit * a.D + d) * a.N + s * kNS + i] = h[i];
    sum_delta = group_sum<4>(sum_delta);
    if (s == 0) a.seg_delta[p.unit * a.D + d] = sum_delta;
  }
}

// The segments of a sequence one after the other: each one's start state from the one before it,
// or with kBack, from the last to the first, what the adjoint sends to its end from behind it.
template <bool kBack>
__global__ __launch_bounds__(256) void k_scan_join(Args a) {
  const int64_t per = int64_t(a.D) * a.N, at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (at >= a.q.S * per) return;
  const Sequence q = sequence(a.q, at / per);
  const int64_t i = at % per, d = i / a.N;
  const int64_t count = (q.len + a.seglen - 1) / a.seglen, first = first_unit(a.q, q, a.seglen);
  const float Ap = -expf(a.A_log[i]) * kLog2e;
  const float* from = kBack ? a.dht : a.h0;
  float h = from ? from[at] : 0.0f;
  if (count == 0) {  // its one unit, without tokens, hands the state on
    a.seg_start[first * per + i] = h;
    return;
  }
  constexpr int kAhead = 8;
  for (int64_t j = 0; j < count; j += kAhead) {
    float end[kAhead], delta[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      const int64_t k = min(j + m, count - 1), unit = first + (kBack ? count - 1 - k : k);
      end[m] = a.seg_end[unit * per + i];
      delta[m] = a.seg_delta[unit * a.D + d];
    }
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      if (j + m >= count) break;
      const int64_t unit = first + (kBack ? count - 1 - (j + m) : j + m);
      a.seg_start[unit * per + i] = h;
      h = fmaf(exp2_hw(Ap * delta[m]), h, end[m]);
    }
  }
}

template <typename T, bool kOut>
int launch_states(const Args& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.units * a.G * a.cbg)), block(kThreads);
  switch (lane_states(a.N)) {
    case 1: hipLaunchKernelGGL((k_scan_tokens<T, 1, kOut>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_scan_tokens<T, 2, kOut>), grid, block, 0, st, a); break;
    case 4: hipLaunchKernelGGL((k_scan_tokens<T, 4, kOut>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((k_scan_tokens<T, 8, kOut>), grid, block, 0, st, a); break;
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_scan_tokens(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_states<float, true>(a, st) : launch_states<uint16_t, true>(a, st);
}

int launch_scan_segments(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_states<float, false>(a, st) : launch_states<uint16_t, false>(a, st);
}

int launch_scan_join(const Args& a, bool back, hipStream_t st) {
  const int64_t n = a.q.S * a.D * a.N;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256)), block(256);
  if (back) hipLaunchKernelGGL(k_scan_join<true>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(k_scan_join<false>, grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace sscan
}  // namespace ss2d
