// The token-order selective scan, forward: whole sequences or segments of them.
//
// A state takes an exponential (two slots of the vector pipe or more), a product for delta A, and three
// multiply-adds per token; a channel softplus, its gate, and the sum over its states.  That, not HBM, is
// what bounds it.  Four lanes share a channel: each computes softplus, delta u and the gate of every
// fourth step, so that these cost a quarter, and hands them to the others.  One lane per channel with B and C as scalar
// operands took 971 us for 598 (16 x 2048 tokens of 4096 channels): nothing hid the scalar loads.
// The chain of a sequence leaves few waves; a segmented call first computes every segment's end
// from zero (no C, no outputs), joins them, and runs again from the joined states.
// Measured, bf16 with gate, 16 states: a prompt of 4096 tokens, 4096 channels, in 16 segments 62 + 5 +
// 89 us (the vector pipes 77% busy; HBM would take 27); 8 x 2048 tokens of 2048 channels, whole, saving
// states, 240 (55% busy, one wave per SIMD); fp32, 2 x 65,536 tokens of 192 channels, 88 + 11 + 115.
#include <algorithm>
#include <type_traits>

#include "ss1d_scan.h"

namespace ss2d {
namespace sscan {
namespace {

// kS lanes share a channel (4: a quad, 16: a row of 16 lanes), each with kNS of its states and every
// kS-th step of a tile.
template <int kS, int kOwner> __device__ __forceinline__ float from_step(float v) {
  if constexpr (kS == 4) return from_owner<4>(v, kOwner);
  else return dpp_move<0x150 + kOwner>(v);  // row_newbcast
}

// Sums each of kS values over the lanes of a channel: lane s gets the sum of v[s].
template <int kS> __device__ __forceinline__ float scatter_sum(const float* v, int s) {
  const bool b0 = s & 1, b1 = s & 2;
  float a[kS / 4];
  if constexpr (kS == 4) return quad_scatter_sum(v[0], v[1], v[2], v[3], b0, b1);
#pragma unroll
  for (int i = 0; i < kS / 4; ++i) a[i] = quad_scatter_sum(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], b0, b1);
  if constexpr (kS == 16) {  // a[i] belongs to quad i: lanes 8 apart first, then 4
    const bool b2 = s & 4, b3 = s & 8;
    float x = (b3 ? a[2] : a[0]) + from_lane<8>(b3 ? a[0] : a[2]);
    float y = (b3 ? a[3] : a[1]) + from_lane<8>(b3 ? a[1] : a[3]);
    a[0] = (b2 ? y : x) + from_lane<4>(b2 ? x : y);
  }
  return a[0];
}

// kOut: outputs, end states and marks; else a segment's end state from a zero start and its sum
// of delta.  B and C of a tile lie in LDS (read by all channels of the block), a lane's steps of u, dt_raw
// and z are loaded a tile ahead.
template <typename T, int kS, int kNS, bool kOut, bool kGate>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 4)))
void k_scan_tokens(Args a) {
  constexpr int kMark = tile_of(kNS), kTile = kS == 4 ? kMark : 64, kOwn = kTile / kS, kNP = kS * kNS;
  constexpr int kWaveCh = 64 / kS, kCh = kThreads / kS;
  constexpr int kBC = kTile * 2 * kNP, kPer = Operands<T, kTile, kNP>::kPer;
  // B and C of a tile: rows of a step (B, then C) for a quad; for 16 lanes rows of a state, padded
  constexpr int kRow = kS == 4 ? 2 * kNP : kTile + 4, kSize = kS == 4 ? kBC : 2 * kNP * kRow;
  __shared__ __align__(16) float sBC[2][kSize];

  const Place p = place_of(a, kCh, blockIdx.x, gridDim.x);
  int64_t idx = 0;
  const Sequence q = uniform(a.seglen ? sequence_of(a.q, p.unit, a.seglen, &idx) : sequence(a.q, p.unit));
  idx = uniform(idx);
  const int64_t t_begin = idx * a.seglen;
  if (idx > 0 && t_begin >= q.len) return;  // an empty unit
  // nothing follows a sequence's last segment, so that nobody needs its end state
  if (!kOut && t_begin + a.seglen >= q.len) return;
  const int64_t t_end = a.seglen ? min(q.len, t_begin + a.seglen) : q.len;

  const int tid = threadIdx.x, lane = tid & 63, s = lane % kS;
  const int Dg = a.D / a.G, c = p.c0 + tid / kS;
  const bool on = c < Dg, wave_on = p.c0 + __builtin_amdgcn_readfirstlane(tid >> 6) * kWaveCh < Dg;
  const int d = p.g * Dg + (on ? c : Dg - 1);

  float Ap[kNS], h[kNS];
#pragma unroll
  for (int i = 0; i < kNS; ++i) {
    const int n = s * kNS + i;
    // states past N decay to nothing; their B and C are zero
    Ap[i] = n < a.N ? decay_rate(a.A_log[int64_t(d) * a.N + n]) : -1.0f;
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
  const T* pz = kGate ? static_cast<const T*>(a.z) + q.b * a.sz.b + row * a.sz.l : nullptr;
  T* py = kOut ? static_cast<T*>(a.y) + (q.b * a.q.L + row) * a.D : nullptr;

  T ru[kOwn] = {}, rd[kOwn] = {}, rz[kOwn] = {};
  Operands<T, kTile, kNP> bc_in;
  bc_in.start(a, q.b, row, p.g, kOut, true);
  // the lane's element of a tile's first kS rows
  const uint32_t ou = s * uint32_t(a.su.l) + d, od = s * uint32_t(a.sd.l) + d, oz = s * uint32_t(a.sz.l) + d,
                 oy = s * uint32_t(a.D) + d;
  auto fetch = [&](int rows) {
    const uint32_t cu = opaque(ou), cd = opaque(od), cz = opaque(oz);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      if (s + kS * j < rows) {
        ru[j] = element(pu + j * kS * a.su.l, cu);
        rd[j] = element(pd + j * kS * a.sd.l, cd);
        if (kGate) rz[j] = element(pz + j * kS * a.sz.l, cz);
      }
    }
    bc_in.load(rows, kTile);
    pu += kTile * a.su.l;
    pd += kTile * a.sd.l;
    if (kGate) pz += kTile * a.sz.l;
  };

  float* mark = nullptr;
  if (kOut && kS == 4 && a.marks)
    mark = a.marks + (first_unit(a.q, q, kMark) + t_begin / kMark) * a.D * a.N;
  const uint32_t om = uint32_t(d) * a.N + s * kNS;
  const bool whole_mark = kNS == 4 && a.N == 16;
  float sum_delta = 0.0f;
  int64_t left = t_end - t_begin;
  if (left > 0) fetch(static_cast<int>(min(left, int64_t(kTile))));
  for (int buf = 0; left > 0; left -= kTile, buf ^= 1) {
    const int rows = static_cast<int>(min(left, int64_t(kTile)));
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const int e = tid + m * kThreads;
      if (kBC % kThreads == 0 || e < kBC) {
        if constexpr (kS == 4) sBC[buf][e] = Elem<T>::to_f32(bc_in.raw[m]);
        else sBC[buf][e % (2 * kNP) * kRow + e / (2 * kNP)] = Elem<T>::to_f32(bc_in.raw[m]);
      }
    }
    float u[kOwn], delta[kOwn], z[kOwn], w[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      u[j] = Elem<T>::to_f32(ru[j]);
      delta[j] = Elem<T>::to_f32(rd[j]);
      z[j] = kGate ? Elem<T>::to_f32(rz[j]) : 0.0f;
    }
    fetch(static_cast<int>(max(int64_t(0), min(left - kTile, int64_t(kTile)))));
    __syncthreads();
    if (wave_on) {
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        delta[j] = softplus_f32(delta[j] + bias);
        w[j] = delta[j] * u[j];
      }
      if (rows < kTile) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const bool in = s + kS * j < rows;
          delta[j] = in ? delta[j] : 0.0f;
          w[j] = in ? w[j] : 0.0f;
        }
      }
      if (!kOut) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) sum_delta += delta[j];
      }
      const float* bc = sBC[buf] + (kS == 4 ? s * kNS : s * kNS * kRow);
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        if (kOut && kS == 4 && kS * j % kMark == 0 && mark && kS * j < rows) {
          if (on && whole_mark) {
            *reinterpret_cast<float4*>(&element(mark, opaque(om))) = make_float4(h[0], h[1 % kNS], h[2 % kNS], h[3 % kNS]);
          } else if (on) {
  #pragma unroll
            for (int i = 0; i < kNS; ++i)
              if (s * kNS + i < a.N) element(mark, opaque(om) + i) = h[i];
          }
          mark += int64_t(a.D) * a.N;
        }
        float B[kS][kNS], C[kS][kNS], as[kS][kNS], y[kS];
        if constexpr (kS == 4) {
#pragma unroll
          for (int r = 0; r < kS; ++r) {
            load_states<kNS>(bc + (kS * j + r) * kRow, B[r]);
            if (kOut) load_states<kNS>(bc + (kS * j + r) * kRow + kNP, C[r]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kNS; ++i)
#pragma unroll
            for (int r = 0; r < kS; r += 4) {
              const float4 vb = *reinterpret_cast<const float4*>(bc + i * kRow + kS * j + r);
              B[r][i] = vb.x, B[r + 1][i] = vb.y, B[r + 2][i] = vb.z, B[r + 3][i] = vb.w;
              if (kOut) {
                const float4 vc = *reinterpret_cast<const float4*>(bc + (kNP + i) * kRow + kS * j + r);
                C[r][i] = vc.x, C[r + 1][i] = vc.y, C[r + 2][i] = vc.z, C[r + 3][i] = vc.w;
              }
            }
        }
        unrolled<0, kS>([&](auto r) {
          const float dt = from_step<kS, r>(delta[j]);
#pragma unroll
          for (int i = 0; i < kNS; ++i) as[r][i] = exp2_hw(dt * Ap[i]);
        });
        unrolled<0, kS>([&](auto r) {
          const float wt = from_step<kS, r>(w[j]);
          y[r] = 0.0f;
#pragma unroll
          for (int i = 0; i < kNS; ++i) {
            h[i] = fmaf(as[r][i], h[i], wt * B[r][i]);
            if (kOut) y[r] = i ? fmaf(C[r][i], h[i], y[r]) : C[r][i] * h[i];
          }
        });
        if constexpr (kOut) {
          float v = fmaf(skip, u[j], scatter_sum<kS>(y, s));
          if (kGate) v *= silu_f32(z[j]);
          if (on && s + kS * j < rows) element(py + j * kS * int64_t(a.D), opaque(oy)) = Elem<T>::from_f32(v);
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
// A thread carries one state.  With kWaves > 1 the block's waves take the same 64 states over parts of
// the segments: each folds its own from zero, then starts from the fold of those before it, for the
// latency of the loads bounds this kernel.  Measured, one wave and 16: 171 segments (2 x 65,536 tokens of
// 192 channels, 16 states) 21.7 and 11 us; 87 segments of 25 packed sequences of 1000 channels 7.5 and
// 57; 16 segments of one prompt of 4096 channels 5.2 and 24.
template <bool kBack, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void k_scan_join(Args a) {
  constexpr int kAhead = kWaves > 1 ? 16 : 8;
  __shared__ float ends[kWaves][64], deltas[kWaves][64];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t per = int64_t(a.D) * a.N, at = int64_t(blockIdx.x) * 64 + lane;
  const bool valid = at < a.q.S * per;
  const Sequence q = sequence(a.q, valid ? at / per : 0);
  const int64_t i = valid ? at % per : 0, d = i / a.N;
  const int64_t count = (q.len + a.seglen - 1) / a.seglen, first = first_unit(a.q, q, a.seglen);
  const int64_t part = (count + kWaves - 1) / kWaves;
  const int64_t k0 = part * wave, k1 = valid ? min(count, k0 + part) : 0;
  const float Ap = decay_rate(a.A_log[i]);
  const float* from = kBack ? a.dht : a.h0;
  float h = from && valid ? from[at] : 0.0f;
  // segments k0 to k1 from the state h
  auto walk = [&](float h, bool write, float& sum) {
    for (int64_t j = k0; j < k1; j += kAhead) {
      float end[kAhead], delta[kAhead];
#pragma unroll
      for (int m = 0; m < kAhead; ++m) {
        // (a load behind a condition of its own would wait for the one before it)
        const int64_t k = min(j + m, k1 - 1), unit = first + (kBack ? count - 1 - k : k);
        end[m] = a.seg_end[unit * per + i];
        delta[m] = a.seg_delta[unit * a.D + d];
      }
#pragma unroll
      for (int m = 0; m < kAhead; ++m) {
        if (j + m >= k1) break;
        const int64_t unit = first + (kBack ? count - 1 - (j + m) : j + m);
        if (write) a.seg_start[unit * per + i] = h;
        if (j + m == count - 1) break;  // of the last segment neither is kept
        h = fmaf(exp2_hw(Ap * delta[m]), h, end[m]);
        sum += delta[m];
      }
    }
    return h;
  };
  float sum = 0.0f;
  if (kWaves > 1) {
    ends[wave][lane] = walk(0.0f, false, sum);
    deltas[wave][lane] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) h = fmaf(exp2_hw(Ap * deltas[w][lane]), h, ends[w][lane]);
  }
  walk(h, true, sum);
  if (valid && count == 0 && wave == 0) a.seg_start[first * per + i] = h;  // a unit without tokens hands it on
}

template <typename T, int kS, int kNS, bool kOut>
int launch_gate(const Args& a, hipStream_t st) {
  const int per = (a.D / a.G + kThreads / kS - 1) / (kThreads / kS);
  const dim3 grid(static_cast<unsigned>(a.units * a.G * per)), block(kThreads);
  if (kOut && a.z) hipLaunchKernelGGL((k_scan_tokens<T, kS, kNS, kOut, kOut>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_scan_tokens<T, kS, kNS, kOut, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T, bool kOut>
int launch_states(const Args& a, hipStream_t st) {
  if (kOut && a.lanes == 16)
    return a.N <= 16 ? launch_gate<T, 16, 1, true>(a, st) : launch_gate<T, 16, 2, true>(a, st);
  switch (lane_states(a.N)) {
    case 1: return launch_gate<T, 4, 1, kOut>(a, st);
    case 2: return launch_gate<T, 4, 2, kOut>(a, st);
    case 4: return launch_gate<T, 4, 4, kOut>(a, st);
    default: return launch_gate<T, 4, 8, kOut>(a, st);
  }
}

}  // namespace

int launch_scan_tokens(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_states<float, true>(a, st) : launch_states<uint16_t, true>(a, st);
}

int launch_scan_segments(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_states<float, false>(a, st) : launch_states<uint16_t, false>(a, st);
}

int launch_scan_join(const Args& a, bool back, hipStream_t st) {
  constexpr int kWaves = 16;
  const int64_t blocks = (a.q.S * a.D * a.N + 63) / 64;
  // more segments a sequence than one wave has in flight, and few enough blocks for one launch
  const bool many = a.units > a.q.S * 16 && blocks < (1 << 21);
  const dim3 grid(static_cast<unsigned>(blocks)), block(many ? 64 * kWaves : 64);
  if (back && many) hipLaunchKernelGGL((k_scan_join<true, kWaves>), grid, block, 0, st, a);
  else if (back) hipLaunchKernelGGL((k_scan_join<true, 1>), grid, block, 0, st, a);
  else if (many) hipLaunchKernelGGL((k_scan_join<false, kWaves>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_scan_join<false, 1>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace sscan
}  // namespace ss2d
