// The token-order selective scan's adjoint: tiles from the last to the first, states recomputed
// from the one that was kept before each tile.
//   g_t = dy_t SiLU(z_t),   lambda_t = g_t C_t + a_{t+1} lambda_{t+1},   a_t = exp(A delta_t),
//   w_t = a_t lambda_t h_{t-1}:   dA = sum_t delta_t w_t,   ddelta_t = sum_n A w_t + u_t sum_n lambda_t B_t,
//   du_t = delta_t sum_n lambda_t B_t + Ds g_t,   dB_t = sum_d lambda_t delta_t u_t,   dC_t = sum_d g_t h_t.
// dB and dC are summed over a wave's 16 channels by the half-wave and row swaps, which halve the
// values with each sum, and two rotations of a row; over the waves in LDS; over the blocks of 64
// channels by a second kernel.  No atomics: every sum has a fixed order.
#include <algorithm>

#include "ss1d_scan.h"

namespace ss2d {
namespace sscan {
namespace {

// Sums of dB[i] and dC[i] over the 16 channels of a wave.  Lanes of the lower half get B's, of the
// upper half C's; with kNS >= 2 out[m] is state 2 m in the even rows of 16 lanes, 2 m + 1 in the odd.
template <int kNS>
__device__ __forceinline__ void channel_sums(float* dB, float* dC, float* out) {
#pragma unroll
  for (int i = 0; i < kNS; ++i) {
    swap_halves(dB[i], dC[i]);
    dB[i] += dC[i];
  }
  if constexpr (kNS == 1) {
    out[0] = add_across<16>(dB[0]);
  } else {
#pragma unroll
    for (int m = 0; m < kNS / 2; ++m) {
      swap_rows(dB[2 * m], dB[2 * m + 1]);
      out[m] = dB[2 * m] + dB[2 * m + 1];
    }
  }
#pragma unroll
  for (int m = 0; m < (kNS + 1) / 2; ++m) {
    out[m] += dpp_move<0x128>(out[m]);  // row_ror:8
    out[m] += dpp_move<0x124>(out[m]);  // row_ror:4
  }
}

// kAll: the gradients; else what a segment's start sends on from nothing behind it, and the
// segment's sum of delta.
template <typename T, int kNS, bool kAll>
__global__ __launch_bounds__(kThreads) void k_scan_adjoint(Args a) {
  constexpr int kTile = tile_of(kNS), kOwn = kTile / 4, kNP = 4 * kNS, kNY = (kNS + 1) / 2;
  constexpr int kBC = kTile * 2 * kNP, kPer = (kBC + kThreads - 1) / kThreads;
  __shared__ __align__(16) float sBC[2][kBC];
  __shared__ float sums[kAll ? 2 : 1][kAll ? 4 * kBC : 1];  // (wave, step, B then C)

  const Place p = place_of(a, blockIdx.x, gridDim.x);
  int64_t idx = 0;
  const Sequence q = a.seglen ? sequence_of(a.q, p.unit, a.seglen, &idx) : sequence(a.q, p.unit);
  const int64_t t_begin = idx * a.seglen;
  const bool empty = idx > 0 && t_begin >= q.len;
  const int64_t t_end = empty ? t_begin : (a.seglen ? min(q.len, t_begin + a.seglen) : q.len);

  const int tid = threadIdx.x, lane = tid & 63, s = lane & 3, wave = tid >> 6;
  const int Dg = a.D / a.G, c = p.c0 + (tid >> 2);
  const bool on = c < Dg, wave_on = p.c0 + wave * 16 < Dg;
  const int waves = min(4, (Dg - p.c0 + 15) / 16);
  const int d = p.g * Dg + (on ? c : Dg - 1);
  const bool odd = s & 1, high = s & 2;
  const int bank = (lane >> 2) & 3;

  float Ap[kNS], carry[kNS], dA[kNS];
  const float* behind = a.seglen ? (kAll ? a.seg_start : nullptr) : a.dht;
#pragma unroll
  for (int i = 0; i < kNS; ++i) {
    const int n = s * kNS + i;
    Ap[i] = n < a.N ? -expf(a.A_log[int64_t(d) * a.N + n]) * kLog2e : -1.0f;
    carry[i] = !empty && behind && n < a.N && on ? behind[(p.unit * a.D + d) * a.N + n] : 0.0f;
    dA[i] = 0.0f;
  }
  const float bias = a.bias[d], skip = a.Ds[d];
  float dD = 0.0f, dbias = 0.0f, sum_delta = 0.0f;

  const int64_t steps = t_end - t_begin, tiles = (steps + kTile - 1) / kTile;
  const int64_t row = q.begin + t_begin + (tiles - 1) * kTile;  // of the tile to load next
  const T* pu = static_cast<const T*>(a.u) + q.b * a.su.b + row * a.su.l;
  const T* pd = static_cast<const T*>(a.dt) + q.b * a.sd.b + row * a.sd.l;
  const T* pz = a.z ? static_cast<const T*>(a.z) + q.b * a.sz.b + row * a.sz.l : nullptr;
  const T* pg = static_cast<const T*>(a.dy) + (q.b * a.q.L + row) * a.D;
  const T* pB = static_cast<const T*>(a.Bs) + q.b * a.sb.b + row * a.sb.l + p.g * a.sbg;
  const T* pC = static_cast<const T*>(a.Cs) + q.b * a.sc.b + row * a.sc.l + p.g * a.scg;
  const uint32_t ul = a.su.l, dl_ = a.sd.l, zl = a.sz.l, gl = a.D;
  int64_t out_row = q.b * a.q.L + row;  // of the tile that is computed
  const float* mark = kAll ? a.marks + ((first_unit(a.q, q, kTile) + t_begin / kTile + tiles - 1) * a.D + d) * a.N
                                 + s * kNS : nullptr;

  T ru[kOwn], rd[kOwn], rz[kOwn], rg[kOwn], rbc[kPer];
  float rh[kNS];
  auto fetch = [&](int64_t left) {
    const int last = left >= kTile ? kTile - 1 : static_cast<int>(left) - 1;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const uint32_t r = min(s + 4 * j, last);
      if (kAll) ru[j] = pu[r * ul + d];
      rd[j] = pd[r * dl_ + d];
      if (pz) rz[j] = pz[r * zl + d];
      rg[j] = pg[r * gl + d];
    }
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const int e = tid + m * kThreads;
      const int n = e % kNP, which = e / kNP % 2, t = e / (2 * kNP);
      rbc[m] = T(0);
      if (e < kBC && n < a.N && t <= last) {
        if (which == 1) rbc[m] = pC[uint32_t(t) * uint32_t(a.sc.l) + n];
        else if (kAll) rbc[m] = pB[uint32_t(t) * uint32_t(a.sb.l) + n];
      }
    }
    if (kAll) {
#pragma unroll
      for (int i = 0; i < kNS; ++i) rh[i] = s * kNS + i < a.N ? mark[i] : 0.0f;
      mark -= int64_t(a.D) * a.N;
    }
    pu -= kTile * a.su.l;
    pd -= kTile * a.sd.l;
    if (pz) pz -= kTile * a.sz.l;
    pg -= int64_t(kTile) * a.D;
    pB -= kTile * a.sb.l;
    pC -= kTile * a.sc.l;
  };
  // the block's sums of a tile whose first row is `first`, of `left` tokens
  auto flush = [&](int buf, int64_t first, int64_t left) {
    const int64_t T_all = a.q.T;
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const int e = tid + m * kThreads;
      const int n = e % kNP, which = e / kNP % 2, t = e / (2 * kNP);
      if (e < kBC && n < a.N && t < left) {
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += sums[buf][w * kBC + e];
        a.bc_parts[((int64_t(p.cb) * T_all + first + t) * a.G + p.g) * 2 * a.N + which * a.N + n] = v;
      }
    }
  };

  if (tiles > 0) fetch(steps - (tiles - 1) * kTile);
  int buf = 0;
  for (int64_t k = tiles - 1; k >= 0; --k, buf ^= 1) {
    const int64_t left = steps - k * kTile;
#pragma unroll
    for (int m = 0; m < kPer; ++m)
      if (tid + m * kThreads < kBC) sBC[buf][tid + m * kThreads] = Elem<T>::to_f32(rbc[m]);
    float u[kOwn], raw[kOwn], z[kOwn], g[kOwn], h0[kNS];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      u[j] = kAll ? Elem<T>::to_f32(ru[j]) : 0.0f;
      raw[j] = Elem<T>::to_f32(rd[j]);
      z[j] = pz ? Elem<T>::to_f32(rz[j]) : 0.0f;
      g[j] = Elem<T>::to_f32(rg[j]);
    }
#pragma unroll
    for (int i = 0; i < kNS; ++i) h0[i] = kAll ? rh[i] : 0.0f;
    if (k > 0) fetch(kTile);
    __syncthreads();
    if (kAll && k < tiles - 1) flush(buf ^ 1, out_row + kTile, left - kTile);
    if (wave_on) {
      float delta[kOwn], w[kOwn], gy[kOwn], sg[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        const bool in = on && s + 4 * j < left;
        raw[j] += bias;
        delta[j] = in ? softplus_f32(raw[j]) : 0.0f;
        w[j] = in ? delta[j] * u[j] : 0.0f;
        gy[j] = in ? g[j] : 0.0f;
        sg[j] = 0.0f;
        if (pz) {
          sg[j] = __builtin_amdgcn_rcpf(1.0f + exp2_hw(-z[j] * kLog2e));
          gy[j] = in ? g[j] * (sg[j] == 0.0f ? -0.0f : z[j] * sg[j]) : 0.0f;
        }
        sum_delta += delta[j];
      }
      const float* bc = sBC[buf] + s * kNS;
      if constexpr (!kAll) {
#pragma unroll
        for (int t = kTile - 1; t >= 0; --t) {
          const float dt = from_owner<4>(delta[t / 4], t % 4), gt = from_owner<4>(gy[t / 4], t % 4);
#pragma unroll
          for (int i = 0; i < kNS; ++i)
            carry[i] = exp2_hw(dt * Ap[i]) * fmaf(gt, bc[t * 2 * kNP + kNP + i], carry[i]);
        }
      } else {
        float as[kTile][kNS], hs[kTile][kNS];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          float y[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = 4 * j + r;
            const float dt = from_owner<4>(delta[j], r), wt = from_owner<4>(w[j], r);
            y[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < kNS; ++i) {
              as[t][i] = exp2_hw(dt * Ap[i]);
              hs[t][i] = fmaf(as[t][i], t ? hs[t ? t - 1 : 0][i] : h0[i], wt * bc[t * 2 * kNP + i]);
              if (pz) y[r] = fmaf(bc[t * 2 * kNP + kNP + i], hs[t][i], y[r]);
            }
          }
          if (pz) {
            const float v = fmaf(skip, u[j], quad_scatter_sum(y[0], y[1], y[2], y[3], odd, high));
            // SiLU'(z) = sigmoid(z) (1 + z (1 - sigmoid(z)))
            const float slope = sg[j] == 0.0f ? 0.0f : (sg[j] == 1.0f ? 1.0f : sg[j] * fmaf(z[j], 1.0f - sg[j], 1.0f));
            if (on && s + 4 * j < left)
              static_cast<T*>(a.dz)[out_row * a.D + uint32_t(s + 4 * j) * gl + d] = Elem<T>::from_f32(g[j] * v * slope);
          }
        }
#pragma unroll
        for (int j = kOwn - 1; j >= 0; --j) {
          float P[4], Q[4], acc[kNY];
#pragma unroll
          for (int r = 3; r >= 0; --r) {
            const int t = 4 * j + r;
            const float dt = from_owner<4>(delta[j], r), wt = from_owner<4>(w[j], r), gt = from_owner<4>(gy[j], r);
            float dB[kNS], dC[kNS], out[kNY];
            P[r] = Q[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < kNS; ++i) {
              const float lam = fmaf(gt, bc[t * 2 * kNP + kNP + i], carry[i]);
              dB[i] = lam * wt;
              dC[i] = gt * hs[t][i];
              Q[r] = fmaf(lam, bc[t * 2 * kNP + i], Q[r]);
              carry[i] = as[t][i] * lam;
              const float v = carry[i] * (t ? hs[t ? t - 1 : 0][i] : h0[i]);
              dA[i] = fmaf(dt, v, dA[i]);
              P[r] = fmaf(v, Ap[i], P[r]);
            }
            channel_sums<kNS>(dB, dC, out);
#pragma unroll
            for (int m = 0; m < kNY; ++m) acc[m] = bank == r ? out[m] : (r == 3 ? 0.0f : acc[m]);
          }
          // a lane's sums are those of step 4 j + bank
          float* to = sums[buf] + wave * kBC + (4 * j + bank) * 2 * kNP + (lane >> 5) * kNP + s * kNS;
          if constexpr (kNS == 1) {
            to[0] = acc[0];
          } else {
#pragma unroll
            for (int m = 0; m < kNY; ++m) to[2 * m + ((lane >> 4) & 1)] = acc[m];
          }
          const float ps = quad_scatter_sum(P[0], P[1], P[2], P[3], odd, high) * kLn2;
          const float qs = quad_scatter_sum(Q[0], Q[1], Q[2], Q[3], odd, high);
          const bool in = on && s + 4 * j < left;
          const float draw = fmaf(u[j], qs, ps) * __builtin_amdgcn_rcpf(1.0f + exp2_hw(-raw[j] * kLog2e));
          const float du = fmaf(delta[j], qs, skip * gy[j]);
          if (in) {
            const int64_t at = out_row * a.D + uint32_t(s + 4 * j) * gl + d;
            static_cast<T*>(a.du)[at] = Elem<T>::from_f32(du);
            static_cast<T*>(a.ddt)[at] = Elem<T>::from_f32(draw);
            dD = fmaf(gy[j], u[j], dD);
            dbias += draw;
          }
        }
      }
    }
    out_row -= kTile;
  }
  if constexpr (kAll) {
    if (tiles > 0) {
      __syncthreads();
      flush(buf ^ 1, out_row + kTile, min(steps, int64_t(kTile)));
    }
    dD = group_sum<4>(dD);
    dbias = group_sum<4>(dbias);
  }
  sum_delta = group_sum<4>(sum_delta);
  if (!on) return;
  if constexpr (kAll) {
    float* parts = a.par_parts + (p.unit * a.D + d) * (a.N + 2);
#pragma unroll
    for (int i = 0; i < kNS; ++i) {
      const int n = s * kNS + i;
      if (n >= a.N) continue;
      parts[n] = dA[i] * (Ap[i] * kLn2);
      if (a.dh0 && !empty && idx == 0) a.dh0[(q.n * a.D + d) * a.N + n] = carry[i];
    }
    if (s == 0) {
      parts[a.N] = dD;
      parts[a.N + 1] = dbias;
    }
  } else if (!empty) {
#pragma unroll
    for (int i = 0; i < kNS; ++i)
      if (s * kNS + i < a.N) a.seg_end[(p.unit * a.D + d) * a.N + s * kNS + i] = carry[i];
    if (s == 0) a.seg_delta[p.unit * a.D + d] = sum_delta;
  }
}

// dB and dC: the sums over the channel blocks, for units of 64 tokens of one sequence.
constexpr int kSumTokens = 64;
template <typename T>
__global__ __launch_bounds__(256) void k_scan_sum_bc(Args a) {
  int64_t idx;
  const Sequence q = sequence_of(a.q, blockIdx.x, kSumTokens, &idx);
  const int64_t t0 = idx * kSumTokens;
  if (t0 >= q.len) return;
  const int64_t row = q.b * a.q.L + q.begin + t0, width = int64_t(a.G) * 2 * a.N;
  const int64_t count = min(q.len - t0, int64_t(kSumTokens)) * width, stride = a.q.T * width;
  const float* parts = a.bc_parts + row * width;
  for (int64_t e = threadIdx.x; e < count; e += 256) {
    float v = 0.0f;
    for (int b = 0; b < a.cbg; ++b) v += parts[b * stride + e];
    const int64_t tg = e / (2 * a.N);
    const int n = static_cast<int>(e % (2 * a.N));
    T* to = static_cast<T*>(n < a.N ? a.dB : a.dC);
    to[(row * a.G + tg) * a.N + (n < a.N ? n : n - a.N)] = Elem<T>::from_f32(v);
  }
}

// dA_log, dDs and ddt_bias: the sums over the units, 64 columns and 16 groups of units per block.
__global__ __launch_bounds__(1024) void k_scan_sum_params(Args a) {
  __shared__ float buffer[16][64];
  const int64_t width = int64_t(a.D) * (a.N + 2), c = int64_t(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float x[4] = {};
  if (c < width) {
    const float* p = a.par_parts + c;
    int64_t b = w;
    for (; b + 48 < a.units; b += 64)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += p[(b + 16 * i) * width];
    for (; b < a.units; b += 16) x[0] += p[b * width];
  }
  buffer[w][threadIdx.x & 63] = (x[0] + x[1]) + (x[2] + x[3]);
  __syncthreads();
  if (w != 0 || c >= width) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += buffer[i][threadIdx.x];
  const int64_t d = c / (a.N + 2);
  const int n = static_cast<int>(c % (a.N + 2));
  if (n < a.N) a.dA[d * a.N + n] = v;
  else if (n == a.N) a.dD[d] = v;
  else a.dbias[d] = v;
}

template <typename T, bool kAll>
int launch_states(const Args& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.units * a.G * a.cbg)), block(kThreads);
  switch (lane_states(a.N)) {
    case 1: hipLaunchKernelGGL((k_scan_adjoint<T, 1, kAll>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((k_scan_adjoint<T, 2, kAll>), grid, block, 0, st, a); break;
    case 4: hipLaunchKernelGGL((k_scan_adjoint<T, 4, kAll>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((k_scan_adjoint<T, 8, kAll>), grid, block, 0, st, a); break;
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_scan_adjoint(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_states<float, true>(a, st) : launch_states<uint16_t, true>(a, st);
}

int launch_scan_adjoint_segments(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_states<float, false>(a, st) : launch_states<uint16_t, false>(a, st);
}

int launch_scan_sums(const Args& a, int dtype, hipStream_t st) {
  const int64_t units = unit_count(a.q.L, a.q.S, a.q.T, a.q.cu != nullptr, kSumTokens);
  if (units > 0 && a.q.S > 0) {
    const dim3 grid(static_cast<unsigned>(units)), block(256);
    if (dtype == 0) hipLaunchKernelGGL(k_scan_sum_bc<float>, grid, block, 0, st, a);
    else hipLaunchKernelGGL(k_scan_sum_bc<uint16_t>, grid, block, 0, st, a);
  }
  const int64_t width = int64_t(a.D) * (a.N + 2);
  hipLaunchKernelGGL(k_scan_sum_params, dim3(static_cast<unsigned>((width + 63) / 64)), dim3(1024), 0, st, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace sscan
}  // namespace ss2d
