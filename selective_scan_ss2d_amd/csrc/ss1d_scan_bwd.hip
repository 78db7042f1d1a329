// The token-order selective scan's adjoint: tiles from the last to the first, states recomputed
// from the one that was kept before each tile.
//   g_t = dy_t SiLU(z_t),   lambda_t = g_t C_t + a_{t+1} lambda_{t+1},   a_t = exp(A delta_t),
//   w_t = a_t lambda_t h_{t-1}:   dA = sum_t delta_t w_t,   ddelta_t = sum_n A w_t + u_t sum_n lambda_t B_t,
//   du_t = delta_t sum_n lambda_t B_t + Ds g_t,   dB_t = sum_d lambda_t delta_t u_t,   dC_t = sum_d g_t h_t.
// dB and dC are summed over a wave's 16 channels by the half-wave and row swaps, which halve the
// values with each sum, and two rotations of a row; over the waves in LDS; over the blocks of 64
// channels by a second kernel.  No atomics: every sum has a fixed order.
// It is bound by the vector pipes: 99.5 instructions per step of 16 channels of 16 states, of which the
// states again take a quarter and the sums over channels a fifth; at 254 registers two waves per SIMD
// keep them 77% busy.  8 x 2048 tokens of 2048 channels, bf16 with gate, in two segments per sequence:
// 100 us (what segments send on) + 5 (join) + 502 + 13 (dB, dC) + 5 (vectors); whole, at one wave per
// SIMD, 758 in all.  Tiles of 32 steps or of more registers spill, and a reload waits for the
// loads ahead of it.
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
template <typename T, int kNS, bool kAll, bool kGate>
__global__ __launch_bounds__(kThreads, 2) void k_scan_adjoint(Args a) {
  constexpr int kTile = tile_of(kNS), kOwn = kTile / 4, kNP = 4 * kNS, kNY = (kNS + 1) / 2;
  constexpr int kBC = kTile * 2 * kNP, kPer = Operands<T, kTile, kNP>::kPer;
  __shared__ __align__(16) float sBC[2][kBC];
  __shared__ float sums[kAll ? 2 : 1][kAll ? 4 * kBC : 1];  // (wave, step, B then C)

  const Place p = place_of(a, kBlockCh, blockIdx.x, gridDim.x);
  int64_t idx = 0;
  const Sequence q = uniform(a.seglen ? sequence_of(a.q, p.unit, a.seglen, &idx) : sequence(a.q, p.unit));
  idx = uniform(idx);
  const int64_t t_begin = idx * a.seglen;
  const bool empty = idx > 0 && t_begin >= q.len;
  if (!kAll && idx == 0) return;  // nothing before a sequence's first segment needs its carry
  const int64_t t_end = empty ? t_begin : (a.seglen ? min(q.len, t_begin + a.seglen) : q.len);

  const int tid = threadIdx.x, lane = tid & 63, s = lane & 3, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    Ap[i] = n < a.N ? decay_rate(a.A_log[int64_t(d) * a.N + n]) : -1.0f;
    carry[i] = !empty && behind && n < a.N && on ? behind[(p.unit * a.D + d) * a.N + n] : 0.0f;
    dA[i] = 0.0f;
  }
  const float bias = a.bias[d], skip = a.Ds[d];
  float dD = 0.0f, dbias = 0.0f, sum_delta = 0.0f;

  const int64_t steps = t_end - t_begin, tiles = (steps + kTile - 1) / kTile;
  const int64_t row = q.begin + t_begin + (tiles - 1) * kTile;  // of the tile to load next
  const T* pu = static_cast<const T*>(a.u) + q.b * a.su.b + row * a.su.l;
  const T* pd = static_cast<const T*>(a.dt) + q.b * a.sd.b + row * a.sd.l;
  const T* pz = kGate ? static_cast<const T*>(a.z) + q.b * a.sz.b + row * a.sz.l : nullptr;
  const T* pg = static_cast<const T*>(a.dy) + (q.b * a.q.L + row) * a.D;
    const int64_t out_row = q.b * a.q.L + row;  // of the last tile
  T* qu = kAll ? static_cast<T*>(a.du) + out_row * a.D : nullptr;
  T* qd = kAll ? static_cast<T*>(a.ddt) + out_row * a.D : nullptr;
  T* qz = kAll && kGate ? static_cast<T*>(a.dz) + out_row * a.D : nullptr;
  const float* mark = kAll ? a.marks + (first_unit(a.q, q, kTile) + t_begin / kTile + tiles - 1) * a.D * a.N : nullptr;
  const bool whole_mark = kNS >= 4 && a.N == 4 * kNS;
  const uint32_t om = uint32_t(d) * a.N + s * kNS;

  T ru[kOwn] = {}, rd[kOwn] = {}, rz[kOwn] = {}, rg[kOwn] = {};
  float rh[kNS] = {};
  Operands<T, kTile, kNP> bc_in;
  bc_in.start(a, q.b, row, p.g, kAll, false);
  // the lane's element of a tile's first four rows
  const uint32_t ou = s * uint32_t(a.su.l) + d, od = s * uint32_t(a.sd.l) + d, oz = s * uint32_t(a.sz.l) + d,
                 og = s * uint32_t(a.D) + d;
  // loads a tile of `rows` steps (none: 0) and goes on to the one before it
  auto fetch = [&](int rows) {
    const uint32_t cu = opaque(ou), cd = opaque(od), cz = opaque(oz), cg = opaque(og), cm = opaque(om);
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      if (s + 4 * j < rows) {
        if (kAll) ru[j] = element(pu + j * 4 * a.su.l, cu);
        rd[j] = element(pd + j * 4 * a.sd.l, cd);
        if (kGate) rz[j] = element(pz + j * 4 * a.sz.l, cz);
        rg[j] = element(pg + j * 4 * int64_t(a.D), cg);
      }
    }
    bc_in.load(rows, -kTile);
    if (kAll && rows > 0) {
      if (whole_mark) {
        load_states<kNS>(&element(mark, cm), rh);
      } else {
#pragma unroll
        for (int i = 0; i < kNS; ++i) rh[i] = s * kNS + i < a.N ? element(mark, cm + i) : 0.0f;
      }
    }
    if (kAll) {
      mark -= int64_t(a.D) * a.N;
      pu -= kTile * a.su.l;
    }
    pd -= kTile * a.sd.l;
    if (kGate) pz -= kTile * a.sz.l;
    pg -= kTile * int64_t(a.D);
  };
  // the block's sums of a tile of `left` tokens, from the last tile on
  float* parts = kAll ? a.bc_parts + ((int64_t(p.cb) * a.q.T + out_row) * a.G + p.g) * 2 * a.N : nullptr;
  auto flush = [&](int buf, int left) {
#pragma unroll
    for (int m = 0; m < kPer; ++m) {
      const int e = tid + m * kThreads, n = tid % kNP, t = e / (2 * kNP);
      if (n < a.N && t < left) {
        const float* from = sums[buf] + e;
        float v = from[0];
        for (int w = 1; w < waves; ++w) v += from[w * kBC];
        element(parts, opaque(uint32_t(t) * uint32_t(a.G * 2 * a.N) + tid / kNP % 2 * a.N + n)) = v;
      }
    }
    parts -= int64_t(kTile) * a.G * 2 * a.N;
  };

  if (tiles > 0) fetch(static_cast<int>(steps - (tiles - 1) * kTile));
  int buf = 0;
  for (int64_t k = tiles - 1; k >= 0; --k, buf ^= 1) {
    const int left = static_cast<int>(min(steps - k * kTile, int64_t(kTile)));
#pragma unroll
    for (int m = 0; m < kPer; ++m)
      if (tid + m * kThreads < kBC) sBC[buf][tid + m * kThreads] = Elem<T>::to_f32(bc_in.raw[m]);
    float u[kOwn], raw[kOwn], z[kOwn], g[kOwn], h0[kNS];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      u[j] = kAll ? Elem<T>::to_f32(ru[j]) : 0.0f;
      raw[j] = Elem<T>::to_f32(rd[j]);
      z[j] = kGate ? Elem<T>::to_f32(rz[j]) : 0.0f;
      g[j] = Elem<T>::to_f32(rg[j]);
    }
#pragma unroll
    for (int i = 0; i < kNS; ++i) h0[i] = kAll ? rh[i] : 0.0f;
    if (!kAll) fetch(k > 0 ? kTile : 0);
    __syncthreads();
    if (kAll && k < tiles - 1) flush(buf ^ 1, static_cast<int>(min(steps - (k + 1) * kTile, int64_t(kTile))));
    if (kAll && !wave_on) fetch(k > 0 ? kTile : 0);  // its share of B and C
    if (wave_on) {
      float delta[kOwn], w[kOwn], gy[kOwn], sg[kOwn];
#pragma unroll
      for (int j = 0; j < kOwn; ++j) {
        raw[j] += bias;
        delta[j] = softplus_f32(raw[j]);
        w[j] = delta[j] * u[j];
        gy[j] = g[j];
        sg[j] = 0.0f;
        if (kGate) {
          sg[j] = __builtin_amdgcn_rcpf(1.0f + exp2_hw(-z[j] * kLog2e));
          gy[j] *= sg[j] == 0.0f ? -0.0f : z[j] * sg[j];
        }
      }
      if (!on || left < kTile) {  // lanes and steps that are not there change nothing
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          const bool in = on && s + 4 * j < left;
          delta[j] = in ? delta[j] : 0.0f;
          w[j] = in ? w[j] : 0.0f;
          gy[j] = in ? gy[j] : 0.0f;
        }
      }
      const float* bc = sBC[buf] + s * kNS;
      if constexpr (!kAll) {
#pragma unroll
        for (int j = kOwn - 1; j >= 0; --j) {
          float C[4][kNS], as[4][kNS];
#pragma unroll
          for (int r = 0; r < 4; ++r) load_states<kNS>(bc + (4 * j + r) * 2 * kNP + kNP, C[r]);
          unrolled<0, 4>([&](auto r) {
            const float dt = from_owner<4>(delta[j], r);
#pragma unroll
            for (int i = 0; i < kNS; ++i) as[r][i] = exp2_hw(dt * Ap[i]);
          });
          unrolled<0, 4>([&](auto k) {
            constexpr int r = 3 - k;
            const float gt = from_owner<4>(gy[j], r);
#pragma unroll
            for (int i = 0; i < kNS; ++i) carry[i] = as[r][i] * fmaf(gt, C[r][i], carry[i]);
          });
          sum_delta += delta[j];
        }
      } else {
        float as[kTile][kNS], hs[kTile + 1][kNS];
#pragma unroll
        for (int i = 0; i < kNS; ++i) hs[0][i] = h0[i];
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          __builtin_amdgcn_sched_barrier(0);
          float B[4][kNS], C[4][kNS], y[4];
          unrolled<0, 4>([&](auto r) {
            const float dt = from_owner<4>(delta[j], r);
#pragma unroll
            for (int i = 0; i < kNS; ++i) as[4 * j + r][i] = exp2_hw(dt * Ap[i]);
          });
          unrolled<0, 4>([&](auto r) {
            if (r % 2 == 0) {  // two steps' operands
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int i = r; i <= r + 1; ++i) {
                load_states<kNS>(bc + (4 * j + i) * 2 * kNP, B[i]);
                if (kGate) load_states<kNS>(bc + (4 * j + i) * 2 * kNP + kNP, C[i]);
              }
            }
            const float wt = from_owner<4>(w[j], r);
            const int t = 4 * j + r;
            y[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < kNS; ++i) {
              hs[t + 1][i] = fmaf(as[t][i], hs[t][i], wt * B[r][i]);
              if (kGate) y[r] = i ? fmaf(C[r][i], hs[t + 1][i], y[r]) : C[r][i] * hs[t + 1][i];
            }
          });
          if (kGate) {
            const float v = fmaf(skip, u[j], quad_scatter_sum(y[0], y[1], y[2], y[3], odd, high));
            // SiLU'(z) = sigmoid(z) (1 + z (1 - sigmoid(z)))
            const float slope = sg[j] == 0.0f ? 0.0f : (sg[j] == 1.0f ? 1.0f : sg[j] * fmaf(z[j], 1.0f - sg[j], 1.0f));
            if (on && s + 4 * j < left) element(qz + j * 4 * int64_t(a.D), opaque(og)) = Elem<T>::from_f32(g[j] * v * slope);
          }
        }
        // B and C are read again: kept from above, they would take 128 registers
        asm volatile("" ::: "memory");
#pragma unroll
        for (int j = kOwn - 1; j >= 0; --j) {
          // groups of steps are kept apart, or their operands would not fit the registers; the next
          // tile is loaded once half of the states held here are used up
          __builtin_amdgcn_sched_barrier(0);
          if (j == kOwn / 2 - 1) fetch(k > 0 ? kTile : 0);
          __builtin_amdgcn_sched_barrier(0);
          float P[4], Q[4], acc[kNY], B[4][kNS], C[4][kNS];
          unrolled<0, 4>([&](auto k) {
            constexpr int r = 3 - k;
            const int t = 4 * j + r;
            if (r % 2 == 1) {  // two steps' operands
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int i = r - 1; i <= r; ++i) {
                load_states<kNS>(bc + (4 * j + i) * 2 * kNP, B[i]);
                load_states<kNS>(bc + (4 * j + i) * 2 * kNP + kNP, C[i]);
              }
            }
            const float dt = from_owner<4>(delta[j], r), wt = from_owner<4>(w[j], r), gt = from_owner<4>(gy[j], r);
            float dB[kNS], dC[kNS], out[kNY];
#pragma unroll
            for (int i = 0; i < kNS; ++i) {
              const float lam = fmaf(gt, C[r][i], carry[i]);
              dB[i] = lam * wt;
              dC[i] = gt * hs[t + 1][i];
              Q[r] = i ? fmaf(lam, B[r][i], Q[r]) : lam * B[r][i];
              carry[i] = as[t][i] * lam;
              const float v = carry[i] * hs[t][i];
              dA[i] = fmaf(dt, v, dA[i]);
              P[r] = i ? fmaf(v, Ap[i], P[r]) : v * Ap[i];
            }
            channel_sums<kNS>(dB, dC, out);
#pragma unroll
            for (int m = 0; m < kNY; ++m) acc[m] = r == 3 || bank == r ? out[m] : acc[m];
          });
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
          const float draw = fmaf(u[j], qs, ps) * __builtin_amdgcn_rcpf(1.0f + exp2_hw(-raw[j] * kLog2e));
          const float du = fmaf(delta[j], qs, skip * gy[j]);
          if (on && s + 4 * j < left) {
            const uint32_t at = opaque(og);
            element(qu + j * 4 * int64_t(a.D), at) = Elem<T>::from_f32(du);
            element(qd + j * 4 * int64_t(a.D), at) = Elem<T>::from_f32(draw);
            dD = fmaf(gy[j], u[j], dD);
            dbias += draw;
          }
        }
      }
    }
    if (kAll) {
      qu -= int64_t(kTile) * a.D;
      qd -= int64_t(kTile) * a.D;
      if (kGate) qz -= int64_t(kTile) * a.D;
    }
  }
  if constexpr (kAll) {
    if (tiles > 0) {
      __syncthreads();
      flush(buf ^ 1, static_cast<int>(min(steps, int64_t(kTile))));
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

// dB and dC: the sums over the channel blocks, for units of kSumTokens tokens of one sequence.
constexpr int kSumTokens = 16;
template <typename T>
__global__ __launch_bounds__(256) void k_scan_sum_bc(Args a) {
  int64_t idx;
  const Sequence q = sequence_of(a.q, blockIdx.x, kSumTokens, &idx);
  const int64_t t0 = idx * kSumTokens;
  if (t0 >= q.len) return;
  const int64_t row = q.b * a.q.L + q.begin + t0;
  const int width = a.G * 2 * a.N, count = static_cast<int>(min(q.len - t0, int64_t(kSumTokens))) * width;
  const int64_t stride = a.q.T * width;
  const float* parts = a.bc_parts + row * width;
  for (int e = threadIdx.x; e < count; e += 256) {
    constexpr int kAhead = 8;
    float x[kAhead] = {};
    const float* p = parts + e;
    int b = 0;
    for (; b + kAhead <= a.cbg; b += kAhead, p += kAhead * stride)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) x[i] += p[i * stride];
    for (; b < a.cbg; ++b, p += stride) x[0] += *p;
    const float v = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    const int tg = e / (2 * a.N), n = e % (2 * a.N);
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

template <typename T, int kNS, bool kAll>
int launch_gate(const Args& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.units * a.G * a.cbg)), block(kThreads);
  if (a.z) hipLaunchKernelGGL((k_scan_adjoint<T, kNS, kAll, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_scan_adjoint<T, kNS, kAll, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T, bool kAll>
int launch_states(const Args& a, hipStream_t st) {
  switch (lane_states(a.N)) {
    case 1: return launch_gate<T, 1, kAll>(a, st);
    case 2: return launch_gate<T, 2, kAll>(a, st);
    case 4: return launch_gate<T, 4, kAll>(a, st);
    default: return launch_gate<T, 8, kAll>(a, st);
  }
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
  if (width == 0) return static_cast<int>(hipGetLastError());  // no channels: dB and dC, of 0, alone
  hipLaunchKernelGGL(k_scan_sum_params, dim3(static_cast<unsigned>((width + 63) / 64)), dim3(1024), 0, st, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace sscan
}  // namespace ss2d
