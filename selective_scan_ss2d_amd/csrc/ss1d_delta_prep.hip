// Chunk matrices of the gated delta rule, every chunk and value head on its own: the gates,
// P (or P^T), N (or N^T) and, once per key head, K^T (and Q^T), all written as the matrix
// fragments that the sequential kernels load with one 16-byte access per lane.
//
// One wave per chunk and value head: k.k and q.k of all pairs on the matrix cores, the solve with
// one row (column) of N per lane.  Bound by HBM: 24.5 KB of records per chunk and head of 64 in
// bfloat16.  64 x 3136 tokens of 3 heads of 64: 461 MB written and 136 read in 124 us (4.8 TB/s,
// a copy reaches 5.0), 152 us for the backward's, which turns Q as well.
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

constexpr int kWaves = 4;

struct Shared {
  double G[kC];
  float beta[kC];
  float m[kC * kC];   // the triangular matrix of the solve, rows of 32
  float t[kC * 36];   // a 32 x 32 tile on its way through a transpose
};

// Transposes one operand tile: lane (token swap23(l % 32)) holds 8 columns per step; the
// result's lane holds column swap23(l % 32), tokens 16 s + 8 half + 0..7.
template <typename T>
__device__ __forceinline__ void transpose_tile(Shared& sh, const Exact<T>* x, Exact<T>* y, int own,
                                               int half) {
  T* t = reinterpret_cast<T*>(sh.t);
  wave_sync();
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const auto v = x[s].v[e];
      t[own * 36 + 16 * s + 8 * half + e] = __builtin_bit_cast(T, v);
    }
  wave_sync();
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const T v = t[(16 * s + 8 * half + e) * 36 + own];
      if constexpr (sizeof(T) == 4) y[s].v[e] = v;
      else y[s].v[e] = __builtin_bit_cast(__bf16, v);
    }
}

template <typename T, int KT, bool kAligned, bool kBackward>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(4)))
void k_delta_prep(Args a) {
  __shared__ Shared shared[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Shared& sh = shared[wave];
  const int64_t unit = int64_t(blockIdx.x) * kWaves + wave;
  const int64_t slot = unit / a.H;
  const int hv = static_cast<int>(unit - slot * a.H);
  if (slot >= a.slots) return;
  int64_t n, c;
  Seq seq;
  if (!find_slot(a, slot, kC, &n, &c, &seq)) return;
  const int hk = hv / a.rep;
  const int half = lane >> 5, col = lane & 31, own = swap23(col);
  const int64_t t0 = c * kC;
  const int valid = static_cast<int>(min<int64_t>(kC, seq.len - t0));

  // K and Q rows of this lane's token; q.k and k.k of all pairs
  const bool on = own < valid;
  const int64_t tok = t0 + (on ? own : 0);
  const T* krow = static_cast<const T*>(a.k) + token_at(a, a.sk, n, seq, tok) + hk * a.sk.h;
  const T* qrow = static_cast<const T*>(a.q) + token_at(a, a.sq, n, seq, tok) + hk * a.sq.h;
  f32x16 kk = {}, qk = {};
  const bool keyed = hv % a.rep == 0;
  constexpr int64_t frag = exact_planes<T>() * kPlane;
  constexpr int64_t operand = KeyRecord<T, KT>::kOperand * kPlane;
  char* const head = a.heads + (slot * a.H + hv) *
                                   (int64_t(head_planes(sizeof(T) == 4, a.p_planes)) * kPlane);
  char* const pf = head + HeadRecord<T, 3>::kPStart * kPlane;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    Exact<T> kx[2], qx[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      load8<kAligned>(kx[s], krow, 32 * kt + 16 * s + 8 * half, a.DK, on);
      load8<kAligned>(qx[s], qrow, 32 * kt + 16 * s + 8 * half, a.DK, on);
      kk = mma(kx[s], kx[s], kk);
      // forward: rows k_j, columns q_i; backward: rows q_i, columns k_j
      qk = kBackward ? mma(qx[s], kx[s], qk) : mma(kx[s], qx[s], qk);
    }
    if (keyed) {
      char* at = a.keys + (slot * a.HK + hk) * (int64_t(KeyRecord<T, KT>::kPlanes) * kPlane) +
                 2 * kt * frag;
      Exact<T> y[2];
      transpose_tile<T>(sh, kx, y, own, half);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        put(at + s * frag, lane, kx[s]);
        put(at + operand + s * frag, lane, y[s]);
      }
      if (kBackward) transpose_tile<T>(sh, qx, y, own, half);
#pragma unroll
      for (int s = 0; s < 2; ++s) put(at + 2 * operand + s * frag, lane, kBackward ? y[s] : qx[s]);
    }
  }

  // gates
  const int64_t row = seq.row + t0 + (col < valid ? col : 0);
  float gv = 0.0f, bv = 0.0f;
  if (col < valid) {
    gv = bounded_log(a.g[row * a.H + hv]);
    bv = a.beta[row * a.H + hv];
  }
  double G = gv * kLog2eWide;
#pragma unroll
  for (int d = 1; d < kC; d *= 2) {
    const double up = __shfl_up(G, d, 32);
    if (col >= d) G += up;
  }
  const double Gend = __shfl(G, 31, 32);
  if (half == 0) {
    sh.G[col] = G;
    sh.beta[col] = bv;
    float* gt = reinterpret_cast<float*>(head + HeadRecord<T, 3>::kGates * kPlane);
    gt[col] = decay_of(G);
    gt[kC + col] = decay_of(Gend - G);
    gt[2 * kC + col] = bv;
  }
  wave_sync();
  const double Gown = sh.G[own];
  const float bown = sh.beta[own];
  float low[16];  // L: forward, row `own`, columns acc_row; backward, column `own`, rows acc_row
  f32x16 p;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int other = acc_row(r, half);
    const double diff = kBackward ? sh.G[other] - Gown : Gown - sh.G[other];
    const bool below = kBackward ? other > own : other < own;
    const float m = (below || other == own) ? decay_of(diff) : 0.0f;
    low[r] = below ? kk[r] * m : 0.0f;
    p[r] = (below || other == own) ? qk[r] * m * a.scale : 0.0f;
  }
  // The unknowns are solved for from the last to the first in either sense: counted upwards the
  // backward's rows of the matrix were all loaded at once, into 450 registers (187 us, now 152).
  // The solve's matrix: forward, row j holds beta_k L_kj over k (N row by row, from
  // n (I + diag(beta) L) = l); backward, row i holds L_ij beta_j over j, with rows, columns and
  // the unknowns in reverse order, so that both are solved from the last to the first
  auto at = [](int i) { return kBackward ? kC - 1 - i : i; };
  float finite = 0.0f;  // NaN if one of this lane's values is not finite
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float value = low[r] * bown;
    sh.m[at(acc_row(r, half)) * kC + at(own)] = value;
    finite = fmaf(value, 0.0f, finite);
  }
  // The solve multiplies by the unknowns' leading zeros too, where a NaN or infinity would reach
  // the tokens before it (backward: behind it).  From the first token that has one on, the matrix
  // is then set to zero, and the unknowns of the tokens past that one to NaN.
  int bad = kC;
  if (__builtin_expect(__any(finite != finite), 0)) {
    bad = finite != finite ? at(own) : kC;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) bad = min(bad, __shfl_xor(bad, d));
    if (at(own) >= bad)
#pragma unroll
      for (int r = 0; r < 16; ++r) sh.m[at(acc_row(r, half)) * kC + at(own)] = 0.0f;
  }
  float x[kC];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float mine = low[8 * s + e], theirs = __shfl_xor(mine, 32);
      x[at(16 * s + e)] = half == 0 ? mine : theirs;
      x[at(16 * s + 8 + e)] = half == 0 ? theirs : mine;
    }
  wave_sync();
#pragma unroll
  for (int j = kC - 2; j >= 0; --j)
#pragma unroll
    for (int k = kC - 1; k > j; --k) x[j] = fmaf(-sh.m[j * kC + k], x[k], x[j]);
  if (__builtin_expect(bad < kC, 0) && at(own) > bad)
#pragma unroll
    for (int i = 0; i < kC; ++i) x[i] = __builtin_nanf("");
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    f32x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = half == 0 ? x[at(16 * s + e)] : x[at(16 * s + 8 + e)];
    Wide<T, 3> w;
    set_wide(w, v);
    put(head + s * wide_planes<T, 3>() * kPlane, lane, w);
    if (a.p_planes == 3) {
      set_wide(w, part(p, s));
      put(pf + s * wide_planes<T, 3>() * kPlane, lane, w);
    } else {
      Wide<T, 2> w2;
      set_wide(w2, part(p, s));
      put(pf + s * wide_planes<T, 2>() * kPlane, lane, w2);
    }
  }
}

template <typename T, int KT, bool kAligned>
int launch_kt(const Args& a, bool backward, hipStream_t st) {
  const int64_t waves = a.slots * a.H;
  const dim3 grid(static_cast<unsigned>((waves + kWaves - 1) / kWaves)), block(64 * kWaves);
  if (backward) hipLaunchKernelGGL((k_delta_prep<T, KT, kAligned, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_prep<T, KT, kAligned, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T, bool kAligned>
int launch_t(const Args& a, bool backward, hipStream_t st) {
  if (a.DK <= 32) return launch_kt<T, 1, kAligned>(a, backward, st);
  if (a.DK <= 64) return launch_kt<T, 2, kAligned>(a, backward, st);
  return launch_kt<T, 4, kAligned>(a, backward, st);
}

}  // namespace

int launch_prep(const Args& a, int dtype, bool aligned, bool backward, hipStream_t st) {
  if (dtype == 0)
    return aligned ? launch_t<float, true>(a, backward, st) : launch_t<float, false>(a, backward, st);
  return aligned ? launch_t<uint16_t, true>(a, backward, st)
                 : launch_t<uint16_t, false>(a, backward, st);
}

}  // namespace delta
}  // namespace ss2d
