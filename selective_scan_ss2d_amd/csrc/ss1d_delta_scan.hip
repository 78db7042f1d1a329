// The sequential pass of the gated delta rule's forward: one wave carries 32 columns of one
// sequence and head's state through its chunks, the state in registers.
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

// kP: bf16 terms of the operands of o (2 leave o to its own rounding; 3 hold fp32, for the
// training forward, whose backward forms the decays' gradient from o).
template <typename T, int KT, bool kAligned, bool kSave>
__global__ __launch_bounds__(64) void k_delta_scan(Args a) {
  constexpr int kP = kSave ? 3 : 2;
  const int lane = threadIdx.x, half = lane >> 5, own = swap23(lane & 31);
  const int tiles = (a.DV + 31) / 32;
  const int64_t unit = blockIdx.x;
  const int64_t head = unit / tiles;
  const int tile = static_cast<int>(unit - head * tiles);
  const int64_t n = head / a.H;
  const int hv = static_cast<int>(head - n * a.H), hk = hv / a.rep;
  const int col = 32 * tile + (lane & 31);
  const bool in = col < a.DV;
  const Seq seq = sequence(a, n);
  const int64_t slot0 = first_slot(a, n, seq, kC);

  f32x16 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int d = 32 * kt + acc_row(r, half);
      S[kt][r] = a.h0 && in && d < a.DK ? a.h0[(head * a.DK + d) * a.DV + col] : 0.0f;
    }

  const int64_t chunks = (seq.len + kC - 1) / kC;
  for (int64_t c = 0; c < chunks; ++c) {
    const int64_t t0 = c * kC, slot = slot0 + c;
    const int valid = static_cast<int>(min<int64_t>(kC, seq.len - t0));
    if (kSave && (c & 1) == 0 && in) {
      const int64_t mark = first_slot(a, n, seq, kMark) + (c >> 1);
      float* at = a.marks + (mark * a.H + hv) * a.DK * a.DV + col;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int d = 32 * kt + acc_row(r, half);
          if (d < a.DK) at[int64_t(d) * a.DV] = S[kt][r];
        }
    }
    const bool on = own < valid;
    const int64_t tok = t0 + (on ? own : 0);
    const T* krow = static_cast<const T*>(a.k) + token_at(a, a.sk, n, seq, tok) + hk * a.sk.h;
    const T* qrow = static_cast<const T*>(a.q) + token_at(a, a.sq, n, seq, tok) + hk * a.sq.h;
    f32x16 ks = {}, qs = {};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> kx, qx;
        load8<kAligned>(kx, krow, 32 * kt + 16 * s + 8 * half, a.DK, on);
        load8<kAligned>(qx, qrow, 32 * kt + 16 * s + 8 * half, a.DK, on);
        Wide<T, 3> w;
        set_wide(w, part(S[kt], s));
        ks = mma(kx, w, ks);
        if constexpr (kP == 3 || sizeof(T) == 4) {
          qs = mma(qx, w, qs);
        } else {
          Wide<T, 2> w2;
          w2.p[0] = w.p[0];
          w2.p[1] = w.p[1];
          qs = mma(qx, w2, qs);
        }
      }
    const float* gate = a.gates + (slot * a.H + hv) * (3 * kC);
    const f32x16 gam = load_gate(gate, half), beta = load_gate(gate + 2 * kC, half);
    const T* vat = static_cast<const T*>(a.v) + token_at(a, a.sv, n, seq, t0) + hv * a.sv.h + col;
    f32x16 t = load_columns<T>(vat, a.sv.l, half, valid, in) - gam * ks;
    const f32x16 br = beta * t;
    const char* nf = a.nf + (slot * a.H + hv) * n_bytes<T>();
    const char* pf = a.pf + (slot * a.H + hv) * p_bytes<T>(kP);
    f32x16 nr = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> nw, rw;
      get(nw, nf + s * wide_planes<T, 3>() * kPlane, lane);
      set_wide(rw, part(br, s));
      nr = mma(nw, rw, nr);
    }
    t -= nr;
    const f32x16 u = beta * t;
    f32x16 pu = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, kP> pw, uw;
      get(pw, pf + s * wide_planes<T, kP>() * kPlane, lane);
      set_wide(uw, part(u, s));
      pu = mma(pw, uw, pu);
    }
    const f32x16 o = a.scale * (gam * qs) + pu;
    if (in) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int i = acc_row(r, half);
        if (i < valid) {
          const int64_t at = ((seq.row + t0 + i) * a.H + hv) * a.DV + col;
          static_cast<T*>(a.o)[at] = Elem<T>::from_f32(o[r]);
          if (kSave) {
            a.ts[at] = t[r];
            a.os[at] = o[r];
          }
        }
      }
    }
    const f32x16 eu = load_gate(gate + kC, half) * u;
    const float whole = gate[kC - 1];
    const char* ktf = a.ktf + (slot * a.HK + hk) * t_bytes<T>(KT);
    Wide<T, 3> uw[2];
    set_wide(uw[0], part(eu, 0));
    set_wide(uw[1], part(eu, 1));
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      S[kt] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> kx;
        get(kx, ktf + (2 * kt + s) * exact_planes<T>() * kPlane, lane);
        S[kt] = mma(kx, uw[s], S[kt]);
      }
    }
  }
  if (in)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int d = 32 * kt + acc_row(r, half);
        if (d >= a.DK) continue;
        if (a.ht) a.ht[(head * a.DK + d) * a.DV + col] = S[kt][r];
        if (kSave) a.ends[(head * a.DK + d) * a.DV + col] = S[kt][r];
      }
}

template <typename T, int KT, bool kAligned>
int launch_kt(const Args& a, bool save, hipStream_t st) {
  const int64_t blocks = a.S * a.H * ((a.DV + 31) / 32);
  const dim3 grid(static_cast<unsigned>(blocks)), block(64);
  if (save) hipLaunchKernelGGL((k_delta_scan<T, KT, kAligned, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_scan<T, KT, kAligned, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T, bool kAligned>
int launch_t(const Args& a, bool save, hipStream_t st) {
  if (a.DK <= 32) return launch_kt<T, 1, kAligned>(a, save, st);
  if (a.DK <= 64) return launch_kt<T, 2, kAligned>(a, save, st);
  return launch_kt<T, 4, kAligned>(a, save, st);
}

}  // namespace

int launch_scan(const Args& a, int dtype, bool aligned, bool save, hipStream_t st) {
  if (dtype == 0)
    return aligned ? launch_t<float, true>(a, save, st) : launch_t<float, false>(a, save, st);
  return aligned ? launch_t<uint16_t, true>(a, save, st) : launch_t<uint16_t, false>(a, save, st);
}

}  // namespace delta
}  // namespace ss2d
