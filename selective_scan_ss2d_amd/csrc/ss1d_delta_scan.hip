// The sequential pass of the gated delta rule's forward: one wave carries 32 columns of one
// sequence and head's state through its chunks, the state in registers, the chunk's operands
// in LDS, where the block's waves (adjacent columns) share them, loaded a chunk ahead.
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

// kP: bf16 terms of the operands of o (2 leave o to its own rounding; 3 hold fp32, for the
// training forward, whose backward forms the decays' gradient from o).
template <typename T, int KT, int kW, bool kSave>
__global__ __launch_bounds__(64 * kW) void k_delta_scan(Args a) {
  constexpr int kP = kSave ? 3 : 2;
  using St = Stage<T, KT, kP, kW>;
  __shared__ __align__(16) char buffers[2][St::kPlanes * kPlane];
  __shared__ __align__(16) char tiles[kW][kTileBytes];
  const Place w = place<kW>(a, blockIdx.x);
  const int lane = w.lane, half = w.half;
  char* const lds = tiles[w.wave];
  const Seq seq = sequence(a, w.n);
  const int64_t slot0 = first_slot(a, w.n, seq, kC), mark0 = first_slot(a, w.n, seq, kMark);
  const int64_t state = w.head * a.DK * a.DV + 32 * w.tile;
  const uint32_t vline = static_cast<uint32_t>(a.sv.l) * sizeof(T), line = a.H * a.DV;

  f32x16 S[KT];
  load_state<KT>(S, a.h0 ? a.h0 + state : nullptr, a, w, lds);
  const int64_t chunks = (seq.len + kC - 1) / kC;
  St stage;
  Tile<T> vx;
  auto fetch = [&](int64_t c) {
    stage.fetch(a, slot0 + c, w.hv, w.hk, w.wave, lane);
    const T* at = static_cast<const T*>(a.v) + token_at(a, a.sv, w.n, seq, c * kC) + w.hv * a.sv.h;
    vx.fetch(at + 32 * w.tile, vline, lane, static_cast<int>(min<int64_t>(kC, seq.len - c * kC)), w.cols);
  };
  if (chunks > 0) {
    fetch(0);
    stage.commit(buffers[0], w.wave, lane);
    __syncthreads();
  }
  for (int64_t c = 0; c < chunks; ++c) {
    const int64_t t0 = c * kC;
    const int valid = static_cast<int>(min<int64_t>(kC, seq.len - t0));
    const char* buf = buffers[c & 1];
    const f32x16 v = vx.columns(lds, lane);
    if (c + 1 < chunks) fetch(c + 1);
    __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the products
    if (kSave && (c & 1) == 0)
      store_state<float, KT>(S, a.marks + ((mark0 + (c >> 1)) * a.H + w.hv) * a.DK * a.DV + 32 * w.tile,
                             a, w, lds);
    f32x16 ks = {}, qs = {};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> kx, qx;
        get(kx, St::operand(buf, 0, kt, s), lane);
        get(qx, St::operand(buf, 2, kt, s), lane);
        Wide<T, 3> sw;
        set_wide(sw, part(S[kt], s));
        ks = mma(kx, sw, ks);
        if constexpr (kP == 3 || sizeof(T) == 4) {
          qs = mma(qx, sw, qs);
        } else {
          Wide<T, 2> w2;
          w2.p[0] = sw.p[0];
          w2.p[1] = sw.p[1];
          qs = mma(qx, w2, qs);
        }
      }
    const float* gate = St::gates(buf);
    const f32x16 gam = load_gate(gate, half), beta = load_gate(gate + 2 * kC, half);
    f32x16 t = v - gam * ks;
    const f32x16 br = beta * t;
    f32x16 nr = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> nw, rw;
      get(nw, St::n(buf, s), lane);
      set_wide(rw, part(br, s));
      nr = mma(nw, rw, nr);
    }
    t -= nr;
    const f32x16 u = beta * t;
    const f32x16 eu = load_gate(gate + kC, half) * u;
    const float whole = gate[kC - 1];
    Wide<T, 3> ew[2];
    set_wide(ew[0], part(eu, 0));
    set_wide(ew[1], part(eu, 1));
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      S[kt] *= whole;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> kx;
        get(kx, St::operand(buf, 1, kt, s), lane);
        S[kt] = mma(kx, ew[s], S[kt]);
      }
    }
    f32x16 pu = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, kP> pw, uw;
      get(pw, St::p(buf, s), lane);
      set_wide(uw, part(u, s));
      pu = mma(pw, uw, pu);
    }
    const f32x16 o = a.scale * (gam * qs) + pu;
    const int64_t at = (seq.row + t0) * line + w.hv * a.DV + 32 * w.tile;
    store_tile<T>(o, static_cast<T*>(a.o) + at, line * sizeof(T), lds, lane, valid, w.store_cols);
    if (kSave) {
      store_tile<float>(t, a.ts + at, line * 4, lds, lane, valid, w.store_cols);
      store_tile<float>(o, a.os + at, line * 4, lds, lane, valid, w.store_cols);
    }
    if (c + 1 < chunks) stage.commit(buffers[(c + 1) & 1], w.wave, lane);
    __syncthreads();
  }
  if (a.ht) store_state<float, KT>(S, a.ht + state, a, w, lds);
  if (kSave) store_state<float, KT>(S, a.ends + state, a, w, lds);
}

template <typename T, int KT, int kW>
int launch_w(const Args& a, bool save, hipStream_t st) {
  const int64_t blocks = a.S * a.H * (((a.DV + 31) / 32 + kW - 1) / kW);
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * kW);
  if (save) hipLaunchKernelGGL((k_delta_scan<T, KT, kW, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_scan<T, KT, kW, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T, int KT>
int launch_kt(const Args& a, bool save, hipStream_t st) {
  if (a.DV <= 32) return launch_w<T, KT, 1>(a, save, st);
  if (a.DV <= 64) return launch_w<T, KT, 2>(a, save, st);
  return launch_w<T, KT, 4>(a, save, st);
}

template <typename T>
int launch_t(const Args& a, bool save, hipStream_t st) {
  if (a.DK <= 32) return launch_kt<T, 1>(a, save, st);
  if (a.DK <= 64) return launch_kt<T, 2>(a, save, st);
  return launch_kt<T, 4>(a, save, st);
}

}  // namespace

int launch_scan(const Args& a, int dtype, bool save, hipStream_t st) {
  return dtype == 0 ? launch_t<float>(a, save, st) : launch_t<uint16_t>(a, save, st);
}

}  // namespace delta
}  // namespace ss2d
