// The sequential pass of the gated delta rule's forward: one wave carries 32 columns of one
// sequence and head's state through its chunks, the state in registers, the chunk's operands
// in LDS, where the block's waves (adjacent columns) share them, loaded a chunk ahead.
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

// Operands hold 24 bits (3 bf16 terms), those of o 17 (2 terms, which leaves o to its own
// rounding); with kSave, the training forward, o's hold 24 as well, because the backward
// forms the decays' gradient from o.
template <typename T, int KT, int kW, bool kSave>
__global__ __launch_bounds__(64 * kW) __attribute__((amdgpu_waves_per_eu(kSave ? 1 : 2)))
void k_delta_scan(Args a) {
  constexpr int kP = kSave ? 3 : 2;
  using St = Stage<T, KT, kP, kW>;
  __shared__ __align__(16) char buffers[2][St::kPlanes * kPlane];
  __shared__ __align__(16) char spare[kW][kTileBytes];
  const Place w = place<kW>(a, blockIdx.x);
  const int lane = w.lane, half = w.half;
  char* const lds = spare[w.wave];
  const Seq seq = sequence(a, w.n);
  const int64_t slot0 = first_slot(a, w.n, seq, kC);
  const int64_t state = w.head * a.DK * a.DV + 32 * w.tile;
  const int64_t chunks = (seq.len + kC - 1) / kC;

  f32x16 S[KT];
  load_state<KT>(S, a.h0 ? a.h0 + state : nullptr, a, w, lds);
  float factor = 1.0f;

  const int64_t first = seq.row * a.H * a.DV + w.hv * a.DV + 32 * w.tile;
  const uint32_t vline = static_cast<uint32_t>(a.sv.l) * sizeof(T), line = a.H * a.DV;
  const T* vat = static_cast<const T*>(a.v) + token_at(a, a.sv, w.n, seq, 0) + w.hv * a.sv.h + 32 * w.tile;
  T* oat = static_cast<T*>(a.o) + first;
  const bool valign = aligned16(vat, vline, w.cols);
  const bool oalign = aligned16(oat, line * sizeof(T), w.store_cols);
  const bool salign = aligned16(nullptr, line * 4, w.store_cols);
  float* tat = kSave ? a.ts + first : nullptr;
  float* pat = kSave ? a.os + first : nullptr;
  float* mat = kSave ? a.marks + (first_slot(a, w.n, seq, kMark) * a.H + w.hv) * a.DK * a.DV + 32 * w.tile
                     : nullptr;
  int left = static_cast<int>(min<int64_t>(seq.len, 1 << 30));  // tokens of this and later chunks

  St stage;
  Tile<T> vx;
  if (chunks > 0) {
    stage.start(a, slot0, w.hv, w.hk, w.wave, lane, 1);
    stage.fetch();
    if (valign && left >= kC) vx.fetch(vat, vline, lane);
    stage.commit(buffers[0]);
    __syncthreads();
  }
  for (int64_t c = 0; c < chunks; ++c) {
    left = static_cast<int>(min<int64_t>(seq.len - c * kC, 1 << 30));
    const bool whole = left >= kC;
    const char* buf = buffers[c & 1];
    const f32x16 v = vx.columns(valign && whole, vat, vline, left, w.cols, lds, lane);
    vat += kC * a.sv.l;
    if (c + 1 < chunks) {
      stage.fetch();
      if (valign && left >= 2 * kC) vx.fetch(vat, vline, lane);
    }
    __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the products
    if (kSave && (c & 1) == 0) {
      store_state<float, KT>(S, mat, factor, a, w, lds);
      mat += int64_t(a.H) * a.DK * a.DV;
    }
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
        qs = mma(qx, first_terms<kP>(sw), qs);
      }
    const float* gate = St::gates(buf);
    const f32x16 gam = load_gate(gate, half) * factor, beta = load_gate(gate + 2 * kC, half);
    f32x16 t = v - gam * ks;
    f32x16 nr = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> nw, rw;
      get(nw, St::n(buf, s), lane);
      set_wide(rw, part(beta * t, s));
      nr = mma(nw, rw, nr);
    }
    t -= nr;
    const f32x16 u = beta * t;
    factor = decay_state<KT>(S, factor, gate[kC - 1]);
    const f32x16 eu = load_gate(gate + kC, half) * (1.0f / factor) * u;
    Wide<T, 3> ew[2];
    set_wide(ew[0], part(eu, 0));
    set_wide(ew[1], part(eu, 1));
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> kx;
        get(kx, St::operand(buf, 1, kt, s), lane);
        S[kt] = mma(kx, ew[s], S[kt]);
      }
    f32x16 pu = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, kP> pw, uw;
      get(pw, St::p(buf, s), lane);
      set_wide(uw, part(u, s));
      pu = mma(pw, uw, pu);
    }
    const f32x16 o = a.scale * gam * qs + pu;
    store_tile<T>(o, oat, line * sizeof(T), oalign && whole, left, w.store_cols, lds, lane);
    oat += kC * int64_t(line);
    if (kSave) {
      store_tile<float>(t, tat, line * 4, salign && whole, left, w.store_cols, lds, lane);
      store_tile<float>(o, pat, line * 4, salign && whole, left, w.store_cols, lds, lane);
      tat += kC * int64_t(line);
      pat += kC * int64_t(line);
    }
    if (c + 1 < chunks) stage.commit(buffers[(c + 1) & 1]);
    __syncthreads();
  }
  if (a.ht) store_state<float, KT>(S, a.ht + state, factor, a, w, lds);
  if (kSave) store_state<float, KT>(S, a.ends + state, factor, a, w, lds);
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
