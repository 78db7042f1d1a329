// Backward of the gated delta rule.
//
// With dS the gradient of the state after a chunk (notation of ss1d_delta.h, e_j =
// e^(G_32 - G_j)), the adjoint runs backwards over the chunks:
//   du = P^T do + e K dS,   w = du - N^T (beta du),   dv = beta w,   dbeta_i = w_i . t_i,
//   dS <- e^G_32 dS + scale Q^T (e^G do) - K^T (e^G dv).
// The decays' gradient needs no products of its own: raising every log decay from token i on
// scales what token i's v contributes and what its o receives, so
//   dg_t = sum_{i >= t, same block} (do_i . o_i - dv_i . v_i) + <dS, S> after the block,
// with o in fp32 (the terms cancel, and its rounding would not).  And over blocks of 64
// tokens, independent of each other, from the states before and the gradients after each:
//   dq = scale e^G do S^T + dP K,   dP_ij = scale e^(G_i - G_j) do_i . u_j      (j <= i)
//   dk = e u dS^T - e^G dv S^T + dP^T Q + (dL + dL^T) K,
//                                   dL_ij = -e^(G_i - G_j) dv_i . u_j           (j < i).
//
// The adjoint is bound by the latency of a chunk's chain, as the forward's scan is, and by its
// registers (256 and up to 256 accumulation registers, one wave per SIMD; held to two waves per
// SIMD it spills 120 of them and takes 486 us instead of 313 in segments of 20 chunks).  64 x
// 3136 tokens of 3 heads of 64 in bfloat16: 478 to 490 us uncut (457 before it kept dv and the
// states' gradients in fp32), dq and dk 266 to 274 us.
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

// Sums each register over the 32 lanes of a half: lane l of the half gets the sum of
// register row_of(l) (each twice).  Halving the registers at every exchange costs 16
// exchanges for 16 sums; the first 8, between rows of 16 lanes, are the swap itself.
template <int kN> __device__ __forceinline__ void halve(float* x, int lane) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    if constexpr (kN == 8) {
      swap_rows(x[i], x[kN + i]);
      x[i] += x[kN + i];
    } else {
      const bool up = lane & (2 * kN);
      const float keep = up ? x[kN + i] : x[i], send = up ? x[i] : x[kN + i];
      x[i] = keep + from_lane<2 * kN>(send);
    }
  }
  if constexpr (kN > 1) halve<kN / 2>(x, lane);
}
__device__ __forceinline__ float sum_columns(const f32x16& v, int lane) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = v[i];
  halve<8>(x, lane);
  return x[0] + from_lane<1>(x[0]);
}
__device__ __forceinline__ int row_of(int lane) { return (lane & 31) >> 1; }

// One wave per (sequence, head, 32 columns), kW adjacent ones per block sharing the chunks'
// operands through LDS, chunks last to first.
// kSpan: the span pass over segments (see the forward): only the gradient before a segment,
// from zero after it, is kept.
template <typename T, int KT, int kW, bool kSpan>
__global__ __launch_bounds__(64 * kW)
__attribute__((amdgpu_waves_per_eu(kSpan ? 2 : 1))) void k_delta_adjoint(Args a) {
  using St = Stage<T, KT, 3, kW>;
  __shared__ __align__(16) char buf[St::kPlanes * kPlane];
  __shared__ __align__(16) char spare[kW][kTileBytes];
  Place w;
  if (!place<kW>(&w, a, blockIdx.x, a.DV)) return;
  const Segment& g = w.g;
  if (kSpan && (g.index == 0 || g.end == g.begin)) return;  // nothing comes before the first one
  const int lane = w.lane, half = w.half, tiles = (a.DV + 31) / 32;
  char* const lds = spare[w.wave];
  const Seq& seq = g.seq;
  const int64_t mark0 = first_slot(a, g.n, seq, kMark);
  const int64_t state = w.head * a.DK * a.DV + 32 * w.tile;
  const int64_t start = (g.slot * a.H + w.hv) * a.DK * a.DV + 32 * w.tile;
  const uint32_t vline = static_cast<uint32_t>(a.sv.l) * sizeof(T), line = a.H * a.DV;

  f32x16 dS[KT];
  const float* after_all = g.last ? (a.dht ? a.dht + state : nullptr) : a.starts + start;
  load_state<KT>(dS, kSpan ? nullptr : after_all, a, w, lds);
  float factor = 1.0f;
  const int64_t chunks = (seq.len + kC - 1) / kC;  // of the sequence
  const int64_t first = seq.row * line + w.hv * a.DV + 32 * w.tile;
  const T* v0 = static_cast<const T*>(a.v) + token_at(a, a.sv, g.n, seq, 0) + w.hv * a.sv.h + 32 * w.tile;
  const T* d0 = static_cast<const T*>(a.dout) + first;
  T* out0 = static_cast<T*>(a.dv) + first;
  const bool valign = aligned16(v0, vline, w.cols), dalign = aligned16(d0, line * sizeof(T), w.cols);
  const bool oalign = aligned16(out0, line * sizeof(T), w.store_cols);
  const bool salign = aligned16(nullptr, line * 4, w.cols), walign = aligned16(nullptr, line * 4, w.store_cols);
  const bool malign = aligned16(nullptr, a.DV * 4, w.cols) && a.DK % 32 == 0;
  St stage;
  Tile<T> vx, dx;
  Tile<float> tx, ox, after[KT];
  if (g.begin < g.end) {
    stage.start(a, first_slot(a, g.n, seq, kC) + g.end - 1, w.hv, w.hk, w.wave, lane, -1);
    stage.fetch();
    if (dalign && g.end * kC <= seq.len) dx.fetch(d0 + (g.end - 1) * kC * line, line * sizeof(T), lane);
    stage.commit(buf);
    __syncthreads();
  }
  for (int64_t c = g.end - 1; c >= g.begin; --c) {
    const int64_t t0 = c * kC, row0 = seq.row + t0, at = t0 * line;
    const int valid = static_cast<int>(min<int64_t>(kC, seq.len - t0));
    const bool whole = valid == kC;
    const f32x16 dout =
        dx.columns(dalign && whole, d0 + at, line * sizeof(T), valid, w.cols, lds, lane);
    if (c > g.begin) {  // what the next chunk wants early
      stage.fetch();
      if (dalign) dx.fetch(d0 + at - kC * int64_t(line), line * sizeof(T), lane);
    }
    const bool ends = !kSpan && ((c & 1) || c == chunks - 1);  // the end of a block of 64 tokens
    const int64_t mark = mark0 + (c >> 1);
    const float* from = c == chunks - 1
                            ? a.ends + state
                            : a.marks + ((mark + 1) * a.H + w.hv) * a.DK * a.DV + 32 * w.tile;
    if (ends && malign) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        if (a.DK > 32 * kt) after[kt].fetch(from + int64_t(32) * kt * a.DV, a.DV * 4u, lane);
    }
    __builtin_amdgcn_sched_barrier(0);  // the loads above go out before the products
    f32x16 ks = {};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> kx;
        get(kx, St::operand(buf, 0, kt, s), lane);
        Wide<T, 3> sw;
        set_wide(sw, part(dS[kt], s));
        ks = mma(kx, sw, ks);
      }
    const float* gate = St::gates(buf);
    const f32x16 gam = load_gate(gate, half), beta = load_gate(gate + 2 * kC, half);
    f32x16 du = load_gate(gate + kC, half) * factor * ks;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> pw;
      Wide<T, 1> dw;  // exact: do is in the data type
      get(pw, St::p(buf, s), lane);
      set_wide(dw, part(dout, s));
      if constexpr (sizeof(T) == 4) {
        du = mma(pw, dw, du);
      } else {
        du = mma(pw, Exact<T>{dw.p[0]}, du);
      }
    }
    settled(du);
    // what this one wants at its end
    if (!kSpan && valign && whole) vx.fetch(v0 + t0 * a.sv.l, vline, lane);
    if (!kSpan && salign && whole) {
      tx.fetch(a.ts + first + at, line * 4, lane);
      ox.fetch(a.os + first + at, line * 4, lane);
    }
    __builtin_amdgcn_sched_barrier(0);
    const f32x16 bu = beta * du;
    f32x16 nr = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> nw, rw;
      get(nw, St::n(buf, s), lane);
      set_wide(rw, part(bu, s));
      nr = mma(nw, rw, nr);
    }
    f32x16 y = du - nr, dv = beta * y;
    settled(y);
    settled(dv);
    if (ends) {
      store_state<float, KT>(dS, a.dmarks + (mark * a.H + w.hv) * a.DK * a.DV + 32 * w.tile, factor, a, w,
                             lds);
      float dot = 0.0f;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        if (a.DK > 32 * kt) {
          const f32x16 S = after[kt].columns(malign, from + int64_t(32) * kt * a.DV, a.DV * 4u,
                                             a.DK - 32 * kt, w.cols, lds, lane);
#pragma unroll
          for (int r = 0; r < 16; ++r) dot = fmaf(dS[kt][r], S[r], dot);
        }
      dot = w.in ? dot * factor : 0.0f;
      dot = lane_sum<64>(dot);
      if (lane == 0 && w.store_cols > 0) a.pdots[(mark * a.H + w.hv) * tiles + w.tile] = dot;
    }
    factor = decay_state<KT>(dS, factor, gate[kC - 1]);
    const f32x16 over = gam * (1.0f / factor);
    const f32x16 gdo = a.scale * over * dout, gdv = -(over * dv);
    Wide<T, 3> ow[2], vw[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      set_wide(ow[s], part(gdo, s));
      set_wide(vw[s], part(gdv, s));
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Exact<T> qx, kx;
        get(qx, St::operand(buf, 2, kt, s), lane);
        get(kx, St::operand(buf, 1, kt, s), lane);
        dS[kt] = mma(qx, ow[s], dS[kt]);
        dS[kt] = mma(kx, vw[s], dS[kt]);
      }
    }
    if constexpr (!kSpan) {
      // dv, and what the gates' gradients take from these 32 columns
      store_tile<T>(dv, out0 + at, line * sizeof(T), oalign && whole, valid, w.store_cols, lds, lane);
      if constexpr (sizeof(T) == 2)
        store_tile<float>(dv, a.dvs + first + at, line * 4, walign && whole, valid, w.store_cols, lds, lane);
      f32x16 sb = y * tx.columns(salign && whole, a.ts + first + at, line * 4, valid, w.cols, lds, lane);
      f32x16 sg = dout * ox.columns(salign && whole, a.os + first + at, line * 4, valid, w.cols, lds, lane) -
                  dv * vx.columns(valign && whole, v0 + t0 * a.sv.l, vline, valid, w.cols, lds, lane);
      if (w.store_cols < 32) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          sb[r] = w.in ? sb[r] : 0.0f;
          sg[r] = w.in ? sg[r] : 0.0f;
        }
      }
      const float beta_sum = sum_columns(sb, lane), gate_sum = sum_columns(sg, lane);
      const int i = acc_row(row_of(lane), half);
      if ((lane & 1) == 0 && i < valid && w.store_cols > 0) {
        const int64_t p = (w.tile * a.T + row0 + i) * a.H + w.hv;
        a.pbeta[p] = beta_sum;
        a.pgate[p] = gate_sum;
      }
    }
    if (c > g.begin) {
      __syncthreads();
      stage.commit(buf);
      __syncthreads();
    }
  }
  if (kSpan) store_state<float, KT>(dS, a.span_z + start, factor, a, w, lds);
  else if (a.dh0 && g.index == 0) store_state<float, KT>(dS, a.dh0 + state, factor, a, w, lds);
}

// dq and dk of one block of 64 tokens and key head, summed over the value heads that share
// it, by eight waves: for the first and second 32 tokens each, one wave for dq, one for dk's
// part from the states and two for dk's part from the block itself (added to the former at
// the end).  The matrices whose columns (DV) are contracted pass through LDS 32 columns at a
// time, split into bfloat16 terms once for all waves, the next 32 already on their way.  For
// bfloat16 data the fp32 operands (u, dv, the states and their gradients, dP and dL) take 2 terms,
// 17 bits: dk is a difference of their products, which with dv and the states' gradients in
// bfloat16 was 1.4 times as far from 64 bits as its own rounding (2.3e-3 against 1.7e-3 without
// decay); a third term would add half as many products again for bits that the results' rounding
// drops.
//
// Bound by the loads' latency: a block is three round trips to memory and little else.  So
// its registers and LDS are held to what lets two blocks share a CU (128 registers up to
// DK = 64 where no value heads share a key head, which needs no second set of sums): six waves
// at 242 registers, one block per CU, loads issued one behind the other: 480 us (64 x 3136
// tokens of 3 heads of 64, dv and the states' gradients then in bfloat16); eight at 128, all loads
// of 32 columns at once: 223 us, and 266 to 274 with those two in fp32 (920 MB).
template <typename T, int KT> struct Panels {  // 32 columns: planes of 32 rows by 16 columns
  // parts of 32 rows by 16 columns: u = beta t, dv, the state and its gradient in 2 terms; do exact
  static constexpr int kWide = 8 + 4 * KT, kNarrow = 4;
  static constexpr int kU = 0;                                   // 64 rows
  static constexpr int kDv = kU + 4 * wide_planes<T, 2>();       // 64 rows
  static constexpr int kS = kDv + 4 * wide_planes<T, 2>();       // DK rows
  static constexpr int kDs = kS + 2 * KT * wide_planes<T, 2>();  // DK rows
  static constexpr int kDo = kDs + 2 * KT * wide_planes<T, 2>(); // 64 rows
  static constexpr int kKeys = kDo + 4 * exact_planes<T>();      // K^T and Q^T of both halves
  static constexpr int kKeyPlanes = 8 * KT * exact_planes<T>();
  static constexpr int kPlanes = kKeys + kKeyPlanes;
};

// A 16- or 32-byte piece of a row, as it comes from memory: 8 values from column c on, of
// which those past the width (and all where !on) are 0 once taken.
template <typename T> struct Piece {
  u32x4 u[sizeof(T) / 2];

  template <bool kAligned>
  __device__ __forceinline__ void load(const T* row, int c, int width) {
    const auto p = global(row);
    if constexpr (kAligned) {
      const auto q = (Global<const u32x4>)(p + (c < width ? c : 0));
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i) u[i] = q[i];
    } else {
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = p[c + i < width ? c + i : 0];
      __builtin_memcpy(u, e, sizeof(e));
    }
  }
  template <bool kAligned>
  __device__ __forceinline__ Piece taken(int c, int width, bool on) const {
    Piece y = *this;
    if constexpr (kAligned) {
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i)
        if (!on || c >= width) y.u[i] = u32x4{0, 0, 0, 0};
    } else {
      T e[8];
      __builtin_memcpy(e, u, sizeof(e));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!on || c + i >= width) e[i] = T(0);
      __builtin_memcpy(y.u, e, sizeof(e));
    }
    return y;
  }
  __device__ __forceinline__ void put(char* at, int lane) const {
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
      reinterpret_cast<u32x4*>(at + i * kPlane)[lane] = u[i];
  }
};

// The block's place and the LDS that its waves share.
struct GradBlock {
  const Args& a;
  char* panels;
  char* spare;   // a tile of each storing wave
  double* G;     // prefix sums of the log decays, of two heads in turn
  int lane, half, own, wave, mine, hk, valid;
  int64_t mark, row0, slot;
};

// One wave's work; kKind: 0 dq, 1 dk's part from the states, 2 dk's part from later outputs of
// the block, 3 dk's part from its other values.  All run the same sequence of barriers.
template <typename T, int KT, bool kAligned, bool kShared, int kKind>
__device__ __forceinline__ void grad_wave(const GradBlock& g) {
  using Pn = Panels<T, KT>;
  constexpr int kNs = (Pn::kNarrow + kGradWaves - 1) / kGradWaves;
  constexpr int kWs = (Pn::kWide + kGradWaves - 1) / kGradWaves;
  constexpr int kKs = (Pn::kKeyPlanes + kGradWaves - 1) / kGradWaves;
  constexpr int kW2 = wide_planes<T, 2>() * kPlane, kEx = exact_planes<T>() * kPlane;
  constexpr int64_t operand = KeyRecord<T, KT>::kOperand * kPlane;
  const Args& a = g.a;
  const int lane = g.lane, half = g.half, own = g.own, mine = g.mine, valid = g.valid;
  char* const panels = g.panels;
  const int64_t line = int64_t(a.H) * a.DV;

  f32x16 total[KT];  // over the key head's value heads
  if constexpr (kShared)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) total[kt] = f32x16{};

  const int rep = kShared ? a.rep : 1;
  for (int hv = g.hk * rep; hv < (g.hk + 1) * rep; ++hv) {
    const bool first = hv == g.hk * rep;
    double* const G = g.G + (hv & 1) * kMark;
    const int64_t head_at = g.row0 * line + int64_t(hv) * a.DV;
    const int64_t state_at = (g.mark * a.H + hv) * a.DK * a.DV;
    float gate = 0.0f;
    if (g.wave == kGradWaves - 1) gate = a.g[(g.row0 + (lane < valid ? lane : 0)) * a.H + hv];

    // This wave's parts of the next 32 columns: two lanes per row.  The loads depend on nothing
    // but addresses, so that all are on their way at once; what is out of range is left out
    // when the parts are written to LDS.
    Piece<T> narrow[kNs];
    Piece<float> wide[kWs];
    float beta[kWs];
    const int prow = lane >> 1, pcol = 8 * (lane & 1), to = 32 * (lane & 1) + swap23(prow);
    auto row_of_part = [&](int part) {  // of a wide one: u, dv, the state, its gradient
      return 32 * ((part < 8 ? part & 3 : part < 8 + 2 * KT ? part - 8 : part - 8 - 2 * KT) >> 1) + prow;
    };
    auto fetch = [&](int c0) {
#pragma unroll
      for (int i = 0; i < kWs; ++i) {
        const int part = min(g.wave + kGradWaves * i, Pn::kWide - 1);
        const bool tokens = part < 8;
        const int row = row_of_part(part);
        const int at = row < (tokens ? valid : a.DK) ? row : 0;
        const float* base = tokens ? (part < 4 ? a.ts : a.dvs) + head_at
                                   : (part < 8 + 2 * KT ? a.marks : a.dmarks) + state_at;
        wide[i].template load<kAligned>(base + at * (tokens ? line : a.DV), c0 + 16 * (part & 1) + pcol, a.DV);
        beta[i] = a.beta[(g.row0 + (tokens ? at : 0)) * a.H + hv];
      }
#pragma unroll
      for (int i = 0; i < kNs; ++i) {
        const int part = min(g.wave + kGradWaves * i, Pn::kNarrow - 1);
        const int row = 32 * (part >> 1) + prow, at = row < valid ? row : 0;
        narrow[i].template load<kAligned>(static_cast<const T*>(a.dout) + head_at + at * line,
                                          c0 + 16 * (part & 1) + pcol, a.DV);
      }
    };
    auto commit = [&](int c0) {
#pragma unroll
      for (int i = 0; i < kWs; ++i) {
        const int part = g.wave + kGradWaves * i;
        if (part >= Pn::kWide) break;
        const Piece<float> x = wide[i].template taken<kAligned>(c0 + 16 * (part & 1) + pcol, a.DV,
                                                                row_of_part(part) < (part < 8 ? valid : a.DK));
        f32x8 v;
        __builtin_memcpy(&v, x.u, 32);
        Wide<T, 2> w;
        set_wide(w, part < 4 ? v * beta[i] : v);
        put(panels + (Pn::kU + part * wide_planes<T, 2>()) * kPlane, to, w);
      }
#pragma unroll
      for (int i = 0; i < kNs; ++i) {
        const int part = g.wave + kGradWaves * i;
        if (part >= Pn::kNarrow) break;
        narrow[i].template taken<kAligned>(c0 + 16 * (part & 1) + pcol, a.DV, 32 * (part >> 1) + prow < valid)
            .put(panels + (Pn::kDo + part * exact_planes<T>()) * kPlane, to);
      }
    };
    fetch(0);
    if (first) {  // K^T and Q^T of the block's two chunks, for all heads
      constexpr int kHalf = Pn::kKeyPlanes / 2;
      u32x4 keys[kKs];
#pragma unroll
      for (int i = 0; i < kKs; ++i) {
        const int p = min(g.wave + kGradWaves * i, Pn::kKeyPlanes - 1), o = p >= kHalf && 32 < valid;
        const char* record = a.keys + ((g.slot + o) * a.HK + g.hk) *
                                          (int64_t(KeyRecord<T, KT>::kPlanes) * kPlane) + operand;
        keys[i] = *(Global<const u32x4>)(global(record) + p % kHalf * kPlane + 16u * lane);
      }
#pragma unroll
      for (int i = 0; i < kKs; ++i) {
        const int p = g.wave + kGradWaves * i;
        if (p < Pn::kKeyPlanes)
          *reinterpret_cast<u32x4*>(panels + (Pn::kKeys + p) * kPlane + 16 * lane) = keys[i];
      }
    }
    if (g.wave == kGradWaves - 1) {  // read after the barriers below
      double x = lane < valid ? bounded_log(gate) * kLog2eWide : 0.0;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double up = __shfl_up(x, d);
        if (lane >= d) x += up;
      }
      G[lane] = x;
    }
    // kind 0: y = do S^T, p[o] = u_o . do;  kind 1: y = u dS^T and dv S^T;  kind 2: p[o] = do_o . u;
    // kind 3: p[o] = u_o . dv (earlier tokens o) or dv_o . u (later ones): o runs over the block's
    // halves in registers' rows, the lanes hold this wave's tokens; q is p of the other sense
    // within this wave's 32 tokens
    constexpr int kY = kKind == 0 ? KT : (kKind == 1 ? 2 * KT : 1);
    f32x16 y[kY], p[2], q = {};
#pragma unroll
    for (int kt = 0; kt < kY; ++kt) y[kt] = f32x16{};
    p[0] = p[1] = f32x16{};
    for (int c0 = 0; c0 < a.DV; c0 += 32) {
      commit(c0);
      __syncthreads();
      if (c0 + 32 < a.DV) fetch(c0 + 32);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        auto wide_of = [&](int first_plane, int o) {
          Wide<T, 2> w;
          get(w, panels + first_plane * kPlane + (2 * o + s) * kW2, lane);
          return w;
        };
        auto exact_of = [&](int first_plane, int o) {
          Exact<T> w;
          get(w, panels + first_plane * kPlane + (2 * o + s) * kEx, lane);
          return w;
        };
        if constexpr (kKind == 0) {
          const Exact<T> d = exact_of(Pn::kDo, mine);
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) y[kt] = mma(d, wide_of(Pn::kS, kt), y[kt]);
          p[0] = mma(wide_of(Pn::kU, 0), d, p[0]);
          if (mine == 1) p[1] = mma(wide_of(Pn::kU, 1), d, p[1]);
        } else if constexpr (kKind == 1) {
          const Wide<T, 2> d = wide_of(Pn::kDv, mine), u = wide_of(Pn::kU, mine);
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            y[KT + kt] = mma(d, wide_of(Pn::kS, kt), y[KT + kt]);
            y[kt] = mma(u, wide_of(Pn::kDs, kt), y[kt]);
          }
        } else if constexpr (kKind == 2) {
          const Wide<T, 2> u = wide_of(Pn::kU, mine);
          p[0] = mma(exact_of(Pn::kDo, 0), u, p[0]);  // not used by the later 32 tokens
          p[1] = mma(exact_of(Pn::kDo, 1), u, p[1]);
        } else {
          const Wide<T, 2> u = wide_of(Pn::kU, mine), d = wide_of(Pn::kDv, mine);
          if (mine == 0) {
            p[0] = mma(u, d, p[0]);
            p[1] = mma(wide_of(Pn::kDv, 1), u, p[1]);
          } else {
            p[0] = mma(wide_of(Pn::kU, 0), d, p[0]);
            p[1] = mma(u, d, p[1]);
          }
          q = mma(d, u, q);
        }
      }
      drained();
      __syncthreads();
    }
    if constexpr (!kShared)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) total[kt] = f32x16{};
    if (32 * mine >= valid) continue;
    const int row = 32 * mine + own;
    const double Gown = G[row], Gend = G[kMark - 1];
    if constexpr (kKind < 2) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const double at = G[32 * mine + acc_row(r, half)];
        const float in = decay_of(at), out = decay_of(Gend - at);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          if constexpr (kKind == 0) total[kt][r] += a.scale * in * y[kt][r];
          else total[kt][r] += out * y[kt][r] - in * y[KT + kt][r];
        }
      }
    }
    if constexpr (kKind != 1) {
      constexpr int kHalf = Pn::kKeyPlanes / 2;
#pragma unroll
      for (int other = 0; other < 2; ++other) {
        if (32 * other >= valid) break;
        if ((kKind == 0 && other > mine) || (kKind == 2 && other < mine)) continue;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int o = 32 * other + acc_row(r, half);
          const double at = G[o];
          const float f = decay_of(o <= row ? Gown - at : at - Gown);
          if constexpr (kKind == 0) p[other][r] = o <= row ? a.scale * f * p[other][r] : 0.0f;
          else if constexpr (kKind == 2) p[other][r] = o >= row ? a.scale * f * p[other][r] : 0.0f;
          else p[other][r] = o == row ? 0.0f : -f * (other == mine && o > row ? q[r] : p[other][r]);
        }
        const char* keys = panels + (Pn::kKeys + other * kHalf) * kPlane + (kKind == 2 ? operand : 0);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Wide<T, 2> pw;
          set_wide(pw, part(p[other], s));
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            Exact<T> x;
            get(x, keys + (2 * kt + s) * kEx, lane);
            total[kt] = mma(pw, x, total[kt]);
          }
        }
        drained();
      }
    }
  }
  // the last readers of the panels' first part are past the loop's barrier
  float* const sums = reinterpret_cast<float*>(panels) + mine * KT * 16 * 64 + lane;
  static_assert(2 * KT * 16 * 64 * 4 <= Pn::kKeys * kPlane, "the sums take the panels' place");
  if constexpr (kKind == 2)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) sums[(16 * kt + r) * 64] = total[kt][r];
  __syncthreads();
  if constexpr (kKind == 3)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r) sums[(16 * kt + r) * 64] += total[kt][r];
  __syncthreads();
  if (kKind > 1 || 32 * mine >= valid) return;
  T* out = static_cast<T*>(kKind ? a.dk : a.dq) +
           ((g.row0 + 32 * mine) * a.HK + g.hk) * int64_t(a.DK);
  const uint32_t stride = a.HK * a.DK * sizeof(T);
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    if constexpr (kKind == 1)
#pragma unroll
      for (int r = 0; r < 16; ++r) total[kt][r] += sums[(16 * kt + r) * 64];
    const int rows = valid - 32 * mine, cols = min(32, a.DK - 32 * kt);
    if (cols > 0)
      store_tile<T>(total[kt], out + 32 * kt, stride,
                    aligned16(out + 32 * kt, stride, cols) && rows >= 32, rows, cols,
                    g.spare + g.wave * kTileBytes, lane, own);
  }
}

template <typename T, int KT, bool kAligned, bool kShared>
__global__ __launch_bounds__(64 * kGradWaves)
__attribute__((amdgpu_waves_per_eu(KT * sizeof(T) <= 4 && !kShared ? 4 : 2)))
void k_delta_grads(Args a) {
  __shared__ __align__(16) char panels[Panels<T, KT>::kPlanes * kPlane];
  __shared__ __align__(16) char spare[4 * kTileBytes];
  __shared__ double G[2 * kMark];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t mark = blockIdx.x / a.HK;
  int64_t n, b;
  Seq seq;
  if (!find_slot(a, mark, kMark, &n, &b, &seq)) return;
  const GradBlock g{a, panels, spare, G, lane, lane >> 5, swap23(lane & 31), wave, wave & 1,
                    static_cast<int>(blockIdx.x - mark * a.HK),
                    static_cast<int>(min<int64_t>(kMark, seq.len - b * kMark)), mark,
                    seq.row + b * kMark, first_slot(a, n, seq, kC) + 2 * b};
  if (wave < 2) grad_wave<T, KT, kAligned, kShared, 0>(g);
  else if (wave < 4) grad_wave<T, KT, kAligned, kShared, 1>(g);
  else if (wave < 6) grad_wave<T, KT, kAligned, kShared, 2>(g);
  else grad_wave<T, KT, kAligned, kShared, 3>(g);
}

// dbeta and dg of one block of 64 tokens and head: sums over the column tiles, then the sum
// over the tokens from each one on.
__global__ __launch_bounds__(256) void k_delta_gate_grads(Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t mark = unit / a.H;
  const int hv = static_cast<int>(unit - mark * a.H);
  if (mark >= a.marks_n) return;
  int64_t n, b;
  Seq seq;
  if (!find_slot(a, mark, kMark, &n, &b, &seq)) return;
  const int tiles = (a.DV + 31) / 32;
  const int64_t t0 = b * kMark;
  const bool on = lane < seq.len - t0;
  const int64_t row = seq.row + t0 + lane;
  double dg = 0.0, db = 0.0, dot = 0.0;
  for (int i = 0; i < tiles; ++i) {
    if (on) {
      db += a.pbeta[(i * a.T + row) * a.H + hv];
      dg += a.pgate[(i * a.T + row) * a.H + hv];
    }
    dot += a.pdots[(mark * a.H + hv) * tiles + i];
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double down = __shfl_down(dg, d);
    if (lane + d < 64) dg += down;
  }
  if (!on) return;
  const int64_t at = row * a.H + hv;
  a.dbeta[at] = static_cast<float>(db);
  a.dg[at] = a.g[at] < kMinLog ? 0.0f : static_cast<float>(dg + dot);
}

template <typename T, int KT, int kW>
int adjoint_w(const Args& a, bool span, hipStream_t st) {
  const int64_t units = a.seglen > 0 ? a.seg_slots : a.S;
  const int64_t blocks = units * a.H * (((a.DV + 31) / 32 + kW - 1) / kW);
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * kW);
  if (span) hipLaunchKernelGGL((k_delta_adjoint<T, KT, kW, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_adjoint<T, KT, kW, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}
template <typename T, int KT>
int adjoint_kt(const Args& a, bool span, hipStream_t st) {
  if (a.DV <= 32) return adjoint_w<T, KT, 1>(a, span, st);
  if (a.DV <= 64) return adjoint_w<T, KT, 2>(a, span, st);
  return adjoint_w<T, KT, 4>(a, span, st);
}
template <typename T, int KT, bool kAligned>
int grads_kt(const Args& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.marks_n * a.HK)), block(64 * kGradWaves);
  if (a.rep > 1) hipLaunchKernelGGL((k_delta_grads<T, KT, kAligned, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_grads<T, KT, kAligned, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int adjoint_t(const Args& a, bool span, hipStream_t st) {
  if (a.DK <= 32) return adjoint_kt<T, 1>(a, span, st);
  if (a.DK <= 64) return adjoint_kt<T, 2>(a, span, st);
  return adjoint_kt<T, 4>(a, span, st);
}
template <typename T, bool kAligned>
int grads_t(const Args& a, hipStream_t st) {
  if (a.DK <= 32) return grads_kt<T, 1, kAligned>(a, st);
  if (a.DK <= 64) return grads_kt<T, 2, kAligned>(a, st);
  return grads_kt<T, 4, kAligned>(a, st);
}

}  // namespace

int launch_adjoint(const Args& a, int dtype, bool span, hipStream_t st) {
  return dtype == 0 ? adjoint_t<float>(a, span, st) : adjoint_t<uint16_t>(a, span, st);
}
int launch_grads(const Args& a, int dtype, bool aligned, hipStream_t st) {
  if (dtype == 0) return aligned ? grads_t<float, true>(a, st) : grads_t<float, false>(a, st);
  return aligned ? grads_t<uint16_t, true>(a, st) : grads_t<uint16_t, false>(a, st);
}
int launch_gate_grads(const Args& a, hipStream_t st) {
  const int64_t waves = a.marks_n * a.H;
  hipLaunchKernelGGL(k_delta_gate_grads, dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0,
                     st, a);
  return static_cast<int>(hipGetLastError());
}

}  // namespace delta
}  // namespace ss2d
