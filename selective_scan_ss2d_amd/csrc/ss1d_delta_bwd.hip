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
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

// Sums each register over the 32 lanes of a half: lane l of the half gets the sum of
// register row_of(l) (each twice).  Halving the registers at every exchange costs 16
// exchanges for 16 sums.
template <int kN> __device__ __forceinline__ void halve(float* x, int lane) {
  const bool up = lane & (2 * kN);
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float keep = up ? x[kN + i] : x[i], send = up ? x[i] : x[kN + i];
    x[i] = keep + __shfl_xor(send, 2 * kN);
  }
  if constexpr (kN > 1) halve<kN / 2>(x, lane);
}
__device__ __forceinline__ float sum_columns(const f32x16& v, int lane) {
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = v[i];
  halve<8>(x, lane);
  return x[0] + __shfl_xor(x[0], 1);
}
__device__ __forceinline__ int row_of(int lane) { return (lane & 31) >> 1; }

// One wave per (sequence, head, 32 columns), kW adjacent ones per block sharing the chunks'
// operands through LDS, chunks last to first.
template <typename T, int KT, int kW>
__global__ __launch_bounds__(64 * kW) void k_delta_adjoint(Args a) {
  using St = Stage<T, KT, 3, kW>;
  __shared__ __align__(16) char buffers[2][St::kPlanes * kPlane];
  __shared__ __align__(16) char spare[kW][kTileBytes];
  const Place w = place<kW>(a, blockIdx.x);
  const int lane = w.lane, half = w.half, tiles = (a.DV + 31) / 32;
  char* const lds = spare[w.wave];
  const Seq seq = sequence(a, w.n);
  const int64_t slot0 = first_slot(a, w.n, seq, kC), mark0 = first_slot(a, w.n, seq, kMark);
  const int64_t state = w.head * a.DK * a.DV + 32 * w.tile;
  const uint32_t vline = static_cast<uint32_t>(a.sv.l) * sizeof(T), line = a.H * a.DV;

  f32x16 dS[KT];
  load_state<KT>(dS, a.dht ? a.dht + state : nullptr, a, w, lds);
  float factor = 1.0f;
  const int64_t chunks = (seq.len + kC - 1) / kC;
  const int64_t first = seq.row * line + w.hv * a.DV + 32 * w.tile;
  const T* v0 = static_cast<const T*>(a.v) + token_at(a, a.sv, w.n, seq, 0) + w.hv * a.sv.h + 32 * w.tile;
  const T* d0 = static_cast<const T*>(a.dout) + first;
  T* out0 = static_cast<T*>(a.dv) + first;
  const bool valign = aligned16(v0, vline, w.cols), dalign = aligned16(d0, line * sizeof(T), w.cols);
  const bool oalign = aligned16(out0, line * sizeof(T), w.store_cols);
  const bool salign = aligned16(nullptr, line * 4, w.cols);
  const bool malign = aligned16(nullptr, a.DV * 4, w.cols) && a.DK % 32 == 0;
  St stage;
  Tile<T> vx, dx;
  Tile<float> tx, ox, after[KT];
  if (chunks > 0) {
    stage.start(a, slot0 + chunks - 1, w.hv, w.hk, w.wave, lane, -1);
    stage.fetch();
    if (dalign && seq.len % kC == 0) dx.fetch(d0 + (chunks - 1) * kC * line, line * sizeof(T), lane);
    stage.commit(buffers[(chunks - 1) & 1]);
    __syncthreads();
  }
  for (int64_t c = chunks - 1; c >= 0; --c) {
    const int64_t t0 = c * kC, row0 = seq.row + t0, at = t0 * line;
    const int valid = static_cast<int>(min<int64_t>(kC, seq.len - t0));
    const bool whole = valid == kC;
    const char* buf = buffers[c & 1];
    const f32x16 dout =
        dx.columns(dalign && whole, d0 + at, line * sizeof(T), valid, w.cols, lds, lane);
    if (c > 0) {  // what the next chunk wants early
      stage.fetch();
      if (dalign) dx.fetch(d0 + at - kC * int64_t(line), line * sizeof(T), lane);
    }
    // what this one wants at its end
    if (valign && whole) vx.fetch(v0 + t0 * a.sv.l, vline, lane);
    if (salign && whole) {
      tx.fetch(a.ts + first + at, line * 4, lane);
      ox.fetch(a.os + first + at, line * 4, lane);
    }
    const bool ends = (c & 1) || c == chunks - 1;  // the end of a block of 64 tokens
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
    const f32x16 bu = beta * du;
    f32x16 nr = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> nw, rw;
      get(nw, St::n(buf, s), lane);
      set_wide(rw, part(bu, s));
      nr = mma(nw, rw, nr);
    }
    const f32x16 y = du - nr, dv = beta * y;
    if (ends) {
      store_state<T, KT>(dS, static_cast<T*>(a.dmarks) + (mark * a.H + w.hv) * a.DK * a.DV + 32 * w.tile,
                         factor, a, w, lds);
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
#pragma unroll
      for (int d = 1; d < 64; d *= 2) dot += __shfl_xor(dot, d);
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
    // dv, and what the gates' gradients take from these 32 columns
    store_tile<T>(dv, out0 + at, line * sizeof(T), oalign && whole, valid, w.store_cols, lds, lane);
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
    if (c > 0) stage.commit(buffers[(c - 1) & 1]);
    __syncthreads();
  }
  if (a.dh0) store_state<float, KT>(dS, a.dh0 + state, factor, a, w, lds);
}

// dq and dk of one block of 64 tokens and key head, summed over the value heads that share
// it: four waves, one for each of (dq, dk) x (first, second 32 tokens).  For bfloat16 data
// one operand of every product has 2 terms (or is exact), so each product carries at most
// one operand rounding besides the output's own.
template <typename T, int KT, bool kAligned>
__global__ __launch_bounds__(256) void k_delta_grads(Args a) {
  __shared__ double G[kMark];
  const int lane = threadIdx.x & 63, half = lane >> 5, own = swap23(lane & 31);
  const int wave = threadIdx.x >> 6, mine = wave & 1;  // this wave's 32 tokens
  const bool keys = wave >> 1;
  const int64_t mark = blockIdx.x / a.HK;
  const int hk = static_cast<int>(blockIdx.x - mark * a.HK);
  int64_t n, b;
  Seq seq;
  if (!find_slot(a, mark, kMark, &n, &b, &seq)) return;
  const int64_t t0 = b * kMark, row0 = seq.row + t0;
  const int valid = static_cast<int>(min<int64_t>(kMark, seq.len - t0));
  const int64_t slot = first_slot(a, n, seq, kC) + 2 * b;  // of the first 32 tokens
  const int64_t line = int64_t(a.H) * a.DV;
  constexpr int64_t frag = exact_planes<T>() * kPlane;
  constexpr int64_t operand = KeyRecord<T, KT>::kOperand * kPlane;
  const bool live = 32 * mine < valid;

  f32x16 total[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) total[kt] = f32x16{};

  for (int hv = hk * a.rep; hv < (hk + 1) * a.rep; ++hv) {
    __syncthreads();
    if (wave == 0) {
      double x = lane < valid ? fmaxf(a.g[(row0 + lane) * a.H + hv], kMinLog) : 0.0;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const double up = __shfl_up(x, d);
        if (lane >= d) x += up;
      }
      G[lane] = x;
    }
    __syncthreads();
    if (!live) continue;
    const int64_t head_at = row0 * line + int64_t(hv) * a.DV;
    const T* dout = static_cast<const T*>(a.dout) + head_at;
    const T* dv = static_cast<const T*>(a.dv) + head_at;
    const float* ts = a.ts + head_at;
    const float* S = a.marks + (mark * a.H + hv) * a.DK * a.DV;
    const T* dS = static_cast<const T*>(a.dmarks) + (mark * a.H + hv) * a.DK * a.DV;
    const int row = 32 * mine + own;             // this lane's token as a row of its tile
    const bool on = row < valid;
    const int64_t at = int64_t(on ? row : 0) * line;
    const float beta_own = on ? a.beta[(row0 + row) * a.H + hv] : 0.0f;
    const double Gown = G[row], Gend = G[kMark - 1];

    // the states' part: rows of this wave's tokens against the states' rows
    f32x16 x[KT], y[KT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) x[kt] = y[kt] = f32x16{};
    for (int c = 0; c < a.DV; c += 16) {
      const int c8 = c + 8 * half;
      if (!keys) {
        Exact<T> d;
        load8<kAligned>(d, dout + at, c8, a.DV, on);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const int k = 32 * kt + own;
          Exact<float> s;
          load8<kAligned>(s, S + int64_t(k < a.DK ? k : 0) * a.DV, c8, a.DV, k < a.DK);
          Wide<T, 2> w;
          set_wide(w, s.v);
          x[kt] = mma(d, w, x[kt]);
        }
      } else {
        Exact<T> d;
        load8<kAligned>(d, dv + at, c8, a.DV, on);
        Exact<float> t;
        load8<kAligned>(t, ts + at, c8, a.DV, on);
        Wide<T, 2> u;
        set_wide(u, t.v * beta_own);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const int k = 32 * kt + own;
          const int64_t r = int64_t(k < a.DK ? k : 0) * a.DV;
          Exact<float> s;
          load8<kAligned>(s, S + r, c8, a.DV, k < a.DK);
          Wide<T, 2> w;
          set_wide(w, s.v);
          y[kt] = mma(d, w, y[kt]);
          Exact<T> g;
          load8<kAligned>(g, dS + r, c8, a.DV, k < a.DK);
          x[kt] = mma(u, g, x[kt]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const double g = G[32 * mine + acc_row(r, half)];
      const float in = expf(static_cast<float>(g)), out = expf(static_cast<float>(Gend - g));
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
        total[kt][r] += keys ? out * x[kt][r] - in * y[kt][r] : a.scale * in * x[kt][r];
    }
    // the block's own part: 32 x 32 tiles with the other tokens in registers' rows and this
    // wave's tokens in lanes, which are left operands as they stand
    for (int other = 0; other < 2; ++other) {
      if (32 * other >= valid) break;
      const bool causal = keys ? other >= mine : other <= mine;
      if (!keys && !causal) continue;
      const int row2 = 32 * other + own;
      const bool on2 = row2 < valid;
      const int64_t at2 = int64_t(on2 ? row2 : 0) * line;
      const float beta2 = on2 ? a.beta[(row0 + row2) * a.H + hv] : 0.0f;
      f32x16 p = {}, l1 = {}, l2 = {};
      for (int c = 0; c < a.DV; c += 16) {
        const int c8 = c + 8 * half;
        Exact<float> t, t2;
        Wide<T, 2> u, u2;
        load8<kAligned>(t, ts + at, c8, a.DV, on);
        load8<kAligned>(t2, ts + at2, c8, a.DV, on2);
        set_wide(u, t.v * beta_own);
        set_wide(u2, t2.v * beta2);
        Exact<T> d;
        if (!keys) {  // u_j . do_i, tokens i in lanes
          load8<kAligned>(d, dout + at, c8, a.DV, on);
          p = mma(u2, d, p);
        } else {
          if (causal) {  // do_i . u_j, tokens j in lanes
            load8<kAligned>(d, dout + at2, c8, a.DV, on2);
            p = mma(d, u, p);
          }
          if (other <= mine) {  // u . dv of this wave's tokens: the later ones
            load8<kAligned>(d, dv + at, c8, a.DV, on);
            l1 = mma(u2, d, l1);
          }
          if (other >= mine) {
            load8<kAligned>(d, dv + at2, c8, a.DV, on2);
            l2 = mma(d, u, l2);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int o = 32 * other + acc_row(r, half);
        const float f = expf(static_cast<float>(o <= row ? Gown - G[o] : G[o] - Gown));
        if (!keys) {
          p[r] = o <= row ? a.scale * f * p[r] : 0.0f;
        } else {
          p[r] = o >= row ? a.scale * f * p[r] : 0.0f;
          l1[r] = o < row ? -f * l1[r] : (o > row ? -f * l2[r] : 0.0f);
        }
      }
      const char* record = a.keys + ((slot + other) * a.HK + hk) *
                                        (int64_t(KeyRecord<T, KT>::kPlanes) * kPlane);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Wide<T, 2> pw, lw;
        set_wide(pw, part(p, s));
        if (keys) set_wide(lw, part(l1, s));
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const char* f = record + operand + (2 * kt + s) * frag;
          Exact<T> kx;
          get(kx, f, lane);
          if (!keys) {
            total[kt] = mma(pw, kx, total[kt]);
          } else {
            total[kt] = mma(lw, kx, total[kt]);
            if (causal) {
              Exact<T> qx;
              get(qx, f + operand, lane);
              total[kt] = mma(pw, qx, total[kt]);
            }
          }
        }
      }
    }
  }
  if (!live) return;
  T* out = static_cast<T*>(keys ? a.dk : a.dq);
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int i = 32 * mine + acc_row(r, half), k = 32 * kt + own;
      if (i < valid && k < a.DK)
        out[((row0 + i) * a.HK + hk) * a.DK + k] = Elem<T>::from_f32(total[kt][r]);
    }
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
int adjoint_w(const Args& a, hipStream_t st) {
  const int64_t blocks = a.S * a.H * (((a.DV + 31) / 32 + kW - 1) / kW);
  hipLaunchKernelGGL((k_delta_adjoint<T, KT, kW>), dim3(static_cast<unsigned>(blocks)), dim3(64 * kW),
                     0, st, a);
  return static_cast<int>(hipGetLastError());
}
template <typename T, int KT>
int adjoint_kt(const Args& a, hipStream_t st) {
  if (a.DV <= 32) return adjoint_w<T, KT, 1>(a, st);
  if (a.DV <= 64) return adjoint_w<T, KT, 2>(a, st);
  return adjoint_w<T, KT, 4>(a, st);
}
template <typename T, int KT, bool kAligned>
int grads_kt(const Args& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.marks_n * a.HK)), block(256);
  hipLaunchKernelGGL((k_delta_grads<T, KT, kAligned>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int adjoint_t(const Args& a, hipStream_t st) {
  if (a.DK <= 32) return adjoint_kt<T, 1>(a, st);
  if (a.DK <= 64) return adjoint_kt<T, 2>(a, st);
  return adjoint_kt<T, 4>(a, st);
}
template <typename T, bool kAligned>
int grads_t(const Args& a, hipStream_t st) {
  if (a.DK <= 32) return grads_kt<T, 1, kAligned>(a, st);
  if (a.DK <= 64) return grads_kt<T, 2, kAligned>(a, st);
  return grads_kt<T, 4, kAligned>(a, st);
}

}  // namespace

int launch_adjoint(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? adjoint_t<float>(a, st) : adjoint_t<uint16_t>(a, st);
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
