// The sequential pass of the gated delta rule's forward: one wave carries 32 columns of one
// sequence and head's state through its chunks, the state in registers, the chunk's operands
// in LDS, where the block's waves (adjacent columns) share them, loaded a chunk ahead.  32
// columns are one 32 x 32 matrix tile.  Each of a chunk's products needs the one before it, so
// the pass is bound by the latency of that chain (S^T k, the solve, the update): 3.7 us a chunk
// for a 64-row state in bfloat16 with everything saved (64 x 3136 tokens of 3 heads of 64: 365
// us), 4.9 us for a 128-row one, the matrix cores busy for less than half of it.  Two waves per
// SIMD hide part of it; a second LDS buffer for the operands saved one barrier a chunk but cost
// the second block of a CU.
//
// With few sequences and heads the chunks' chain leaves most of the chip idle.  Then the
// sequences are cut into segments: what a segment makes of the state before it is affine,
// S -> M S + Z, and the span pass computes M (from the identity's columns, no v) and Z (from
// zero) of all segments at once with the same recurrence, the join pass runs S through them,
// and the forward then starts every segment from its state.  4096 tokens of 32 heads of 128 in
// 8 segments: span 86 us, join 27, run 78; 2 x 65536 fp32 tokens of 3 heads of 64 in 86
// segments: span 156, join 134 (1.5 us a segment, one after the other), run 224, and with the
// chunk matrices 604 in all, where the uncut call took 10.5 ms.
#include "ss1d_delta.h"

namespace ss2d {
namespace delta {
namespace {

// A product over the chunk's tokens multiplies by the structural zeros of N and P too, where a NaN
// or an infinity would reach the tokens before it.  So its operand is clamped to the largest value
// that its terms hold (NaN becomes the lowest); the state's update takes the values as they are, all
// rows of its column follow them, and where they have, o is set to NaN from the first such token on.
template <typename T> constexpr float kLargest = sizeof(T) == 4 ? 0x1.fffffep127f : 0x1.fep127f;
template <typename T> __device__ __forceinline__ f32x16 clamped(const f32x16& x) {
  f32x16 y;
#pragma unroll
  for (int r = 0; r < 16; ++r) y[r] = __builtin_amdgcn_fmed3f(x[r], -kLargest<T>, kLargest<T>);
  return y;
}
// That token, kC without one, and the column with NaN from token `from` on.
template <typename T> __device__ __forceinline__ int first_bad(const f32x16& x, int half) {
  int token = kC;
#pragma unroll
  for (int r = 15; r >= 0; --r)
    if (!(fabsf(x[r]) <= kLargest<T>)) token = acc_row(r, half);
  return min(token, __shfl_xor(token, 32));
}
__device__ __forceinline__ void set_nan(f32x16& x, int from, int half) {
#pragma unroll
  for (int r = 0; r < 16; ++r) x[r] = acc_row(r, half) >= from ? __builtin_nanf("") : x[r];
}

// Operands hold 24 bits (3 bf16 terms), those of o 17 (2 terms, which leaves o to its own
// rounding); with kSave, the training forward, o's hold 24 as well, because the backward
// forms the decays' gradient from o.  kSpan: the span pass, no o; the tiles are those of Z,
// then those of M.
enum Mode { kForward, kSaving, kSpanning };
template <typename T, int KT, int kW, Mode kMode>
__global__ __launch_bounds__(64 * kW)
__attribute__((amdgpu_waves_per_eu(kMode == kSaving && KT == 4 ? 1 : 2))) void k_delta_scan(Args a) {
  constexpr bool kSave = kMode == kSaving, kSpan = kMode == kSpanning;
  constexpr int kP = kSave ? 3 : 2;
  using St = Stage<T, KT, kP, kW, kSpan>;
  __shared__ __align__(16) char buf[St::kPlanes * kPlane];
  __shared__ __align__(16) char spare[kW][kTileBytes];
  Place w;
  // the span pass counts whole tiles: DV's first, then DK's
  const int vtiles = (a.DV + 31) / 32;
  if (!place<kW>(&w, a, blockIdx.x, kSpan ? 32 * (vtiles + KT) : a.DV)) return;
  const Segment& g = w.g;
  // nothing starts from the last segment's end; the backward takes its M all the same
  if (kSpan && (g.end == g.begin || (g.last && a.marks == nullptr))) return;
  const bool matrix = kSpan && w.tile >= vtiles;
  if (kSpan) {
    w.cols = matrix ? max(0, min(32, a.DK - 32 * (w.tile - vtiles))) : min(32, a.DV - 32 * w.tile);
    w.store_cols = min(w.cols, w.store_cols);
    w.in = (w.lane & 31) < w.store_cols;
  }
  const int lane = w.lane, half = w.half;
  char* const lds = spare[w.wave];
  const Seq& seq = g.seq;
  const int64_t state = w.head * a.DK * a.DV + 32 * w.tile;
  const int64_t start = (g.slot * a.H + w.hv) * a.DK * a.DV + 32 * w.tile;
  const int64_t chunks = g.end, t0 = g.begin * kC;

  f32x16 S[KT];
  if constexpr (kSpan) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        S[kt][r] = matrix && 32 * kt + acc_row(r, half) == 32 * (w.tile - vtiles) + (lane & 31) ? 1.0f : 0.0f;
  } else {
    // a sequence of several segments starts from the join's copy of h0: its last segment, another
    // wave, may write the end state over h0 itself
    const bool copied = g.index > 0 || !g.last;
    load_state<KT>(S, a.h0 == nullptr && g.index == 0 ? nullptr : (copied ? a.starts + start : a.h0 + state),
                   a, w, lds);
  }
  float factor = 1.0f;

  const int64_t first = (seq.row + t0) * a.H * a.DV + w.hv * a.DV + 32 * w.tile;
  const uint32_t vline = static_cast<uint32_t>(a.sv.l) * sizeof(T), line = a.H * a.DV;
  const T* vat = static_cast<const T*>(a.v) + token_at(a, a.sv, g.n, seq, t0) + w.hv * a.sv.h + 32 * w.tile;
  T* oat = static_cast<T*>(a.o) + first;
  const bool valign = !matrix && aligned16(vat, vline, w.cols);
  const bool oalign = aligned16(oat, line * sizeof(T), w.store_cols);
  const bool salign = aligned16(nullptr, line * 4, w.store_cols);
  float* tat = kSave ? a.ts + first : nullptr;
  float* pat = kSave ? a.os + first : nullptr;
  float* mat = kSave ? a.marks + ((first_slot(a, g.n, seq, kMark) + g.begin / 2) * a.H + w.hv) * a.DK * a.DV +
                           32 * w.tile
                     : nullptr;
  int left = static_cast<int>(min<int64_t>(seq.len - t0, 1 << 30));  // tokens from this chunk on

  St stage;
  Tile<T> vx;
  if (g.begin < g.end) {
    stage.start(a, first_slot(a, g.n, seq, kC) + g.begin, w.hv, w.hk, w.wave, lane, 1);
    stage.fetch();
    if (valign && left >= kC) vx.fetch(vat, vline, lane);
    stage.commit(buf);
    __syncthreads();
  }
  for (int64_t c = g.begin; c < chunks; ++c) {
    left = static_cast<int>(min<int64_t>(seq.len - c * kC, 1 << 30));
    const bool whole = left >= kC;
    f32x16 v = {};
    if (!matrix) v = vx.columns(valign && whole, vat, vline, left, w.cols, lds, lane);
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
        Wide<T, 3> sw;
        set_wide(sw, part(S[kt], s));
        get(kx, St::operand(buf, 0, kt, s), lane);
        ks = mma(kx, sw, ks);
        if constexpr (!kSpan) {
          get(qx, St::operand(buf, 2, kt, s), lane);
          qs = mma(qx, first_terms<kP>(sw), qs);
        }
      }
    const float* gate = St::gates(buf);
    const f32x16 gam = load_gate(gate, half) * factor, beta = load_gate(gate + 2 * kC, half);
    f32x16 t = v - gam * ks;
    f32x16 nr = {};
    const f32x16 br = kSpan ? beta * t : clamped<T>(beta * t);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> nw, rw;
      get(nw, St::n(buf, s), lane);
      set_wide(rw, part(br, s));
      nr = mma(nw, rw, nr);
    }
    t -= nr;
    f32x16 u = beta * t;
    settled(t);
    settled(u);
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
    if constexpr (!kSpan) {
      int bad = kC;
      settled(S[0]);
      const bool any_bad = __any(!(fabsf(S[0][0]) < __builtin_inff()));
      if (__builtin_expect(any_bad, 0)) bad = first_bad<T>(u, half);
      u = clamped<T>(u);
      f32x16 pu = {};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Wide<T, kP> pw, uw;
        get(pw, St::p(buf, s), lane);
        set_wide(uw, part(u, s));
        pu = mma(pw, uw, pu);
      }
      f32x16 o = a.scale * gam * qs + pu;
      settled(o);
      if (__builtin_expect(any_bad, 0)) {
        set_nan(o, bad, half);
        if (kSave) set_nan(t, bad + 1, half);
      }
      store_tile<T>(o, oat, line * sizeof(T), oalign && whole, left, w.store_cols, lds, lane);
      oat += kC * int64_t(line);
      if (kSave) {
        store_tile<float>(t, tat, line * 4, salign && whole, left, w.store_cols, lds, lane);
        store_tile<float>(o, pat, line * 4, salign && whole, left, w.store_cols, lds, lane);
        tat += kC * int64_t(line);
        pat += kC * int64_t(line);
      }
    }
    if (c + 1 < chunks) {
      __syncthreads();
      stage.commit(buf);
      __syncthreads();
    }
  }
  if constexpr (kSpan) {
    if (!matrix) {
      store_state<float, KT>(S, a.span_z + start, factor, a, w, lds);
    } else {
      // M in the join's operand order, fp32: this tile's columns are two steps of every 32 rows;
      // for the backward M^T, whose operands the registers hold as they are
      const int mt = w.tile - vtiles;
      const int64_t at = (g.slot * a.H + w.hv) * matrix_bytes(KT);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const f32x16 x = S[kt] * factor;
        wave_sync();
        char* to = lds + 8 * half * tile_pitch<float>() + (lane & 31) * 4;
#pragma unroll
        for (int r = 0; r < 16; ++r)
          *reinterpret_cast<float*>(to + row_base(r) * tile_pitch<float>()) = x[r];
        wave_sync();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const char* from = lds + swap23(lane & 31) * tile_pitch<float>() + (16 * s + 8 * half) * 4;
          f32x8 v;
          __builtin_memcpy(&v, from, 32);
          put_planes(a.span_m + at + matrix_plane(KT, kt, 2 * mt + s), lane, v);
          if (a.span_t != nullptr)  // lane l holds column l: row swap23 of the operand
            put_planes(a.span_t + at + matrix_plane(KT, mt, 2 * kt + s), 32 * half + swap23(lane & 31),
                       part(x, s));
        }
      }
    }
  } else if (g.last) {
    if (a.ht) store_state<float, KT>(S, a.ht + state, factor, a, w, lds);
    if (kSave) store_state<float, KT>(S, a.ends + state, factor, a, w, lds);
  }
}

// Runs the state of 32 columns through its sequence's segments, S <- M S + Z (forward; the
// state before every segment goes to `starts`, except a zero one before the first) or, last to
// first, dS <- M^T dS + Z (backward; the gradient after every segment but the last).  One wave
// per 32 of the state's rows: each publishes its rows as operand terms in LDS and multiplies its
// rows of M with all.
template <int KT, bool kBackward>
__global__ __launch_bounds__(64 * KT) void k_delta_join(Args a) {
  using T = uint16_t;  // fp32 operands as 3 bfloat16 terms, whatever the data
  __shared__ __align__(16) char operand[2 * KT * wide_planes<T, 3>() * kPlane];
  __shared__ __align__(16) char spare[KT][kTileBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* const lds = spare[wave];
  const int tiles = (a.DV + 31) / 32;
  const int64_t head = blockIdx.x / tiles, n = head / a.H;
  const int tile = static_cast<int>(blockIdx.x - head * tiles), hv = static_cast<int>(head - n * a.H);
  const Seq seq = sequence(a, n);
  const int64_t chunks = (seq.len + kC - 1) / kC, count = (chunks + a.seglen - 1) / a.seglen;
  if (count < 2) return;
  const int64_t slot0 = first_slot(a, n, seq, static_cast<int>(a.seglen * kC));
  const int cols = min(32, a.DV - 32 * tile), rows = a.DK - 32 * wave;  // of this wave's tile
  const uint32_t stride = a.DV * 4u;
  const int64_t at = int64_t(32) * wave * a.DV + 32 * tile;
  const int64_t size = int64_t(a.DK) * a.DV;
  const bool whole = aligned16(nullptr, stride, cols) && rows >= 32;
  const int64_t first = kBackward ? count - 1 : 0, step = kBackward ? -1 : 1;

  const float* from = kBackward ? a.dht : a.h0;
  Tile<float> z;
  f32x16 S = {};
  if (from != nullptr && rows > 0) {
    from += head * size + at;
    const bool w0 = whole && aligned16(from, stride, cols);
    if (w0) z.fetch(from, stride, lane);
    S = z.columns(w0, from, stride, rows, cols, lds, lane);
    if (!kBackward)
      store_tile<float>(S, a.starts + (slot0 * a.H + hv) * size + at, stride, whole, rows, cols, lds, lane);
  }
  // this wave's rows of M (or M^T), loaded a segment ahead
  f32x8 m[2 * KT];
  const char* const matrices = kBackward ? a.span_t : a.span_m;
  auto fetch = [&](int64_t i) {
    const char* p = matrices + ((slot0 + i) * a.H + hv) * matrix_bytes(KT);
#pragma unroll
    for (int s = 0; s < 2 * KT; ++s) {
      const auto q = (Global<const f32x4>)global(p + matrix_plane(KT, wave, s)) + lane;
      const f32x4 u = q[0], v = q[64];
#pragma unroll
      for (int e = 0; e < 4; ++e) { m[s][e] = u[e]; m[s][4 + e] = v[e]; }
    }
    if (whole) z.fetch(a.span_z + ((slot0 + i) * a.H + hv) * size + at, stride, lane);
  };
  fetch(first);
  for (int64_t i = first, left = count - 1; left > 0; i += step, --left) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Wide<T, 3> w;
      set_wide(w, part(S, s));
      put(operand + (2 * wave + s) * wide_planes<T, 3>() * kPlane, lane, w);
    }
    Wide<T, 3> mw[2 * KT];
#pragma unroll
    for (int s = 0; s < 2 * KT; ++s) set_wide(mw[s], m[s]);
    f32x16 next = {};
    if (rows > 0)
      next = z.columns(whole, a.span_z + ((slot0 + i) * a.H + hv) * size + at, stride, rows, cols, lds,
                       lane);
    if (left > 1) fetch(i + step);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2 * KT; ++s) {
      Wide<T, 3> w;
      get(w, operand + s * wide_planes<T, 3>() * kPlane, lane);
      next = mma(mw[s], w, next);
    }
    S = next;
    if (rows > 0)
      store_tile<float>(S, a.starts + ((slot0 + i + step) * a.H + hv) * size + at, stride, whole, rows, cols,
                        lds, lane);
    __syncthreads();
  }
}

int64_t units(const Args& a) { return a.seglen > 0 ? a.seg_slots : a.S; }

template <typename T, int KT, int kW>
int launch_w(const Args& a, Mode mode, hipStream_t st) {
  const int tiles = (a.DV + 31) / 32 + (mode == kSpanning ? KT : 0);
  const int64_t blocks = units(a) * a.H * ((tiles + kW - 1) / kW);
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * kW);
  if (mode == kSaving) hipLaunchKernelGGL((k_delta_scan<T, KT, kW, kSaving>), grid, block, 0, st, a);
  else if (mode == kSpanning)
    hipLaunchKernelGGL((k_delta_scan<T, KT, kW, kSpanning>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_scan<T, KT, kW, kForward>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}

template <typename T, int KT>
int launch_kt(const Args& a, Mode mode, hipStream_t st) {
  const int width = a.DV + (mode == kSpanning ? 32 * KT : 0);
  if (width <= 32) return launch_w<T, KT, 1>(a, mode, st);
  if (width <= 64) return launch_w<T, KT, 2>(a, mode, st);
  return launch_w<T, KT, 4>(a, mode, st);
}

template <typename T>
int launch_t(const Args& a, Mode mode, hipStream_t st) {
  if (a.DK <= 32) return launch_kt<T, 1>(a, mode, st);
  if (a.DK <= 64) return launch_kt<T, 2>(a, mode, st);
  return launch_kt<T, 4>(a, mode, st);
}

template <int KT>
int join_kt(const Args& a, bool backward, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.S * a.H * ((a.DV + 31) / 32))), block(64 * KT);
  if (backward) hipLaunchKernelGGL((k_delta_join<KT, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_delta_join<KT, false>), grid, block, 0, st, a);
  return static_cast<int>(hipGetLastError());
}
}  // namespace

int launch_scan(const Args& a, int dtype, bool save, hipStream_t st) {
  const Mode mode = save ? kSaving : kForward;
  return dtype == 0 ? launch_t<float>(a, mode, st) : launch_t<uint16_t>(a, mode, st);
}
int launch_span(const Args& a, int dtype, hipStream_t st) {
  return dtype == 0 ? launch_t<float>(a, kSpanning, st) : launch_t<uint16_t>(a, kSpanning, st);
}
int launch_join(const Args& a, bool backward, hipStream_t st) {
  if (a.DK <= 32) return join_kt<1>(a, backward, st);
  if (a.DK <= 64) return join_kt<2>(a, backward, st);
  return join_kt<4>(a, backward, st);
}

}  // namespace delta
}  // namespace ss2d
