// The short causal convolution: forward, backward, and the form for single tokens.  A thread takes
// four adjacent channels through a unit of tokens of one sequence, its last KW - 1 inputs in
// registers; blocks lay their threads over channels first, then over units.
// Every tensor passes once, which is what bounds it: forward 12,007 tokens of 4096 channels, 198 MB, bf16,
// 37 us (5.3 TB/s); 25,216 tokens of 768 channels 17 us; backward there, with x, dy and dx, 116 MB, 35, of
// which a third is vector work (the activation's slope, KW products three times) that three waves per
// SIMD do not hide.  Eight channels a thread leave too few threads in flight, eight rows ahead too few
// registers (62 us for 46).
#include <algorithm>

#include "ss1d_conv.h"

namespace ss2d {
namespace conv {
namespace {

// kV adjacent channels as they come from memory, in one access.
template <typename T, int kV> struct alignas(kV * sizeof(T)) Values { T v[kV]; };
template <typename T, int kV> struct Piece {
  T v[kV];
  __device__ __forceinline__ void load(const T* p) {
    const auto x = *reinterpret_cast<const Values<T, kV>*>(p);
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = x.v[i];
  }
  __device__ __forceinline__ void store(T* p) const {
    Values<T, kV> x;
#pragma unroll
    for (int i = 0; i < kV; ++i) x.v[i] = v[i];
    *reinterpret_cast<Values<T, kV>*>(p) = x;
  }
  __device__ __forceinline__ void to(float* x) const {
#pragma unroll
    for (int i = 0; i < kV; ++i) x[i] = Elem<T>::to_f32(v[i]);
  }
  __device__ __forceinline__ void from(const float* x) {
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = Elem<T>::from_f32(x[i]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = T(0);
  }
};

// The taps of a thread's channels: w[v * KW + j].
template <int kKW, int kV>
__device__ __forceinline__ void load_taps(const Args& a, int c, float (&w)[kV * kKW], float (&b)[kV]) {
#pragma unroll
  for (int i = 0; i < kV * kKW; ++i) w[i] = a.w[int64_t(c) * kKW + i];
#pragma unroll
  for (int i = 0; i < kV; ++i) b[i] = a.b ? a.b[c + i] : 0.0f;
}

template <int kKW, int kV>
__device__ __forceinline__ float taps(const float (*x)[kV], const float* w, float b, int v) {
#pragma unroll
  for (int j = 0; j < kKW; ++j) b = fmaf(w[v * kKW + j], x[j][v], b);
  return b;
}

// The state's row i of sequence n.
template <typename T> __device__ __forceinline__ T* state_row(const Args& a, void* state, int64_t n, int i, int c) {
  return static_cast<T*>(state) + (n * (a.KW - 1) + i) * a.D + c;
}

// What comes before token t0 of a sequence: its own tokens, the initial state, or zeros.
template <typename T, int kKW, int kV>
__device__ __forceinline__ void load_before(const Args& a, const Sequence& q, const T* x, int64_t t0, int c,
                                            Piece<T, kV>* before) {
#pragma unroll
  for (int i = 0; i < kKW - 1; ++i) {
    const int64_t t = t0 - (kKW - 1) + i;
    if (t >= 0) before[i].load(x + t * a.sx.l);
    else if (a.h0) before[i].load(state_row<const T>(a, const_cast<void*>(a.h0), q.n, static_cast<int>(t + kKW - 1), c));
    else before[i].zero();
  }
}

template <typename T, int kKW, int kV>
__global__ __launch_bounds__(kThreads) void k_conv(Args a, int lanes, int cblocks) {
  constexpr int kRows = 4;
  const int c = (static_cast<int>(blockIdx.x % cblocks) * lanes + static_cast<int>(threadIdx.x) % lanes) * kV;
  const int64_t unit = int64_t(blockIdx.x / cblocks) * (kThreads / lanes) + threadIdx.x / lanes;
  if (c >= a.D || unit >= a.units) return;
  int64_t idx = 0;
  const Sequence q = sequence_of(a.q, unit, a.run, &idx);
  const int64_t t0 = idx * a.run, end = min(q.len, t0 + a.run);
  if (idx > 0 && t0 >= q.len) return;
  float w[kV * kKW], b[kV];
  load_taps<kKW, kV>(a, c, w, b);
  const T* x = static_cast<const T*>(a.x) + q.b * a.sx.b + q.begin * a.sx.l + c;
  T* y = static_cast<T*>(a.y) + (q.b * a.q.L + q.begin) * a.D + c;
  float xs[kKW - 1 + kRows][kV];
  {
    Piece<T, kV> before[kKW > 1 ? kKW - 1 : 1];
    load_before<T, kKW, kV>(a, q, x, t0, c, before);
#pragma unroll
    for (int i = 0; i < kKW - 1; ++i) before[i].to(xs[i]);
  }
  Piece<T, kV> next[kRows];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) next[i].load(x + min(t + i, end - 1) * a.sx.l);
  };
  if (t0 < end) fetch(t0);
  for (int64_t t = t0; t < end; t += kRows) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) next[i].to(xs[kKW - 1 + i]);
    if (t + kRows < end) fetch(t + kRows);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (t + i >= end) break;
      float v[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        v[k] = taps<kKW, kV>(xs + i, w, b[k], k);
        if (a.silu) v[k] = silu_f32(v[k]);
      }
      Piece<T, kV> out;
      out.from(v);
      out.store(y + (t + i) * a.D);
    }
#pragma unroll
    for (int i = 0; i < kKW - 1; ++i)
#pragma unroll
      for (int k = 0; k < kV; ++k) xs[i][k] = xs[i + kRows][k];
  }
  if (a.ht && idx == 0 && kKW > 1) {
    // the last inputs; the first unit alone reads the initial state, which this may replace
    Piece<T, kV> last[kKW > 1 ? kKW - 1 : 1];
    load_before<T, kKW, kV>(a, q, x, q.len, c, last);
#pragma unroll
    for (int i = 0; i < kKW - 1; ++i) last[i].store(state_row<T>(a, a.ht, q.n, i, c));
  }
}

// dpre_t = dy_t act'(pre_t);  dx_t = sum_j w_j dpre_{t + KW - 1 - j},  dw_j = sum_t dpre_t x_{t - KW + 1 + j}.
// A thread recomputes the KW - 1 tokens behind its unit that its own tokens' gradients need; dw and db are
// summed over the block's threads of the same channels in LDS, over blocks by k_conv_sums.
template <typename T, int kKW, int kV>
__global__ __launch_bounds__(kThreads) void k_conv_bwd(Args a, int lanes, int cblocks) {
  constexpr int kRows = 4;
  __shared__ float buffer[kThreads * kV];
  const int c = (static_cast<int>(blockIdx.x % cblocks) * lanes + static_cast<int>(threadIdx.x) % lanes) * kV;
  const int64_t rows = kThreads / lanes, block = blockIdx.x / cblocks, blocks = gridDim.x / cblocks;
  const bool on = c < a.D;
  float w[kV * kKW] = {}, b[kV] = {}, dw[kKW][kV] = {}, db[kV] = {};
  if (on) load_taps<kKW, kV>(a, c, w, b);
  for (int64_t unit = block * rows + threadIdx.x / lanes; unit < a.units && on; unit += blocks * rows) {
    int64_t idx = 0;
    const Sequence q = sequence_of(a.q, unit, a.run, &idx);
    const int64_t t0 = idx * a.run, end = min(q.len, t0 + a.run);
    if (idx > 0 && t0 >= q.len) continue;
    const T* x = static_cast<const T*>(a.x) + q.b * a.sx.b + q.begin * a.sx.l + c;
    const int64_t at = (q.b * a.q.L + q.begin) * a.D + c;
    const T* dy = static_cast<const T*>(a.dy) + at;
    T* dx = static_cast<T*>(a.dx) + at;
    float xs[kKW - 1 + kRows][kV], ds[kKW - 1 + kRows][kV];
    {
      Piece<T, kV> before[kKW > 1 ? kKW - 1 : 1];
      load_before<T, kKW, kV>(a, q, x, t0, c, before);
#pragma unroll
      for (int i = 0; i < kKW - 1; ++i) {
        before[i].to(xs[i]);
#pragma unroll
        for (int k = 0; k < kV; ++k) ds[i][k] = 0.0f;
      }
    }
    Piece<T, kV> nx[kRows], nd[kRows];
    auto fetch = [&](int64_t t) {
      if (q.len == 0) return;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t r = min(t + i, q.len - 1);
        nx[i].load(x + r * a.sx.l);
        nd[i].load(dy + r * a.D);
      }
    };
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      nx[i].zero();
      nd[i].zero();
    }
    fetch(t0);
    const int64_t first = idx == 0 ? -(kKW - 1) : t0;  // the unit's inputs, the state's among them
    for (int64_t t = t0; t < end + kKW - 1; t += kRows) {
      float g[kRows][kV];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        nx[i].to(xs[kKW - 1 + i]);
        nd[i].to(g[i]);
      }
      if (t + kRows < end + kKW - 1) fetch(t + kRows);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t s = t + i;
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          float d = g[i][k];
          if (a.silu) {
            const float pre = taps<kKW, kV>(xs + i, w, b[k], k);
            const float sg = __builtin_amdgcn_rcpf(1.0f + exp2_hw(-pre * kLog2e));
            // sigmoid (1 + pre (1 - sigmoid)), its limits where pre is infinite
            d *= sg == 0.0f ? 0.0f : (sg == 1.0f ? 1.0f : sg * fmaf(pre, 1.0f - sg, 1.0f));
          }
          ds[kKW - 1 + i][k] = s < q.len ? d : 0.0f;
          if (s < end) {
            db[k] += d;
#pragma unroll
            for (int j = 0; j < kKW; ++j) dw[j][k] = fmaf(d, xs[i + j][k], dw[j][k]);
          }
        }
        const int64_t p = s - (kKW - 1);  // whose gradient is complete
        if (p < first || p >= end) continue;
        float v[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          v[k] = 0.0f;
#pragma unroll
          for (int j = 0; j < kKW; ++j) v[k] = fmaf(w[k * kKW + j], ds[kKW - 1 + i - j][k], v[k]);
        }
        if (a.dht && p >= q.len - (kKW - 1)) {
          Piece<T, kV> e;
          float ev[kV];
          e.load(state_row<const T>(a, const_cast<void*>(a.dht), q.n, static_cast<int>(p - q.len + kKW - 1), c));
          e.to(ev);
#pragma unroll
          for (int k = 0; k < kV; ++k) v[k] += ev[k];
        }
        Piece<T, kV> out;
        out.from(v);
        if (p >= 0) out.store(dx + p * a.D);
        else if (a.dh0) out.store(state_row<T>(a, a.dh0, q.n, static_cast<int>(p + kKW - 1), c));
      }
#pragma unroll
      for (int i = 0; i < kKW - 1; ++i)
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          xs[i][k] = xs[i + kRows][k];
          ds[i][k] = ds[i + kRows][k];
        }
    }
  }
  // the block's sums, over its threads of the same channels in order
  const int cols = lanes * kV, c0 = static_cast<int>(blockIdx.x % cblocks) * cols;
  float* out = a.parts + block * (kKW + 1) * a.D;
#pragma unroll
  for (int j = 0; j <= kKW; ++j) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kV; ++k) buffer[threadIdx.x * kV + k] = j < kKW ? dw[j < kKW ? j : 0][k] : db[k];
    __syncthreads();
    for (int i = threadIdx.x; i < cols && c0 + i < a.D; i += kThreads) {
      float v = 0.0f;
      for (int r = 0; r < rows; ++r) v += buffer[r * cols + i];
      out[int64_t(j) * a.D + c0 + i] = v;
    }
  }
}

// dw and db: sums over the blocks, 64 columns and 16 groups of blocks per block.
__global__ __launch_bounds__(1024) void k_conv_sums(Args a, int64_t count) {
  __shared__ float buffer[16][64];
  const int64_t width = int64_t(a.KW + 1) * a.D, c = int64_t(blockIdx.x) * 64 + (threadIdx.x & 63);
  const int g = threadIdx.x >> 6;
  float x[4] = {};
  if (c < width) {
    const float* p = a.parts + c;
    int64_t b = g;
    for (; b + 48 < count; b += 64)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] += p[(b + 16 * i) * width];
    for (; b < count; b += 16) x[0] += p[b * width];
  }
  buffer[g][threadIdx.x & 63] = (x[0] + x[1]) + (x[2] + x[3]);
  __syncthreads();
  if (g != 0 || c >= width) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += buffer[i][threadIdx.x];
  const int64_t j = c / a.D, d = c % a.D;
  if (j < a.KW) a.dw[d * a.KW + j] = v;
  else if (a.db) a.db[d] = v;
}

// q.L tokens of each row, states in place: 64 rows of 5 tokens of 4096 channels in 5 us, the latency of
// its loads.
template <typename T, int kKW, int kV>
__global__ __launch_bounds__(64) void k_conv_step(Args a, int cblocks) {
  const int c = (static_cast<int>(blockIdx.x % cblocks) * 64 + static_cast<int>(threadIdx.x)) * kV;
  __shared__ uint32_t seen[2];
  int r = blockIdx.x / cblocks;
  find_repeats(a.slots, r, 1, seen);
  const int slot = slot_of(a.slots, r, 0, seen);
  if (slot < 0) return;
  const bool more = a.slots.at && seen[1];
  const bool on = c < a.D;
  const int cc = on ? c : 0;
  float w[kV * kKW], b[kV], xs[kKW][kV];
  Piece<T, kV> held[kKW];
  load_taps<kKW, kV>(a, cc, w, b);
#pragma unroll
  for (int i = 0; i < kKW - 1; ++i) held[i].load(state_row<T>(a, a.state, slot, i, cc));
  for (;;) {
    for (int64_t t = 0; t < a.q.L; ++t) {
      held[kKW - 1].load(static_cast<const T*>(a.x) + r * a.sx.b + t * a.sx.l + cc);
#pragma unroll
      for (int i = 0; i < kKW; ++i) held[i].to(xs[i]);
      float v[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        v[k] = taps<kKW, kV>(xs, w, b[k], k);
        if (a.silu) v[k] = silu_f32(v[k]);
      }
      Piece<T, kV> out;
      out.from(v);
      if (on) out.store(static_cast<T*>(a.y) + (r * a.q.L + t) * a.D + c);
#pragma unroll
      for (int i = 0; i < kKW - 1; ++i) held[i] = held[i + 1];
    }
    if (!more) break;
    r = next_of(a.slots, r, slot);
    if (r >= a.slots.rows) break;
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < kKW - 1; ++i) held[i].store(state_row<T>(a, a.state, slot, i, c));
}

enum Kind { kForward, kBackward, kStep };

template <typename T, int kKW, int kV> int launch_one(const Args& a, Kind kind, hipStream_t st) {
  if (kind == kStep) {
    const int cblocks = (a.D + 64 * kV - 1) / (64 * kV);
    const int64_t blocks = int64_t(a.slots.rows) * cblocks;
    hipLaunchKernelGGL((k_conv_step<T, kKW, kV>), dim3(static_cast<unsigned>(blocks)), dim3(64), 0, st, a, cblocks);
    return static_cast<int>(hipGetLastError());
  }
  const int lanes = lanes_of(a.D, kV), cblocks = (a.D + lanes * kV - 1) / (lanes * kV);
  const int64_t per = kThreads / lanes;
  const int64_t blocks = kind == kForward ? (a.units + per - 1) / per : unit_blocks(a, kV);
  const dim3 grid(static_cast<unsigned>(blocks * cblocks)), block(kThreads);
  if (kind == kForward) hipLaunchKernelGGL((k_conv<T, kKW, kV>), grid, block, 0, st, a, lanes, cblocks);
  else hipLaunchKernelGGL((k_conv_bwd<T, kKW, kV>), grid, block, 0, st, a, lanes, cblocks);
  return static_cast<int>(hipGetLastError());
}

template <typename T, int kV> int launch_taps(const Args& a, Kind kind, hipStream_t st) {
  switch (a.KW) {
    case 1: return launch_one<T, 1, kV>(a, kind, st);
    case 2: return launch_one<T, 2, kV>(a, kind, st);
    case 3: return launch_one<T, 3, kV>(a, kind, st);
    case 4: return launch_one<T, 4, kV>(a, kind, st);
    case 5: return launch_one<T, 5, kV>(a, kind, st);
    case 6: return launch_one<T, 6, kV>(a, kind, st);
    case 7: return launch_one<T, 7, kV>(a, kind, st);
    default: return launch_one<T, 8, kV>(a, kind, st);
  }
}

int launch_types(const Args& a, int dtype, bool vec, Kind kind, hipStream_t st) {
  if (dtype == 0) return vec ? launch_taps<float, 4>(a, kind, st) : launch_taps<float, 1>(a, kind, st);
  return vec ? launch_taps<uint16_t, 4>(a, kind, st) : launch_taps<uint16_t, 1>(a, kind, st);
}

}  // namespace

// The widest row of threads, of 256 down to 8 (32 of single channels: 333 of them by 32 threads and by 16,
// 51.6 and 71.0 us a training step of 8 x 3000), whose blocks leave the fewest threads idle: a training
// step of 8 x 20,000 tokens of 40 channels, 10 of 32 threads at work and 10 of 16, 66.4 and 44.6 us.
int lanes_of(int64_t D, int width) {
  const int64_t pieces = (D + width - 1) / width;
  int best = width == 1 && pieces > 16 ? 32 : 8;
  int64_t least = (pieces + best - 1) / best * best;
  for (int lanes = 2 * best; lanes <= kThreads; lanes *= 2) {
    const int64_t covered = (pieces + lanes - 1) / lanes * lanes;
    if (covered <= least) {
      least = covered;
      best = lanes;
    }
  }
  return best;
}

// Tokens of a thread: as few (8 at least, backward 12) as let all waves be on the chip at once, in equal
// runs; each run reads KW - 1 tokens of its neighbour again, and waves that come in a second round
// wait for the first.  Where that takes runs above 64 tokens there are many rounds, and runs of 24 do.  With
// runs of 13, 16, 20, 25, 32 and 41 tokens, us, the rule's marked: forward 128 x 197 x 768 19.5, *17.4,
// 17.2, 17.2, 19.4, 18.8; 12,007 packed tokens of 4096 channels 46.2, 43.6, 41.3, 43.2, 44.1, *39.5 (37:
// 45.5); with the forward before it, backward 128 x 197 x 768 63.9, 64.2, 64.4, *56.4, 61.7, 61.3; 64 of
// them *37.2, 39.1, 38.4, 40.4, 45.8, 46.5; fp32 128 of them 99.9, 99.9, 94.9, 97.0, 102.6, *88.1.
int run_of(int64_t rows, int64_t tokens, int64_t S, int64_t D, int KW, int dtype, bool backward) {
  // waves on a SIMD, by the kernels' registers
  const int wide = dtype == 0 ? 1 : 0, deep = KW > 4 ? 1 : 0;
  const int64_t waves = 1024 * (backward ? (wide || deep ? 2 : 3) : 5 - wide - deep);
  // runs of a dense row; or of all packed tokens, of which each sequence may end in one of its own
  const int64_t all = waves * 256 / std::max<int64_t>(1, D);
  const int64_t runs = rows > 0 ? all / rows : all - S;
  const int64_t length = rows > 0 ? tokens / rows : tokens;
  const int64_t run = runs > 0 ? (length + runs - 1) / runs : length;
  return static_cast<int>(run > 64 ? 24 : std::max<int64_t>(run, backward ? 12 : 8));
}

int64_t unit_blocks(const Args& a, int width) {
  const int lanes = lanes_of(a.D, width);
  const int64_t per = kThreads / lanes, all = (a.units + per - 1) / per;
  const int64_t cblocks = (a.D + int64_t(lanes) * width - 1) / (int64_t(lanes) * width);
  return std::min(all, std::max<int64_t>(1, 2048 / cblocks));
}

int launch_conv(const Args& a, int dtype, bool vec, hipStream_t st) { return launch_types(a, dtype, vec, kForward, st); }
int launch_conv_bwd(const Args& a, int dtype, bool vec, hipStream_t st) { return launch_types(a, dtype, vec, kBackward, st); }
int launch_conv_step(const Args& a, int dtype, bool vec, hipStream_t st) { return launch_types(a, dtype, vec, kStep, st); }

int launch_conv_sums(const Args& a, int64_t blocks, hipStream_t st) {
  const int64_t width = int64_t(a.KW + 1) * a.D;
  hipLaunchKernelGGL(k_conv_sums, dim3(static_cast<unsigned>((width + 63) / 64)), dim3(1024), 0, st, a, blocks);
  return static_cast<int>(hipGetLastError());
}

}  // namespace conv
}  // namespace ss2d
