// The group norm with its activation, channels last, in two ways.
//
// A block holds whole groups of an image in registers: x is read once, its mean and then the squares
// about it are summed over the block, and y is written.  Where a group is too large for that, chunks
// of positions give every channel's mean and sum of squares about it, one wave per group joins
// them, and another pass normalises.
#include <algorithm>
#include <numeric>

#include "ss2d_group.h"

namespace ss2d {
namespace group {
namespace {

template <typename T, int kV> struct Piece {
  T v[kV];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kV * sizeof(T) == 16) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    else v[0] = *p;
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kV * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    else *p = v[0];
  }
  __device__ __forceinline__ float at(int i) const { return Elem<T>::to_f32(v[i]); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = T(0);
  }
};

// SiLU and its derivative sigmoid(v) (1 + v (1 - sigmoid(v))), with their limits.
__device__ __forceinline__ float slope(float v) {
  const float s = __builtin_amdgcn_rcpf(1.0f + exp2_hw(-v * kLog2e));
  return s == 0.0f ? 0.0f : (s == 1.0f ? 1.0f : s * fmaf(v, 1.0f - s, 1.0f));
}

__device__ __forceinline__ float affine(float unit, float w, float b) { return fmaf(unit, w, b); }

// ---- groups in registers -----------------------------------------------------------------------
// The threads of a block over a set's channels (kV adjacent ones each, `cv` counting them) and over
// positions row, row + pass, ...
struct Tile {
  int cv, row, pass, nv;
  bool on;
};
template <int kThreads> __device__ __forceinline__ Tile tile_of(const Args& a, int width) {
  Tile t;
  t.nv = a.set / width;
  t.pass = kThreads / t.nv;
  t.cv = threadIdx.x % t.nv;
  t.row = threadIdx.x / t.nv;
  t.on = t.row < t.pass;
  return t;
}

// Sums of every channel of a set over the block's threads, from part[row][set]: rows p, p + P, ...
// into row p, in place (row p is read by the thread that writes it alone).  Returns P.
template <int kThreads> __device__ __forceinline__ int column_sums(float* part, int set, int rows) {
  const int P = min(max(1, kThreads / set), rows);
  __syncthreads();
  for (int i = threadIdx.x; i < P * set; i += kThreads) {
    const int c = i % set, p = i / set;
    float v = part[p * set + c];
    for (int r = p + P; r < rows; r += P) v += part[r * set + c];
    part[p * set + c] = v;
  }
  __syncthreads();
  return P;
}

// Every group's sum of part[0 .. P - 1][set], over `count`, into out[group].
template <int kThreads>
__device__ __forceinline__ void group_sums(const float* part, int set, int P, int cg, float count, float* out) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int g = wave; g < set / cg; g += kThreads / 64) {
    float v = 0.0f;
    for (int i = lane; i < P * cg; i += 64) v += part[i / cg * set + g * cg + i % cg];
    v = lane_sum<64>(v);
    if (lane == 0) out[g] = v / count;
  }
  __syncthreads();
}

// The mean and r of every group of the set, of values held in registers.
template <typename T, int kV, int kRows, int kThreads>
__device__ __forceinline__ void statistics(const Args& a, const Tile& t, const Piece<T, kV>* x, float* part,
                                           float* mean, float* r) {
  const float count = static_cast<float>(a.L) * a.cg;
  float s[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    s[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[k] += x[i].at(k);  // rows past the end hold zeros
    if (t.on) part[t.row * a.set + t.cv * kV + k] = s[k];
  }
  group_sums<kThreads>(part, a.set, column_sums<kThreads>(part, a.set, t.pass), a.cg, count, mean);
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const float m = mean[(t.cv * kV + k) / a.cg];
    s[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float d = x[i].at(k) - m;
      s[k] = t.row + i * t.pass < a.L ? fmaf(d, d, s[k]) : s[k];
    }
  }
#pragma unroll
  for (int k = 0; k < kV; ++k)
    if (t.on) part[t.row * a.set + t.cv * kV + k] = s[k];
  group_sums<kThreads>(part, a.set, column_sums<kThreads>(part, a.set, t.pass), a.cg, count, r);
  for (int g = threadIdx.x; g < a.set / a.cg; g += kThreads) r[g] = 1.0f / sqrtf(r[g] + a.eps);
  __syncthreads();
}

constexpr int kMaxGroups = 256;  // of a set

template <typename T, int kV, int kRows, int kThreads>
__global__ __launch_bounds__(kThreads) void k_group(Args a) {
  __shared__ float part[kThreads * kV], mean[kMaxGroups], r[kMaxGroups];
  const unsigned id = xcd_local_order(blockIdx.x, gridDim.x);
  const int64_t b = id / a.sets;
  const int c0 = static_cast<int>(id % a.sets) * a.set;
  const Tile t = tile_of<kThreads>(a, kV);
  const int c = c0 + t.cv * kV;
  const int64_t base = b * a.L * a.C + c;
  const T* x = static_cast<const T*>(a.x) + base;
  Piece<T, kV> rows[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    rows[i].zero();
    if (t.on && t.row + i * t.pass < a.L) rows[i].load(x + int64_t(t.row + i * t.pass) * a.C);
  }
  float w[kV], bias[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    w[k] = a.w ? a.w[c + k] : 1.0f;
    bias[k] = a.b ? a.b[c + k] : 0.0f;
  }
  statistics<T, kV, kRows, kThreads>(a, t, rows, part, mean, r);
  if (a.stats)
    for (int g = threadIdx.x; g < a.set / a.cg; g += kThreads) {
      float* to = a.stats + (b * a.G + c0 / a.cg + g) * 2;
      to[0] = mean[g];
      to[1] = r[g];
    }
  if (!t.on) return;
  float m[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int g = (t.cv * kV + k) / a.cg;
    m[k] = mean[g];
    w[k] *= r[g];
  }
  T* y = static_cast<T*>(a.y) + base;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (t.row + i * t.pass >= a.L) break;
    Piece<T, kV> out;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float v = affine(rows[i].at(k) - m[k], w[k], bias[k]);
      if (a.silu) v = silu_f32(v);
      out.v[k] = Elem<T>::from_f32(v);
    }
    out.store(y + int64_t(t.row + i * t.pass) * a.C);
  }
}

// With d = dy act'(.), e = d w, n the unit values:  dw = sum d n, db = sum d,
// dx = r (e - mean(e) - n mean(e n)).
template <typename T, int kV, int kRows, int kThreads>
__global__ __launch_bounds__(kThreads) void k_group_bwd(Args a) {
  __shared__ float part[2][kThreads * kV], mean[kMaxGroups], r[kMaxGroups];
  const unsigned id = xcd_local_order(blockIdx.x, gridDim.x);
  const int64_t b = id / a.sets;
  const int c0 = static_cast<int>(id % a.sets) * a.set;
  const Tile t = tile_of<kThreads>(a, kV);
  const int c = c0 + t.cv * kV;
  const int64_t base = b * a.L * a.C + c;
  const T *x = static_cast<const T*>(a.x) + base, *dy = static_cast<const T*>(a.dy) + base;
  Piece<T, kV> xs[kRows], ds[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    xs[i].zero();
    ds[i].zero();
    if (t.on && t.row + i * t.pass < a.L) {
      xs[i].load(x + int64_t(t.row + i * t.pass) * a.C);
      ds[i].load(dy + int64_t(t.row + i * t.pass) * a.C);
    }
  }
  float w[kV], bias[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    w[k] = a.w ? a.w[c + k] : 1.0f;
    bias[k] = a.b ? a.b[c + k] : 0.0f;
  }
  if (a.given) {
    for (int g = threadIdx.x; g < a.set / a.cg; g += kThreads) {
      const float* from = a.stats + (b * a.G + c0 / a.cg + g) * 2;
      mean[g] = from[0];
      r[g] = from[1];
    }
    __syncthreads();
  } else {
    statistics<T, kV, kRows, kThreads>(a, t, xs, part[0], mean, r);
  }
  float m[kV], rs[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int g = (t.cv * kV + k) / a.cg;
    m[k] = mean[g];
    rs[k] = r[g];
    float sd = 0.0f, sn = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float n = (xs[i].at(k) - m[k]) * rs[k];
      float d = ds[i].at(k);
      if (a.silu) d *= slope(affine(n, w[k], bias[k]));
      const bool in = t.row + i * t.pass < a.L;
      sd += in ? d : 0.0f;
      sn = in ? fmaf(d, n, sn) : sn;
    }
    if (t.on) {
      part[0][t.row * a.set + t.cv * kV + k] = sd;
      part[1][t.row * a.set + t.cv * kV + k] = sn;
    }
  }
  const int P = column_sums<kThreads>(part[0], a.set, t.pass);
  column_sums<kThreads>(part[1], a.set, t.pass);
  for (int i = threadIdx.x; i < a.set; i += kThreads) {
    float sd = 0.0f, sn = 0.0f;
    for (int p = 0; p < P; ++p) {
      sd += part[0][p * a.set + i];
      sn += part[1][p * a.set + i];
    }
    if (a.parts) {
      a.parts[(b * 2) * a.C + c0 + i] = sd;
      a.parts[(b * 2 + 1) * a.C + c0 + i] = sn;
    }
    const float wi = a.w ? a.w[c0 + i] : 1.0f;
    part[0][i] = sd * wi;
    part[1][i] = sn * wi;
  }
  __syncthreads();
  const float count = static_cast<float>(a.L) * a.cg;
  group_sums<kThreads>(part[0], a.set, 1, a.cg, count, mean);
  group_sums<kThreads>(part[1], a.set, 1, a.cg, count, r);
  if (!t.on) return;
  T* dx = static_cast<T*>(a.dx) + base;
  float se[kV], sn[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int g = (t.cv * kV + k) / a.cg;
    se[k] = mean[g];
    sn[k] = r[g];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (t.row + i * t.pass >= a.L) break;
    Piece<T, kV> out;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const float n = (xs[i].at(k) - m[k]) * rs[k];
      float d = ds[i].at(k);
      if (a.silu) d *= slope(affine(n, w[k], bias[k]));
      out.v[k] = Elem<T>::from_f32(rs[k] * (fmaf(d, w[k], -se[k]) - n * sn[k]));
    }
    out.store(dx + int64_t(t.row + i * t.pass) * a.C);
  }
}

// ---- chunks of positions ------------------------------------------------------------------------
// A block of 256 threads takes a chunk of an image's positions and lanes * kV channels; each thread
// every (256 / lanes)-th position.
struct Part {
  int c, row, rows, cols;
  int64_t b, chunk, first, count;
};
template <int kV> __device__ __forceinline__ Part part_of(const Args& a, int lanes, int cblocks) {
  Part p;
  const int64_t id = blockIdx.x / cblocks;
  p.cols = lanes * kV;
  p.c = static_cast<int>(blockIdx.x % cblocks) * p.cols + static_cast<int>(threadIdx.x) % lanes * kV;
  p.row = threadIdx.x / lanes;
  p.rows = 256 / lanes;
  p.b = id / a.chunks;
  p.chunk = id % a.chunks;
  p.first = p.chunk * a.chunk;
  p.count = min(a.L - p.first, a.chunk);
  return p;
}

// Every channel's mean over the chunk and sum of squares about it.  Eight positions at a time give
// both from the values in registers; they join what came before by
//   mean += f (m - mean), M2 += q + (m - mean)^2 f n_before,  f = n / (n_before + n).
template <typename T, int kV>
__global__ __launch_bounds__(256) void k_group_chunks(Args a, int lanes, int cblocks) {
  constexpr int kAhead = 8;
  __shared__ float buffer[2][256 * kV];
  const Part p = part_of<kV>(a, lanes, cblocks);
  const bool on = p.c < a.C;
  const T* x = static_cast<const T*>(a.x) + (p.b * a.L + p.first) * a.C + (on ? p.c : 0);
  float mean[kV] = {}, M2[kV] = {};
  float count = 0.0f;
  for (int64_t t = p.row; t < p.count; t += kAhead * p.rows) {
    Piece<T, kV> v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i].load(x + min(t + i * p.rows, p.count - 1) * a.C);
    const int n = static_cast<int>(min(int64_t(kAhead), (p.count - t + p.rows - 1) / p.rows));
    const float by = 1.0f / n, f = n / (count + n);
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      float s = 0.0f, q = 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s += i < n ? v[i].at(k) : 0.0f;
      s *= by;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float d = v[i].at(k) - s;
        q = i < n ? fmaf(d, d, q) : q;
      }
      const float d = s - mean[k];
      mean[k] = fmaf(d, f, mean[k]);
      M2[k] += fmaf(d * d, f * count, q);
    }
    count += n;
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    buffer[0][threadIdx.x * kV + k] = mean[k];
    buffer[1][threadIdx.x * kV + k] = M2[k];
  }
  __syncthreads();
  const int c0 = static_cast<int>(blockIdx.x % cblocks) * p.cols;
  float* out = a.parts + (p.b * a.chunks + p.chunk) * 2 * a.C;
  for (int i = threadIdx.x; i < p.cols && c0 + i < a.C; i += 256) {
    float m = 0.0f, q = 0.0f, before = 0.0f;
    for (int r = 0; r < p.rows; ++r) {
      const float n = static_cast<float>((p.count - r + p.rows - 1) / p.rows);  // of row r
      if (n <= 0.0f) break;
      const float d = buffer[0][r * p.cols + i] - m, f = n / (before + n);
      m = fmaf(d, f, m);
      q += fmaf(d * d, f * before, buffer[1][r * p.cols + i]);
      before += n;
    }
    out[c0 + i] = m;
    out[a.C + c0 + i] = q;
  }
}

// One wave per image and group: its statistics from its channels' in every chunk.
__global__ __launch_bounds__(256) void k_group_join(Args a) {
  const int64_t id = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (id >= a.B * a.G) return;
  const int64_t b = id / a.G, items = a.chunks * a.cg;
  const int c0 = static_cast<int>(id % a.G) * a.cg;
  const float* parts = a.parts + b * a.chunks * 2 * a.C + c0;
  const float total = static_cast<float>(a.L) * a.cg;
  auto positions = [&](int64_t k) { return static_cast<float>(min(a.L - k * a.chunk, a.chunk)); };
  float s = 0.0f;
  for (int64_t i = lane; i < items; i += 64)
    s = fmaf(positions(i / a.cg), parts[i / a.cg * 2 * a.C + i % a.cg], s);
  const float mean = lane_sum<64>(s) / total;
  float q = 0.0f;
  for (int64_t i = lane; i < items; i += 64) {
    const float* at = parts + i / a.cg * 2 * a.C + i % a.cg;
    const float d = at[0] - mean;
    q += fmaf(d * d, positions(i / a.cg), at[a.C]);
  }
  q = lane_sum<64>(q) / total;
  if (lane == 0) {
    a.stats[id * 2] = mean;
    a.stats[id * 2 + 1] = 1.0f / sqrtf(q + a.eps);
  }
}

// A thread's channels: mean, r, weight and bias.
template <int kV>
__device__ __forceinline__ void load_vectors(const Args& a, const Part& p, float* m, float* r, float* w, float* b) {
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const float* s = a.stats + (p.b * a.G + (p.c + k) / a.cg) * 2;
    m[k] = s[0];
    r[k] = s[1];
    w[k] = a.w ? a.w[p.c + k] : 1.0f;
    b[k] = a.b ? a.b[p.c + k] : 0.0f;
  }
}

template <typename T, int kV>
__global__ __launch_bounds__(256) void k_group_apply(Args a, int lanes, int cblocks) {
  constexpr int kAhead = 4;
  const Part p = part_of<kV>(a, lanes, cblocks);
  if (p.c >= a.C) return;
  float m[kV], r[kV], w[kV], b[kV];
  load_vectors<kV>(a, p, m, r, w, b);
#pragma unroll
  for (int k = 0; k < kV; ++k) w[k] *= r[k];
  const int64_t base = (p.b * a.L + p.first) * a.C + p.c;
  const T* x = static_cast<const T*>(a.x) + base;
  T* y = static_cast<T*>(a.y) + base;
  for (int64_t t = p.row; t < p.count; t += kAhead * p.rows) {
    Piece<T, kV> v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i].load(x + min(t + i * p.rows, p.count - 1) * a.C);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i * p.rows >= p.count) break;
      Piece<T, kV> out;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        float f = affine(v[i].at(k) - m[k], w[k], b[k]);
        if (a.silu) f = silu_f32(f);
        out.v[k] = Elem<T>::from_f32(f);
      }
      out.store(y + (t + i * p.rows) * a.C);
    }
  }
}

// Every channel's sums of d and d n over a chunk.
template <typename T, int kV>
__global__ __launch_bounds__(256) void k_group_bwd_chunks(Args a, int lanes, int cblocks) {
  constexpr int kAhead = 4;
  __shared__ float buffer[2][256 * kV];
  const Part p = part_of<kV>(a, lanes, cblocks);
  float sd[kV] = {}, sn[kV] = {};
  if (p.c < a.C) {
    float m[kV], r[kV], w[kV], b[kV];
    load_vectors<kV>(a, p, m, r, w, b);
    const int64_t base = (p.b * a.L + p.first) * a.C + p.c;
    const T *x = static_cast<const T*>(a.x) + base, *dy = static_cast<const T*>(a.dy) + base;
    for (int64_t t = p.row; t < p.count; t += kAhead * p.rows) {
      Piece<T, kV> v[kAhead], g[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t at = min(t + i * p.rows, p.count - 1) * a.C;
        v[i].load(x + at);
        g[i].load(dy + at);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (t + i * p.rows >= p.count) break;
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          const float n = (v[i].at(k) - m[k]) * r[k];
          float d = g[i].at(k);
          if (a.silu) d *= slope(affine(n, w[k], b[k]));
          sd[k] += d;
          sn[k] = fmaf(d, n, sn[k]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    buffer[0][threadIdx.x * kV + k] = sd[k];
    buffer[1][threadIdx.x * kV + k] = sn[k];
  }
  __syncthreads();
  const int c0 = static_cast<int>(blockIdx.x % cblocks) * p.cols;
  float* out = a.parts + (p.b * a.chunks + p.chunk) * 2 * a.C;
  for (int i = threadIdx.x; i < p.cols && c0 + i < a.C; i += 256) {
    float d = 0.0f, n = 0.0f;
    for (int r = 0; r < p.rows; ++r) {
      d += buffer[0][r * p.cols + i];
      n += buffer[1][r * p.cols + i];
    }
    out[c0 + i] = d;
    out[a.C + c0 + i] = n;
  }
}

// One wave per image and group: the means of e and e n.
__global__ __launch_bounds__(256) void k_group_bwd_join(Args a) {
  const int64_t id = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (id >= a.B * a.G) return;
  const int64_t b = id / a.G, items = a.chunks * a.cg;
  const int c0 = static_cast<int>(id % a.G) * a.cg;
  const float* parts = a.parts + b * a.chunks * 2 * a.C + c0;
  float se = 0.0f, sn = 0.0f;
  for (int64_t i = lane; i < items; i += 64) {
    const float* at = parts + i / a.cg * 2 * a.C + i % a.cg;
    const float w = a.w ? a.w[c0 + i % a.cg] : 1.0f;
    se = fmaf(w, at[0], se);
    sn = fmaf(w, at[a.C], sn);
  }
  const float total = static_cast<float>(a.L) * a.cg;
  se = lane_sum<64>(se) / total;
  sn = lane_sum<64>(sn) / total;
  if (lane == 0) {
    a.sums[id * 2] = se;
    a.sums[id * 2 + 1] = sn;
  }
}

template <typename T, int kV>
__global__ __launch_bounds__(256) void k_group_bwd_apply(Args a, int lanes, int cblocks) {
  constexpr int kAhead = 4;
  const Part p = part_of<kV>(a, lanes, cblocks);
  if (p.c >= a.C) return;
  float m[kV], r[kV], w[kV], b[kV], se[kV], sn[kV];
  load_vectors<kV>(a, p, m, r, w, b);
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const float* s = a.sums + (p.b * a.G + (p.c + k) / a.cg) * 2;
    se[k] = s[0];
    sn[k] = s[1];
  }
  const int64_t base = (p.b * a.L + p.first) * a.C + p.c;
  const T *x = static_cast<const T*>(a.x) + base, *dy = static_cast<const T*>(a.dy) + base;
  T* dx = static_cast<T*>(a.dx) + base;
  for (int64_t t = p.row; t < p.count; t += kAhead * p.rows) {
    Piece<T, kV> v[kAhead], g[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = min(t + i * p.rows, p.count - 1) * a.C;
      v[i].load(x + at);
      g[i].load(dy + at);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i * p.rows >= p.count) break;
      Piece<T, kV> out;
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const float n = (v[i].at(k) - m[k]) * r[k];
        float d = g[i].at(k);
        if (a.silu) d *= slope(affine(n, w[k], b[k]));
        out.v[k] = Elem<T>::from_f32(r[k] * (fmaf(d, w[k], -se[k]) - n * sn[k]));
      }
      out.store(dx + (t + i * p.rows) * a.C);
    }
  }
}

// dw and db: the sums over images and chunks, 64 columns and 16 groups of them per block.
__global__ __launch_bounds__(1024) void k_group_sums(Args a, int64_t count) {
  __shared__ float buffer[16][64];
  const int64_t width = 2 * int64_t(a.C), c = int64_t(blockIdx.x) * 64 + (threadIdx.x & 63);
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
  float* out = c < a.C ? a.db : a.dw;
  if (out) out[c % a.C] = v;
}

// The widest row of threads, of 256, 128, 64 and 32, whose blocks leave the fewest threads idle.
int lanes_of(int64_t C, int width) {
  const int64_t pieces = (C + width - 1) / width;
  int best = 32;
  int64_t least = (pieces + 31) / 32 * 32;
  for (int lanes = 64; lanes <= 256; lanes *= 2) {
    const int64_t covered = (pieces + lanes - 1) / lanes * lanes;
    if (covered <= least) {
      least = covered;
      best = lanes;
    }
  }
  return best;
}

template <typename T, int kV, int kThreads, bool kBack>
int launch_rows(const Args& a, int rows, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.B * a.sets)), block(kThreads);
#define SS2D_GROUP_ROWS(n)                                                                      \
  if (rows <= n) {                                                                              \
    if constexpr (kBack) hipLaunchKernelGGL((k_group_bwd<T, kV, n, kThreads>), grid, block, 0, st, a); \
    else hipLaunchKernelGGL((k_group<T, kV, n, kThreads>), grid, block, 0, st, a);              \
    return static_cast<int>(hipGetLastError());                                                 \
  }
  SS2D_GROUP_ROWS(1)
  SS2D_GROUP_ROWS(2)
  SS2D_GROUP_ROWS(4)
  SS2D_GROUP_ROWS(8)
  if constexpr (!kBack) {
    SS2D_GROUP_ROWS(16)
  }
#undef SS2D_GROUP_ROWS
  return static_cast<int>(hipErrorInvalidValue);
}

template <typename T, int kV> int launch_t(const Args& a, const Plan& p, bool back, hipStream_t st) {
  if (p.rows > 0) {
    if (back) return p.threads == 256 ? launch_rows<T, kV, 256, true>(a, p.rows, st)
                                      : launch_rows<T, kV, 512, true>(a, p.rows, st);
    return p.threads == 256 ? launch_rows<T, kV, 256, false>(a, p.rows, st)
                            : launch_rows<T, kV, 1024, false>(a, p.rows, st);
  }
  const int lanes = lanes_of(a.C, kV), cblocks = (a.C + lanes * kV - 1) / (lanes * kV);
  const dim3 grid(static_cast<unsigned>(a.B * a.chunks * cblocks)), block(256);
  const dim3 groups(static_cast<unsigned>((a.B * a.G + 3) / 4));
  if (!a.given) {
    hipLaunchKernelGGL((k_group_chunks<T, kV>), grid, block, 0, st, a, lanes, cblocks);
    hipLaunchKernelGGL(k_group_join, groups, block, 0, st, a);
  }
  if (!back) {
    hipLaunchKernelGGL((k_group_apply<T, kV>), grid, block, 0, st, a, lanes, cblocks);
  } else {
    hipLaunchKernelGGL((k_group_bwd_chunks<T, kV>), grid, block, 0, st, a, lanes, cblocks);
    hipLaunchKernelGGL(k_group_bwd_join, groups, block, 0, st, a);
    hipLaunchKernelGGL((k_group_bwd_apply<T, kV>), grid, block, 0, st, a, lanes, cblocks);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_any(const Args& a, const Plan& p, int dtype, bool back, hipStream_t st) {
  if (dtype == 0) return p.width == 4 ? launch_t<float, 4>(a, p, back, st) : launch_t<float, 1>(a, p, back, st);
  return p.width == 8 ? launch_t<uint16_t, 8>(a, p, back, st) : launch_t<uint16_t, 1>(a, p, back, st);
}

}  // namespace

Plan plan(int64_t B, int64_t L, int64_t C, int64_t G, int dtype, bool vec, bool backward) {
  Plan p{vec ? (dtype == 0 ? 4 : 8) : 1, 0, 0, 0};
  const int64_t cg = C / G, e = dtype == 0 ? 4 : 2;
  const int most = backward ? 512 : 1024, deepest = backward ? 8 : 16;
  auto rows = [&](int64_t set, int threads) {  // 0: does not fit
    const int64_t nv = set / p.width, pass = nv <= threads ? threads / nv : 0;
    const int64_t r = pass ? (L + pass - 1) / pass : deepest + 1;
    return r <= deepest ? static_cast<int>(std::max<int64_t>(r, 1)) : 0;
  };
  int64_t set = std::lcm(cg, int64_t(p.width));
  if (set / cg > kMaxGroups || !rows(set, most)) return p;
  // rows of a set grow to 64 bytes, where that still fits
  for (int64_t f = 2; set * e < 64 && f <= C / set; ++f)
    if (C % (set * f) == 0 && set * f / cg <= kMaxGroups && rows(set * f, most)) {
      set *= f;
      f = 1;
    }
  const int threads = rows(set, 256) && rows(set, 256) <= 4 ? 256 : most;
  if (B > ((int64_t(1) << 32) - 1) / threads / (C / set)) return p;  // threads of one launch
  p.set = static_cast<int>(set);
  p.threads = threads;
  p.rows = rows(set, threads);
  return p;
}

// About 2048 blocks of the chip, at least 32 positions each.
int64_t chunk_positions(int64_t B, int64_t L, int64_t C) {
  const int64_t per_image = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, B * ((C + 1023) / 1024)));
  return std::max<int64_t>(32, (L + per_image - 1) / per_image);
}

int launch_group(const Args& a, const Plan& p, int dtype, hipStream_t st) { return launch_any(a, p, dtype, false, st); }

int launch_group_bwd(const Args& a, const Plan& p, int dtype, hipStream_t st) {
  int err = a.B > 0 && a.L > 0 ? launch_any(a, p, dtype, true, st) : 0;
  if (err || (!a.dw && !a.db)) return err;
  const int64_t count = a.B > 0 && a.L > 0 ? a.B * (p.rows > 0 ? 1 : a.chunks) : 0;
  hipLaunchKernelGGL(k_group_sums, dim3((2 * a.C + 63) / 64), dim3(1024), 0, st, a, count);
  return static_cast<int>(hipGetLastError());
}

}  // namespace group
}  // namespace ss2d
