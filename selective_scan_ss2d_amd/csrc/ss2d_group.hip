// The group norm with its activation, channels last, in two ways.
//
// A block holds whole groups of an image in registers: x is read once, its mean and then the squares
// about it are summed over the block, and y is written.  Where a group is too large for that, chunks
// of positions give every channel's mean and sum of squares about it, one block per group joins
// them, and another pass normalises.
// What bounds it is HBM where a block's loads of a few hundred KB are in flight at once: bf16, 64 maps of
// 56 x 56 x 192, 154 MB, 40 us (3.8 TB/s: one block of 1024 threads per CU loads, sums and writes in
// turn); fp32, 64 of 28 x 28 x 384, 154 MB forward 28 us, 231 MB backward 62 to 68 (its registers hold x
// and dy of 10 rows: 125, two blocks of 512 threads per CU).  In bfloat16 the backward's pieces of eight
// channels take 169 registers there, one block per CU.
#include <algorithm>
#include <numeric>

#include "ss2d_group.h"

namespace ss2d {
namespace group {
namespace {

// kV adjacent values as they come from memory: one 16-byte access, or one value.
template <typename T, int kV> struct Piece {
  static constexpr bool kWide = kV > 1;
  static constexpr int kWords = kWide ? 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWide) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (sizeof(T) == 4) {
      w[0] = __float_as_uint(*p);
    } else {
      w[0] = uint32_t(*p) << 16;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (!kWide) return __uint_as_float(w[0]);
    else return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  static __device__ __forceinline__ void store(T* p, const float* x) {
    if constexpr (kWide) {
      T v[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) v[i] = Elem<T>::from_f32(x[i]);
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    } else {
      *p = Elem<T>::from_f32(x[0]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // Conversions on either side of this are made twice rather than kept in registers between.
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
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

// Sums of every channel of a set over the rows of part[row][set], in part[0]: rows are folded by 8 at
// most, rows p, p + P, ... into row p, in place (row p is read by the thread that writes it alone).
template <int kThreads, int kParts>
__device__ __forceinline__ void fold(float (*part)[kThreads * kParts], int arrays, int set, int rows) {
  while (rows > 1) {
    const int P = (rows + 7) / 8;
    __syncthreads();
    for (int i = threadIdx.x; i < P * set; i += kThreads)
      for (int k = 0; k < arrays; ++k) {
        float v = part[k][i];
        for (int r = i + P * set; r < rows * set; r += P * set) v += part[k][r];
        part[k][i] = v;
      }
    rows = P;
  }
  __syncthreads();
}

// Every group's sum of row[set], over `count`, into out[group].
template <int kThreads>
__device__ __forceinline__ void group_sums(const float* row, int set, int cg, float count, float* out) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int g = wave; g < set / cg; g += kThreads / 64) {
    float v = 0.0f;
    for (int i = lane; i < cg; i += 64) v += row[g * cg + i];
    v = lane_sum<64>(v);
    if (lane == 0) out[g] = v / count;
  }
  __syncthreads();
}

// The mean and r of every group of the set, of values held in registers.
template <typename T, int kV, int kRows, int kThreads>
__device__ __forceinline__ void statistics(const Args& a, const Tile& t, Piece<T, kV>* x,
                                           float (*part)[kThreads * kV], float* mean, float* r) {
  const float count = static_cast<float>(a.L) * a.cg;
  const int at = t.row * a.set + t.cv * kV;
  float s[kV] = {};
#pragma unroll
  for (int i = 0; i < kRows; ++i)  // rows past the end hold zeros
#pragma unroll
    for (int k = 0; k < kV; ++k) s[k] += x[i].at(k);
#pragma unroll
  for (int k = 0; k < kV; ++k)
    if (t.on) part[0][at + k] = s[k];
  fold<kThreads, kV>(part, 1, a.set, t.pass);
  group_sums<kThreads>(part[0], a.set, a.cg, count, mean);
  float m[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    m[k] = mean[(t.cv * kV + k) / a.cg];
    s[k] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    x[i].renew();
    if (t.row + i * t.pass < a.L)
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const float d = x[i].at(k) - m[k];
        s[k] = fmaf(d, d, s[k]);
      }
  }
#pragma unroll
  for (int k = 0; k < kV; ++k)
    if (t.on) part[0][at + k] = s[k];
  fold<kThreads, kV>(part, 1, a.set, t.pass);
  group_sums<kThreads>(part[0], a.set, a.cg, count, r);
  for (int g = threadIdx.x; g < a.set / a.cg; g += kThreads) r[g] = 1.0f / sqrtf(r[g] + a.eps);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRows; ++i) x[i].renew();
}

constexpr int kMaxGroups = 256;  // of a set
// Rows of a thread that there are kernels for.  Two blocks of 512 threads fit a CU at 128 registers: the
// forward keeps to that at 20 rows (126), the backward at 10 in fp32 (125), but at 4 in bfloat16 (121; 6, 8
// and 10 take 137, 153 and 169).
constexpr int kDeepestBack = 10;
template <int... kRows> struct RowCounts {
  static int least(int64_t rows, int deepest) {  // 0: none holds as many
    int found = 0;
    ((found = !found && kRows <= deepest && rows <= kRows ? kRows : found), ...);
    return found;
  }
};
using Rows = RowCounts<1, 2, 4, 6, 8, 10, 14, 16, 20>;
int rows_of(int64_t rows, bool backward) { return Rows::least(rows, backward ? kDeepestBack : 20); }

template <typename T, int kV, int kRows, int kThreads>
__global__ __launch_bounds__(kThreads) void k_group(Args a) {
  __shared__ float part[1][kThreads * kV], mean[kMaxGroups], r[kMaxGroups];
  const unsigned id = xcd_local_order(blockIdx.x, gridDim.x);
  const int64_t b = id / a.sets;
  const int c0 = static_cast<int>(id % a.sets) * a.set;
  const Tile t = tile_of<kThreads>(a, kV);
  const int c = c0 + t.cv * kV;
  const int64_t base = b * a.L * a.C + c, step = int64_t(t.pass) * a.C;
  Piece<T, kV> x[kRows];
  const T* from = static_cast<const T*>(a.x) + base + int64_t(t.row) * a.C;
#pragma unroll
  for (int i = 0; i < kRows; ++i, from += step) {
    x[i].zero();
    if (t.on && t.row + i * t.pass < a.L) x[i].load(from);
  }
  statistics<T, kV, kRows, kThreads>(a, t, x, part, mean, r);
  if (a.stats)
    for (int g = threadIdx.x; g < a.set / a.cg; g += kThreads) {
      float* to = a.stats + (b * a.G + c0 / a.cg + g) * 2;
      to[0] = mean[g];
      to[1] = r[g];
    }
  if (!t.on) return;
  float m[kV], w[kV], bias[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int g = (t.cv * kV + k) / a.cg;
    m[k] = mean[g];
    w[k] = (a.w ? a.w[c + k] : 1.0f) * r[g];
    bias[k] = a.b ? a.b[c + k] : 0.0f;
  }
  T* to = static_cast<T*>(a.y) + base + int64_t(t.row) * a.C;
#pragma unroll
  for (int i = 0; i < kRows; ++i, to += step) {
    if (t.row + i * t.pass >= a.L) break;
    float v[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      v[k] = affine(x[i].at(k) - m[k], w[k], bias[k]);
      if (a.silu) v[k] = silu_f32(v[k]);
    }
    Piece<T, kV>::store(to, v);
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
  const int64_t base = b * a.L * a.C + c + int64_t(t.row) * a.C, step = int64_t(t.pass) * a.C;
  const T *from = static_cast<const T*>(a.x) + base, *dfrom = static_cast<const T*>(a.dy) + base;
  Piece<T, kV> xs[kRows], ds[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i, from += step, dfrom += step) {
    xs[i].zero();
    ds[i].zero();
    if (t.on && t.row + i * t.pass < a.L) {
      xs[i].load(from);
      ds[i].load(dfrom);
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
      const float* s = a.stats + (b * a.G + c0 / a.cg + g) * 2;
      mean[g] = s[0];
      r[g] = s[1];
    }
    __syncthreads();
  } else {
    statistics<T, kV, kRows, kThreads>(a, t, xs, part, mean, r);
  }
  float m[kV], rs[kV], sd[kV] = {}, sn[kV] = {};
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int g = (t.cv * kV + k) / a.cg;
    m[k] = mean[g];
    rs[k] = r[g];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (t.row + i * t.pass < a.L)
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const float n = (xs[i].at(k) - m[k]) * rs[k];
        float d = ds[i].at(k);
        if (a.silu) d *= slope(affine(n, w[k], bias[k]));
        sd[k] += d;
        sn[k] = fmaf(d, n, sn[k]);
        if constexpr (sizeof(T) == 4) ds[i].w[k] = __float_as_uint(d);  // else d is made again below
      }
    xs[i].renew();
    ds[i].renew();
  }
#pragma unroll
  for (int k = 0; k < kV; ++k)
    if (t.on) {
      part[0][t.row * a.set + t.cv * kV + k] = sd[k];
      part[1][t.row * a.set + t.cv * kV + k] = sn[k];
    }
  fold<kThreads, kV>(part, 2, a.set, t.pass);
  for (int i = threadIdx.x; i < a.set; i += kThreads) {
    const float wi = a.w ? a.w[c0 + i] : 1.0f, d = part[0][i], n = part[1][i];
    if (a.dw || a.db) {
      a.parts[(b * 2) * a.C + c0 + i] = d;
      a.parts[(b * 2 + 1) * a.C + c0 + i] = n;
    }
    part[0][i] = d * wi;
    part[1][i] = n * wi;
  }
  __syncthreads();
  const float count = static_cast<float>(a.L) * a.cg;
  group_sums<kThreads>(part[0], a.set, a.cg, count, mean);
  group_sums<kThreads>(part[1], a.set, a.cg, count, r);
  if (!t.on) return;
  T* to = static_cast<T*>(a.dx) + base;
  float se[kV], sx[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) {
    const int g = (t.cv * kV + k) / a.cg;
    se[k] = mean[g];
    sx[k] = r[g];
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i, to += step) {
    if (t.row + i * t.pass >= a.L) break;
    float v[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) {
      const float n = (xs[i].at(k) - m[k]) * rs[k];
      float d = ds[i].at(k);
      if (sizeof(T) != 4 && a.silu) d *= slope(affine(n, w[k], bias[k]));
      v[k] = rs[k] * (fmaf(d, w[k], -se[k]) - n * sx[k]);
    }
    Piece<T, kV>::store(to, v);
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

// One block per image and group joins its channels' parts of every chunk: f(first, second, chunk,
// channel within the group), summed over the block for every thread.  Eight items of a thread are
// loaded at once: with one wave and one load per group, 2048 chunks of a map of 256 x 256 x 256 took
// 200 us.
template <typename F> __device__ __forceinline__ float join_sum(const float* parts, const Args& a, float* waves, F f) {
  constexpr uint32_t kAhead = 8;
  const uint32_t items = static_cast<uint32_t>(a.chunks) * a.cg, threads = blockDim.x;
  float s = 0.0f;
  for (uint32_t i = threadIdx.x; i < items; i += kAhead * threads) {
    float x[kAhead], y[kAhead];
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k) {
      const uint32_t j = min(i + k * threads, items - 1);
      const float* at = parts + int64_t(j / a.cg) * 2 * a.C + j % a.cg;
      x[k] = at[0];
      y[k] = at[a.C];
    }
#pragma unroll
    for (uint32_t k = 0; k < kAhead; ++k) {
      const uint32_t j = i + k * threads;
      if (j < items) s += f(x[k], y[k], j / a.cg, j % a.cg);
    }
  }
  s = lane_sum<64>(s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0f;
  for (uint32_t w = 0; w < threads / 64; ++w) s += waves[w];
  return s;
}

// Its statistics from the chunks' means and sums of squares about them.
__global__ __launch_bounds__(1024) void k_group_join(Args a) {
  __shared__ float waves[16];
  const int64_t id = blockIdx.x, b = id / a.G;
  const float* parts = a.parts + b * a.chunks * 2 * a.C + id % a.G * a.cg;
  const float total = static_cast<float>(max(a.L, int64_t(1))) * a.cg;  // (without positions 0 / cg)
  auto positions = [&](uint32_t k) { return static_cast<float>(min(a.L - k * a.chunk, a.chunk)); };
  const float mean =
      join_sum(parts, a, waves, [&](float m, float, uint32_t k, uint32_t) { return positions(k) * m; }) / total;
  const float q = join_sum(parts, a, waves, [&](float m, float M2, uint32_t k, uint32_t) {
    return fmaf((m - mean) * (m - mean), positions(k), M2);
  }) / total;
  if (threadIdx.x == 0) {
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
      float f[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        f[k] = affine(v[i].at(k) - m[k], w[k], b[k]);
        if (a.silu) f[k] = silu_f32(f[k]);
      }
      Piece<T, kV>::store(y + (t + i * p.rows) * a.C, f);
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

// The means of e and e n of an image's group.
__global__ __launch_bounds__(1024) void k_group_bwd_join(Args a) {
  __shared__ float waves[16];
  const int64_t id = blockIdx.x, b = id / a.G;
  const int c0 = static_cast<int>(id % a.G) * a.cg;
  const float* parts = a.parts + b * a.chunks * 2 * a.C + c0;
  auto weight = [&](uint32_t c) { return a.w ? a.w[c0 + c] : 1.0f; };
  const float total = static_cast<float>(a.L) * a.cg;
  const float se =
      join_sum(parts, a, waves, [&](float d, float, uint32_t, uint32_t c) { return weight(c) * d; }) / total;
  const float sn =
      join_sum(parts, a, waves, [&](float, float n, uint32_t, uint32_t c) { return weight(c) * n; }) / total;
  if (threadIdx.x == 0) {
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
      float f[kV];
#pragma unroll
      for (int k = 0; k < kV; ++k) {
        const float n = (v[i].at(k) - m[k]) * r[k];
        float d = g[i].at(k);
        if (a.silu) d *= slope(affine(n, w[k], b[k]));
        f[k] = r[k] * (fmaf(d, w[k], -se[k]) - n * sn[k]);
      }
      Piece<T, kV>::store(dx + (t + i * p.rows) * a.C, f);
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

// The widest row of threads, of 256 down to 8 (32 of single values of rows of more than 16, which would
// be read in pieces of 32 bytes), whose blocks leave the fewest threads idle: bf16 64 x 3136 x 64 in one
// group, 8 of 32 threads at work and 8 of 8, 44.9 and 32.1 us; 256 x 7778 x 5, 5 of 32 and of 8, 99.9 and
// 41.1.
int lanes_of(int64_t C, int width) {
  const int64_t pieces = (C + width - 1) / width;
  int best = width == 1 && pieces > 16 ? 32 : 8;
  int64_t least = (pieces + best - 1) / best * best;
  for (int lanes = 2 * best; lanes <= 256; lanes *= 2) {
    const int64_t covered = (pieces + lanes - 1) / lanes * lanes;
    if (covered <= least) {
      least = covered;
      best = lanes;
    }
  }
  return best;
}

template <typename T, int kV, int kThreads, int kRows>
void launch_one(const Args& a, bool back, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.B * a.sets)), block(kThreads);
  if (!back) {
    hipLaunchKernelGGL((k_group<T, kV, kRows, kThreads>), grid, block, 0, st, a);
  } else {
    if constexpr (kThreads < 1024 && kRows <= kDeepestBack)
      hipLaunchKernelGGL((k_group_bwd<T, kV, kRows, kThreads>), grid, block, 0, st, a);
  }
}

template <typename T, int kV, int kThreads, int... kRows>
int launch_rows(const Args& a, int rows, bool back, hipStream_t st, RowCounts<kRows...>) {
  ((rows == kRows ? launch_one<T, kV, kThreads, kRows>(a, back, st) : void()), ...);
  return static_cast<int>(hipGetLastError());
}

template <typename T, int kV> int launch_t(const Args& a, const Plan& p, bool back, hipStream_t st) {
  if (p.rows > 0) {
    if (p.threads == 256) return launch_rows<T, kV, 256>(a, p.rows, back, st, Rows());
    if (p.threads == 512) return launch_rows<T, kV, 512>(a, p.rows, back, st, Rows());
    return launch_rows<T, kV, 1024>(a, p.rows, back, st, Rows());
  }
  const int lanes = lanes_of(a.C, kV), cblocks = (a.C + lanes * kV - 1) / (lanes * kV);
  const dim3 grid(static_cast<unsigned>(a.B * a.chunks * cblocks)), block(256);
  const dim3 groups(static_cast<unsigned>(a.B * a.G));
  int joined = 64;  // threads of a join, of eight items each
  while (joined < 1024 && joined * 8 < a.chunks * a.cg) joined *= 2;
  if (!a.given) {
    if (a.chunks > 0) hipLaunchKernelGGL((k_group_chunks<T, kV>), grid, block, 0, st, a, lanes, cblocks);
    hipLaunchKernelGGL(k_group_join, groups, dim3(joined), 0, st, a);
  }
  if (a.chunks == 0) return static_cast<int>(hipGetLastError());  // no positions: the statistics alone
  if (!back) {
    hipLaunchKernelGGL((k_group_apply<T, kV>), grid, block, 0, st, a, lanes, cblocks);
  } else {
    hipLaunchKernelGGL((k_group_bwd_chunks<T, kV>), grid, block, 0, st, a, lanes, cblocks);
    hipLaunchKernelGGL(k_group_bwd_join, groups, dim3(joined), 0, st, a);
    hipLaunchKernelGGL((k_group_bwd_apply<T, kV>), grid, block, 0, st, a, lanes, cblocks);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_any(const Args& a, const Plan& p, int dtype, bool back, hipStream_t st) {
  if (dtype == 0) return p.width == 4 ? launch_t<float, 4>(a, p, back, st) : launch_t<float, 1>(a, p, back, st);
  return p.width == 8 ? launch_t<uint16_t, 8>(a, p, back, st) : launch_t<uint16_t, 1>(a, p, back, st);
}

}  // namespace

// The channels of a block (whole groups of them, at most 1 KB of a row where more than one set is
// possible), its threads, and the rows of a thread: what the estimate below finds cheapest, or chunks
// where nothing fits (bf16 64 x 784 x 384: 22.9 us in registers, 40.4 by chunks).  It is fitted to 60
// shapes of 0.1 to 150 MB.  Its terms, with us per call on both sides:
//   threads and rows that hold nothing: bf16 128 x 196 x 768 in 32 groups, sets of 24, 48 and 96 channels,
//     58, 78 and 92% of the registers in use: 27.4, 27.3 and 23.1;
//   two blocks of 512 threads for every CU, or calls are as long as a thread has rows: 8 x 1024 x 512 by
//     1024, 512 and 256 threads, 2, 4 and 8 rows: 12.4, 13.2, 13.3; then wide pieces gain nothing, and
//     many threads cost: 1 x 256 x 256 by 32 blocks of 256 and by 8 of 1024: 6.8 and 10.0;
//   pieces of a row that lines hold in part: 64 x 1024 x 512, pieces of 32, 64 and 128 bytes: 36.5, 36.7,
//     29.9; fp32, 64, 128 and 256 bytes: 64.0, 54.9, 58.3 (the last by 1024 threads);
//   barriers of many threads: 100 x 100 x 1000, 10 rows of 256 threads and 5 of 512: 16.9 and 18.7;
//   the backward's registers: 64 x 1024 x 512 by 4 and 8 rows: 95 and 104; 1024 threads: 70 for 64.
Plan plan(int64_t B, int64_t L, int64_t C, int64_t G, int dtype, bool vec, bool backward) {
  Plan p{vec ? (dtype == 0 ? 4 : 8) : 1, 0, 0, 0};
  const int64_t cg = C / G, e = dtype == 0 ? 4 : 2, base = std::lcm(cg, int64_t(p.width));
  const double call = static_cast<double>(B) * L * C / p.width / (512 * 512);  // rows that fill the CUs
  double least = 1e30;
  for (int64_t set = base; set <= C && set / cg <= kMaxGroups && (set == base || set * e <= 1024); set += base) {
    if (C % set) continue;
    for (int threads = 256; threads <= (backward ? 512 : 1024); threads *= 2) {
      const int64_t nv = set / p.width, pass = threads / nv;
      if (pass == 0 || B > ((int64_t(1) << 32) - 1) / threads / (C / set)) continue;  // threads of one launch
      const int rows = rows_of((L + pass - 1) / pass, backward);
      if (!rows) continue;
      const double width = 1 + (backward ? 8.0 : 24.0) / (set * e);
      const double held = static_cast<double>(rows) * threads / (static_cast<double>(L) * nv);
      double cost = std::max(held * width, rows / call);
      if (backward) cost *= (1 + 0.035 * rows) * (threads > 256 ? 1.05 : 1.0);
      else cost *= threads > 512 ? 1.25 : threads > 256 ? 1.1 : rows > 10 ? 1.2 : 1.0;
      if (cost < least) {
        least = cost;
        p.set = static_cast<int>(set);
        p.threads = threads;
        p.rows = rows;
      }
    }
  }
  return p;
}

// About 1024 blocks of the chip, of eight positions of a thread at least (1 x 16,384 x 512, four and eight:
// 39 and 29 us).
int64_t chunk_positions(int64_t B, int64_t L, int64_t C, int dtype) {
  const int width = dtype == 0 ? 4 : 8, lanes = lanes_of(C, width);
  const int64_t blocks = B * ((C + lanes * width - 1) / (lanes * width));
  const int64_t per_image = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, blocks));
  return std::max<int64_t>(8 * 256 / lanes, (L + per_image - 1) / per_image);
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
