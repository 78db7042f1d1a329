// The block norm with channels last: rows of D values, 8 per thread, a row on 8 to 1024
// threads.  Every tensor is read once and written once; statistics, gate and both norms run
// on the values in registers, the means and squares in two passes over them.  Bound by HBM.
// 8 values per thread are one 16-byte load of bfloat16, and the narrowest rows still fill a wave
// with 8 of them.  602112 rows of 64 with gate, bfloat16: 38 us in the kernel (6.0 TB/s, part of
// it from the last-level cache).  The backward holds the sums of its rows' four vectors in
// registers and loads the next row while it computes: 25216 rows of 768: 103 us, of a floor of
// 62; with LDS permutes for the sums 124, the loads one behind the other and two barriers per sum
// as well 180.  Above D = 4096 a row takes 1024 threads of 128 registers, which the backward exceeds
// by 86 to 187: 4704 rows of 8192, bfloat16 with an fp32 residual stream: 521 us of a floor of 138
// (forward 140 of 92), where 9408 rows of 4096 take 193 (92).
#include <algorithm>

#include "ss2d_norm.h"

namespace ss2d {
namespace norm {
namespace {

constexpr int kV = 8;  // values per thread

// A thread's 8 values of a row as they come from memory.  Loading and converting are apart, so
// that all loads of a row are on their way before the first is waited for.
template <typename T, bool kVec> struct Raw { T v[kV]; };
template <typename T> struct Raw<T, true> { uint4 u[sizeof(T) / 2]; };

__device__ __forceinline__ void unpack(const Raw<uint16_t, true>& r, float* x) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float, true>& r, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.u[i].x);
    x[4 * i + 1] = __uint_as_float(r.u[i].y);
    x[4 * i + 2] = __uint_as_float(r.u[i].z);
    x[4 * i + 3] = __uint_as_float(r.u[i].w);
  }
}
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T, false>& r, float* x) {
#pragma unroll
  for (int i = 0; i < kV; ++i) x[i] = Elem<T>::to_f32(r.v[i]);
}

// A thread's columns of a row: kVec, 8 adjacent ones (rows on 16 bytes, D a multiple of 8);
// else every kLanes-th.
template <int kLanes, bool kVec>
struct Row {
  int lane, D;
  __device__ __forceinline__ int col(int i) const { return kVec ? lane * kV + i : lane + kLanes * i; }
  __device__ __forceinline__ bool in(int i) const { return col(kVec ? 0 : i) < D; }
  template <typename T>
  __device__ __forceinline__ void fetch(const void* base, int64_t row, Raw<T, kVec>& r) const {
    const T* p = static_cast<const T*>(base) + row * D;
    if constexpr (kVec) {
      const uint4* q = reinterpret_cast<const uint4*>(p + (in(0) ? lane * kV : 0));
#pragma unroll
      for (int i = 0; i < int(sizeof(T) / 2); ++i) r.u[i] = q[i];
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) r.v[i] = p[in(i) ? col(i) : 0];
    }
  }
  template <typename T>
  __device__ __forceinline__ void take(const Raw<T, kVec>& r, float* x) const {
    unpack(r, x);
#pragma unroll
    for (int i = 0; i < kV; ++i) x[i] = in(i) ? x[i] : 0.0f;
  }
  template <typename T>
  __device__ __forceinline__ void load(const void* base, int64_t row, float* x) const {
    Raw<T, kVec> r;
    fetch<T>(base, row, r);
    take<T>(r, x);
  }
  template <typename T>
  __device__ __forceinline__ void store(void* base, int64_t row, const float* x) const {
    T* p = static_cast<T*>(base) + row * D;
    if constexpr (kVec) {
      if (!in(0)) return;
      T v[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) v[i] = Elem<T>::from_f32(x[i]);
#pragma unroll
      for (unsigned i = 0; i < sizeof(v) / 16; ++i)
        reinterpret_cast<uint4*>(p + lane * kV)[i] = reinterpret_cast<const uint4*>(v)[i];
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (in(i)) p[col(i)] = Elem<T>::from_f32(x[i]);
    }
  }
};

// Sums two values over the kLanes threads of a row.  Rows on several waves meet in LDS, in two
// buffers in turn: one barrier then is enough.
template <int kLanes>
struct RowSum {
  static constexpr int kThreads = kLanes > 256 ? kLanes : 256, kW = kLanes > 64 ? kLanes / 64 : 1;
  float2 (*shared)[kThreads / 64];
  int turn = 0;
  __device__ __forceinline__ void operator()(float& a, float& b) {
    a = lane_sum<(kLanes < 64 ? kLanes : 64)>(a);
    b = lane_sum<(kLanes < 64 ? kLanes : 64)>(b);
    if constexpr (kLanes > 64) {
      const int wave = threadIdx.x >> 6;
      float2* buffer = shared[turn];
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) buffer[wave] = make_float2(a, b);
      __syncthreads();
      const int first = wave / kW * kW;
      a = b = 0.0f;
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        a += buffer[first + i].x;
        b += buffer[first + i].y;
      }
    }
  }
};

// x becomes (x - mean) r (layer) or x r; returns r.  Two passes over the registers.
template <int kLanes, bool kVec>
__device__ __forceinline__ float unit(const Row<kLanes, kVec>& row, float* x, bool layer, float eps,
                                      RowSum<kLanes>& sum) {
  const float inv = 1.0f / static_cast<float>(row.D);
  float s = 0.0f, q = 0.0f, none = 0.0f;
  if (layer) {
#pragma unroll
    for (int i = 0; i < kV; ++i) s += x[i];
    sum(s, none);
    s *= inv;
#pragma unroll
    for (int i = 0; i < kV; ++i) x[i] = row.in(i) ? x[i] - s : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) q = fmaf(x[i], x[i], q);
  sum(q, none);
  const float r = 1.0f / sqrtf(fmaf(q, inv, eps));
#pragma unroll
  for (int i = 0; i < kV; ++i) x[i] *= r;
  return r;
}

// From the gradient d at unit(x)'s output to the one at its input.
template <int kLanes, bool kVec>
__device__ __forceinline__ void through(const Row<kLanes, kVec>& row, float* d, const float* x,
                                        float r, bool layer, RowSum<kLanes>& sum) {
  const float inv = 1.0f / static_cast<float>(row.D);
  float sx = 0.0f, s = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    sx = fmaf(d[i], x[i], sx);
    s += d[i];
  }
  sum(sx, s);
  sx *= inv;
  s = layer ? s * inv : 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) d[i] = row.in(i) ? r * (d[i] - fmaf(x[i], sx, s)) : 0.0f;
}

template <typename T, typename Y, int kLanes, bool kVec>
__global__ __launch_bounds__(kLanes > 256 ? kLanes : 256) void k_norm(Args a) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256, kRows = kThreads / kLanes;
  __shared__ float2 shared[2][kThreads / 64];
  RowSum<kLanes> sum{shared};
  const Row<kLanes, kVec> row{static_cast<int>(threadIdx.x % kLanes), a.D};
  float wp[kV], bp[kV], wn[kV], bn[kV], sc[kV];
  if (a.w_post) row.template load<float>(a.w_post, 0, wp);
  if (a.b_post) row.template load<float>(a.b_post, 0, bp);
  if (a.w_pre) row.template load<float>(a.w_pre, 0, wn);
  if (a.b_pre) row.template load<float>(a.b_pre, 0, bn);
  if (a.scale) row.template load<float>(a.scale, 0, sc);
  const int64_t rows = a.B * a.L;
  for (int64_t base = int64_t(blockIdx.x) * kRows; base < rows; base += int64_t(gridDim.x) * kRows) {
    const int64_t at = base + threadIdx.x / kLanes;
    const bool on = at < rows;            // rows past the end run along for the barriers
    const int64_t i0 = on ? at : rows - 1;
    Raw<T, kVec> rh, rz;
    Raw<Y, kVec> rr;
    row.template fetch<T>(a.h, i0, rh);
    if (a.z) row.template fetch<T>(a.z, i0, rz);
    if (a.residual) row.template fetch<Y>(a.residual, i0, rr);
    if (a.scale && a.G > 1) row.template load<float>(a.scale, i0 / a.group, sc);
    float x[kV], z[kV], res[kV];
    row.template take<T>(rh, x);
    if (a.z) row.template take<T>(rz, z);
    if (a.residual) row.template take<Y>(rr, res);
    if (a.w_post) {
      unit(row, x, a.layer, a.eps, sum);
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] = a.b_post ? fmaf(x[i], wp[i], bp[i]) : x[i] * wp[i];
    }
    if (a.z) {
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] *= gate_value(z[i], sigmoid_f32(z[i]));
    }
    if (a.scale) {
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] *= sc[i];
    }
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] += res[i];
    }
    if (a.y && on) row.template store<Y>(a.y, at, x);
    if (a.w_pre) {
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] = row.in(i) ? x[i] : 0.0f;
      unit(row, x, a.layer, a.eps, sum);
#pragma unroll
      for (int i = 0; i < kV; ++i) x[i] = a.b_pre ? fmaf(x[i], wn[i], bn[i]) : x[i] * wn[i];
      if (on) row.template store<T>(a.n, at, x);
    }
  }
}

// Adds a block's sums of one vector over its concurrent rows and writes them.
template <int kLanes, bool kVec>
__device__ __forceinline__ void write_sums(const Row<kLanes, kVec>& row, const float* x, float* out,
                                           float* buffer) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256, kRows = kThreads / kLanes;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (row.in(i)) out[row.col(i)] = x[i];
  } else {
    __syncthreads();
    float* mine = buffer + threadIdx.x / kLanes * (kLanes * kV);
#pragma unroll
    for (int i = 0; i < kV; ++i) mine[row.col(i)] = x[i];
    __syncthreads();
    for (int c = threadIdx.x; c < row.D; c += kThreads) {
      float s = 0.0f;
      for (int r = 0; r < kRows; ++r) s += buffer[r * (kLanes * kV) + c];
      out[c] = s;
    }
  }
}

// A block takes part of one group's rows or several whole groups, so that res_scale's
// gradient is summed per group; the other sums run over all of a block's rows.
template <typename T, typename Y, int kLanes, bool kVec>
__global__ __launch_bounds__(kLanes > 256 ? kLanes : 256) void k_norm_bwd(Args a) {
  constexpr int kThreads = kLanes > 256 ? kLanes : 256, kRows = kThreads / kLanes;
  __shared__ float2 shared[2][kThreads / 64];
  RowSum<kLanes> sum{shared};
  __shared__ float buffer[kRows == 1 ? 1 : kThreads * kV];
  const Row<kLanes, kVec> row{static_cast<int>(threadIdx.x % kLanes), a.D};
  float wp[kV], bp[kV], wn[kV], sc[kV];
  if (a.w_post) row.template load<float>(a.w_post, 0, wp);
  if (a.b_post) row.template load<float>(a.b_post, 0, bp);
  if (a.w_pre) row.template load<float>(a.w_pre, 0, wn);
  float dwp[kV] = {}, dbp[kV] = {}, dwn[kV] = {}, dbn[kV] = {};
  const int64_t part = blockIdx.x % a.blocks_per_group;
  const int64_t g0 = blockIdx.x / a.blocks_per_group * a.groups_per_block;
  const int64_t g1 = min(a.G, g0 + a.groups_per_block);
  for (int64_t g = g0; g < g1; ++g) {
    float dsc[kV] = {};
    if (a.scale) row.template load<float>(a.scale, g, sc);
    const int64_t end = (g + 1) * a.group;
    const int64_t step = a.blocks_per_group * kRows;
    Raw<T, kVec> rh, rz, rn;
    Raw<Y, kVec> rd, ry;
    auto fetch = [&](int64_t base) {
      const int64_t i = min(base + threadIdx.x / kLanes, end - 1);
      row.template fetch<T>(a.h, i, rh);
      if (a.z) row.template fetch<T>(a.z, i, rz);
      if (a.dy) row.template fetch<Y>(a.dy, i, rd);
      if (a.w_pre) {
        row.template fetch<Y>(a.y, i, ry);
        row.template fetch<T>(a.dn, i, rn);
      }
    };
    int64_t base = g * a.group + part * kRows;
    if (base < end) fetch(base);
    for (; base < end; base += step) {
      const int64_t at = base + threadIdx.x / kLanes;
      const bool on = at < end;  // rows past the end run along for the barriers
      float d[kV] = {}, x[kV], e[kV], hx[kV], z[kV];
      row.template take<T>(rh, hx);
      if (a.z) row.template take<T>(rz, z);
      if (a.dy) row.template take<Y>(rd, d);
      if (a.w_pre) {
        row.template take<Y>(ry, x);
        row.template take<T>(rn, e);
      }
      fetch(base + step);  // the next row's values come in meanwhile
      if (a.w_pre) {
        const float r = unit(row, x, a.layer, a.eps, sum);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          if (on) {
            dwn[i] = fmaf(e[i], x[i], dwn[i]);
            dbn[i] += e[i];
          }
          e[i] *= wn[i];
        }
        through(row, e, x, r, a.layer, sum);
#pragma unroll
        for (int i = 0; i < kV; ++i) d[i] += e[i];
      }
      if (a.dres && on) row.template store<Y>(a.dres, at, d);
      float r = 0.0f;
      if (a.w_post) r = unit(row, hx, a.layer, a.eps, sum);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        float p = hx[i];
        if (a.w_post) p = a.b_post ? fmaf(p, wp[i], bp[i]) : p * wp[i];
        float gated = p, sg = 0.0f, gv = 1.0f;
        if (a.z) {
          sg = sigmoid_f32(z[i]);
          gv = gate_value(z[i], sg);
          gated = p * gv;
        }
        if (a.scale) {
          if (on) dsc[i] = fmaf(d[i], gated, dsc[i]);
          d[i] *= sc[i];
        }
        if (a.z) {
          e[i] = d[i] * p * gate_slope(z[i], sg);
          d[i] *= gv;
        }
        if (a.w_post) {
          if (on) {
            dwp[i] = fmaf(d[i], hx[i], dwp[i]);
            dbp[i] += d[i];
          }
          d[i] *= wp[i];
        }
      }
      if (a.z && on) row.template store<T>(a.dz, at, e);
      if (a.w_post) {
#pragma unroll
        for (int i = 0; i < kV; ++i) d[i] = row.in(i) ? d[i] : 0.0f;
        through(row, d, hx, r, a.layer, sum);
      }
      if (on) row.template store<T>(a.dh, at, d);
    }
    if (a.scale)
      write_sums(row, dsc, a.scale_parts + (g * a.blocks_per_group + part) * a.D, buffer);
  }
  float* out = a.parts + int64_t(blockIdx.x) * kSums * a.D;
  if (a.dw_post) write_sums(row, dwp, out, buffer);
  if (a.db_post) write_sums(row, dbp, out + a.D, buffer);
  if (a.dw_pre) write_sums(row, dwn, out + 2 * a.D, buffer);
  if (a.db_pre) write_sums(row, dbn, out + 3 * a.D, buffer);
}

// Adds partial sums in a fixed order: out[v][c] = sum over b of parts[(b, v)][c], 64 columns
// and 16 groups of b per block.
struct Sums {
  const float* parts;
  float* out[kSums];
  int64_t count, stride, first;  // partial vectors; floats from one to the next; from v to v + 1
  int D;
};
__global__ __launch_bounds__(1024) void k_norm_sums(Sums s) {
  __shared__ float buffer[16][64];
  float* out = s.out[0];
  if (blockIdx.y == 1) out = s.out[1];
  if (blockIdx.y == 2) out = s.out[2];
  if (blockIdx.y == 3) out = s.out[3];
  if (!out) return;
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  const float* p = s.parts + blockIdx.y * s.first + c;
  float x[8] = {};
  if (c < s.D) {
    int64_t b = g;
    for (; b + 112 < s.count; b += 128)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += p[(b + 16 * i) * s.stride];
    for (; b < s.count; b += 16) x[0] += p[b * s.stride];
  }
  buffer[g][threadIdx.x & 63] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  __syncthreads();
  if (g == 0 && c < s.D) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += buffer[i][threadIdx.x];
    out[c] = t;
  }
}

// The same per group of res_scale: out[g][c] = sum over its parts, 64 columns and a group of
// parts per wave of a block.
__global__ __launch_bounds__(1024) void k_norm_group_sums(const float* parts, float* out, int64_t count,
                                                          int D) {
  __shared__ float buffer[16][64];
  const int c = blockIdx.y * 64 + (threadIdx.x & 63), w = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t g = blockIdx.x;
  const float* p = parts + g * count * D + c;
  float x[8] = {};
  if (c < D) {
    int64_t b = w;
    for (; b + 7 * waves < count; b += 8 * waves)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += p[(b + i * waves) * D];
    for (; b < count; b += waves) x[0] += p[b * D];
  }
  buffer[w][threadIdx.x & 63] = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  __syncthreads();
  if (w == 0 && c < D) {
    float t = 0.0f;
    for (int i = 0; i < waves; ++i) t += buffer[i][threadIdx.x];
    out[g * D + c] = t;
  }
}

int lanes_of(int D) {
  int lanes = 8;
  while (lanes * kV < D) lanes *= 2;
  return lanes;
}

template <typename T, typename Y, int kLanes, bool kVec>
void launch(const Args& a, bool bwd, int64_t blocks, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(blocks)), block(kLanes > 256 ? kLanes : 256);
  if (bwd) hipLaunchKernelGGL((k_norm_bwd<T, Y, kLanes, kVec>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_norm<T, Y, kLanes, kVec>), grid, block, 0, st, a);
}

template <typename T, typename Y, bool kVec>
int launch_lanes(const Args& a, bool bwd, int64_t blocks, hipStream_t st) {
  switch (lanes_of(a.D)) {
    case 8: launch<T, Y, 8, kVec>(a, bwd, blocks, st); break;
    case 16: launch<T, Y, 16, kVec>(a, bwd, blocks, st); break;
    case 32: launch<T, Y, 32, kVec>(a, bwd, blocks, st); break;
    case 64: launch<T, Y, 64, kVec>(a, bwd, blocks, st); break;
    case 128: launch<T, Y, 128, kVec>(a, bwd, blocks, st); break;
    case 256: launch<T, Y, 256, kVec>(a, bwd, blocks, st); break;
    case 512: launch<T, Y, 512, kVec>(a, bwd, blocks, st); break;
    default: launch<T, Y, 1024, kVec>(a, bwd, blocks, st); break;
  }
  return static_cast<int>(hipGetLastError());
}

template <bool kVec>
int launch_types(const Args& a, int dtype, int ytype, bool bwd, int64_t blocks, hipStream_t st) {
  if (dtype == 0) return launch_lanes<float, float, kVec>(a, bwd, blocks, st);
  if (ytype == 0) return launch_lanes<uint16_t, float, kVec>(a, bwd, blocks, st);
  return launch_lanes<uint16_t, uint16_t, kVec>(a, bwd, blocks, st);
}

int64_t rows_of_block(int D) {
  const int lanes = lanes_of(D);
  return lanes > 256 ? 1 : 256 / lanes;
}

}  // namespace

int launch_norm_first(const Args& a, int dtype, int ytype, bool vec, bool bwd, int64_t blocks,
                      hipStream_t st);
int64_t tiles_first(const Args& a, bool bwd);

int launch_norm(const Args& a, int dtype, int ytype, bool first, bool vec, hipStream_t st) {
  if (first) return launch_norm_first(a, dtype, ytype, vec, false, 0, st);
  const int64_t rows = a.B * a.L, per = rows_of_block(a.D);
  const int64_t blocks = std::min<int64_t>((rows + per - 1) / per, 256 * 8);
  return vec ? launch_types<true>(a, dtype, ytype, false, blocks, st)
             : launch_types<false>(a, dtype, ytype, false, blocks, st);
}

// About 2 blocks per CU, what their registers allow, each with at least 4 rounds of its
// concurrent rows where there are that many (25216 rows of 768: 102 us and 9 for the sums; with
// twice the blocks 104 and 11); small groups share a block.
int64_t plan_norm_bwd(Args* a, bool first) {
  constexpr int64_t kBlocks = 512;
  const int64_t per = first ? 1 : rows_of_block(a->D);
  const int64_t rounds = first ? tiles_first(*a, true) : (a->group + per - 1) / per;  // of a group
  a->groups_per_block = 1;
  a->blocks_per_group = std::max<int64_t>(1, std::min((rounds + 3) / 4, kBlocks / a->G));
  if (a->G > kBlocks) a->groups_per_block = (a->G + kBlocks - 1) / kBlocks;
  return (a->G + a->groups_per_block - 1) / a->groups_per_block * a->blocks_per_group;
}

int launch_norm_bwd(const Args& a, int dtype, int ytype, bool first, bool vec, hipStream_t st) {
  const int64_t blocks = (a.G + a.groups_per_block - 1) / a.groups_per_block * a.blocks_per_group;
  if (first) return launch_norm_first(a, dtype, ytype, vec, true, blocks, st);
  return vec ? launch_types<true>(a, dtype, ytype, true, blocks, st)
             : launch_types<false>(a, dtype, ytype, true, blocks, st);
}

int launch_norm_sums(const Args& a, int64_t blocks, hipStream_t st) {
  if (a.dw_post || a.db_post || a.dw_pre || a.db_pre) {
    Sums s{a.parts, {a.dw_post, a.db_post, a.dw_pre, a.db_pre}, blocks, int64_t(kSums) * a.D, a.D,
           a.D};
    hipLaunchKernelGGL(k_norm_sums, dim3((a.D + 63) / 64, kSums), dim3(1024), 0, st, s);
  }
  if (a.dscale && a.scale_parts != a.dscale)
    hipLaunchKernelGGL(k_norm_group_sums, dim3(static_cast<unsigned>(a.G), (a.D + 63) / 64),
                       dim3(a.blocks_per_group >= 64 ? 1024 : 256), 0, st, a.scale_parts, a.dscale,
                       a.blocks_per_group, a.D);
  return static_cast<int>(hipGetLastError());
}

}  // namespace norm
}  // namespace ss2d
