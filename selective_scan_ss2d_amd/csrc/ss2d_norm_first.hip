// The block norm with channels first, (B, D, L): a block takes a tile of adjacent positions
// and all channels, 16 lanes across the positions and the other threads across the channels;
// sums over the channels run in registers, across a wave and through LDS.  Every tensor is
// read once and written once.  Bound by HBM up to D = 192.  64 maps of 192 x 56 x 56, bfloat16 with an
// fp32 residual stream: 122 us, of a floor of 92; blocks of 512 threads at 128 registers, two per CU
// (one, at 134 registers: 184 us; 256 threads with 12 channels each: 163).  Wider maps (as many
// values, L = 784) take 183 us at D = 256, 197 at 384 and 261 at 768: one block per CU, narrower tiles.
// The backward takes 312 us of a floor of 138 at D = 192, 377 at 384, and is far from it above:
// a thread's channels with their five sums do not fit the 128 registers that 1024 threads leave
// each, 40 of them go to scratch for D 385 to 512 (538 us), 150 to 180 up to 768 (824 us) and 320 to
// 340 up to 1024 (1012 us).
#include <algorithm>

#include "ss2d_norm.h"

namespace ss2d {
namespace norm {
namespace {

constexpr int kP = 16;  // lanes across the positions

template <typename T, int kN> struct alignas(sizeof(T) * kN) Pack { T v[kN]; };
// A pack as one word of memory.
template <int kBytes> struct WordOf { using type = uint32_t __attribute__((ext_vector_type(kBytes / 4))); };
template <> struct WordOf<2> { using type = uint16_t; };
template <> struct WordOf<4> { using type = uint32_t; };
template <typename T, int kN> using Word = typename WordOf<sizeof(T) * kN>::type;

template <typename T>
using Global = __attribute__((address_space(1))) T*;

// A thread's kVec positions of a tile (adjacent with kWide: L a multiple of kVec, planes
// aligned; else every 16th) and kC channels, every kGroups-th.  Addresses are a base that all
// threads share, per channel, and a 32-bit offset of the thread (kGroups L 4 bytes fit).
template <int kThreads, int kC, int kVec, bool kWide>
struct Tile {
  static constexpr int kGroups = kThreads / kP;
  int lane, group, D;
  int64_t L;
  int pos;  // first position of this thread
  __device__ __forceinline__ int channel(int i) const { return group + kGroups * i; }
  __device__ __forceinline__ int at(int j) const { return pos + (kWide ? j : kP * j); }
  __device__ __forceinline__ bool in(int j) const { return at(j) < L; }
  template <typename T>
  __device__ __forceinline__ Global<T> base_of(T* base, int64_t image, int i) const {
    return (Global<T>)(base + (image * D + (kGroups * i < D ? kGroups * i : 0)) * L);
  }
  __device__ __forceinline__ uint32_t offset(int p) const {
    return static_cast<uint32_t>(group) * static_cast<uint32_t>(L) + static_cast<uint32_t>(p);
  }
  // Loading and converting are apart and free of conditions, so that all loads of a tile are on
  // their way before the first is waited for; what is out of range reads the base's first value.
  template <typename T>
  __device__ __forceinline__ void fetch(const void* base, int64_t image, int i, Pack<T, kVec>& r) const {
    const Global<const T> p = base_of(static_cast<const T*>(base), image, i);
    const bool on = channel(i) < D;
    if constexpr (kWide) {
      const Word<T, kVec> u = *(Global<const Word<T, kVec>>)(p + (on && in(0) ? offset(pos) : 0u));
      __builtin_memcpy(&r, &u, sizeof(r));
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) r.v[j] = p[on && in(j) ? offset(at(j)) : 0u];
    }
  }
  template <typename T>
  __device__ __forceinline__ void take(const Pack<T, kVec>& r, int i, float* x) const {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      x[j] = channel(i) < D && in(kWide ? 0 : j) ? Elem<T>::to_f32(r.v[j]) : 0.0f;
  }
  template <typename T>
  __device__ __forceinline__ void store(void* base, int64_t image, int i, const float* x) const {
    if (channel(i) >= D) return;
    const Global<T> p = base_of(static_cast<T*>(base), image, i);
    if constexpr (kWide) {
      if (!in(0)) return;
      Pack<T, kVec> u;
#pragma unroll
      for (int j = 0; j < kVec; ++j) u.v[j] = Elem<T>::from_f32(x[j]);
      *(Global<Word<T, kVec>>)(p + offset(pos)) = __builtin_bit_cast(Word<T, kVec>, u);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (in(j)) p[offset(at(j))] = Elem<T>::from_f32(x[j]);
    }
  }
  __device__ __forceinline__ float channel_value(const float* w, int i) const {
    return channel(i) < D ? w[channel(i)] : 0.0f;
  }
};

// Sums a[j] and b[j] over the channel groups: across the wave's four, then the waves'.
template <int kThreads, int kVec>
__device__ __forceinline__ void channel_sum2(float* a, float* b, float2* shared) {
  constexpr int kWaves = kThreads / 64;
  const int lane = threadIdx.x & (kP - 1), wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    a[j] = add_across<32>(add_across<16>(a[j]));
    b[j] = add_across<32>(add_across<16>(b[j]));
  }
  __syncthreads();  // the last use of `shared` is over
  if ((threadIdx.x & 63) < kP)
#pragma unroll
    for (int j = 0; j < kVec; ++j) shared[(wave * kVec + j) * kP + lane] = make_float2(a[j], b[j]);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    a[j] = b[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float2 u = shared[(w * kVec + j) * kP + lane];
      a[j] += u.x;
      b[j] += u.y;
    }
  }
}

// x becomes (x - mean) r (layer) or x r along the channels; r of each position, 0 for
// positions past the end (whose values are 0).
template <int kThreads, int kC, int kVec, bool kWide>
__device__ __forceinline__ void unit(const Tile<kThreads, kC, kVec, kWide>& t, float (*x)[kVec],
                                     float* r, bool layer, float eps, float2* shared) {
  const float inv = 1.0f / static_cast<float>(t.D);
  float s[kVec] = {}, q[kVec] = {};
  if (layer) {
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) s[j] += x[i][j];
    channel_sum2<kThreads, kVec>(s, q, shared);
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) x[i][j] = t.channel(i) < t.D ? x[i][j] - s[j] * inv : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) s[j] = q[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) q[j] = fmaf(x[i][j], x[i][j], q[j]);
  channel_sum2<kThreads, kVec>(q, s, shared);
#pragma unroll
  for (int j = 0; j < kVec; ++j) r[j] = t.in(j) ? 1.0f / sqrtf(fmaf(q[j], inv, eps)) : 0.0f;
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[i][j] *= r[j];
}

// From the gradient d at unit(x)'s output to the one at its input.
template <int kThreads, int kC, int kVec, bool kWide>
__device__ __forceinline__ void through(const Tile<kThreads, kC, kVec, kWide>& t, float (*d)[kVec],
                                        const float (*x)[kVec], const float* r, bool layer,
                                        float2* shared) {
  const float inv = 1.0f / static_cast<float>(t.D);
  float sx[kVec] = {}, s[kVec] = {};
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      sx[j] = fmaf(d[i][j], x[i][j], sx[j]);
      s[j] += d[i][j];
    }
  channel_sum2<kThreads, kVec>(sx, s, shared);
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      d[i][j] = r[j] * (d[i][j] - fmaf(x[i][j], sx[j] * inv, layer ? s[j] * inv : 0.0f));
}

template <typename T, typename Y, int kThreads, int kC, int kVec, bool kWide>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(kC * kVec <= 24 ? 4 : 2)))
void k_norm_first(Args a) {
  __shared__ float2 shared[kThreads / 64 * kVec * kP];
  Tile<kThreads, kC, kVec, kWide> t;
  t.lane = threadIdx.x & (kP - 1);
  t.group = threadIdx.x / kP;
  t.D = a.D;
  t.L = a.L;
  const int64_t per = (a.L + kP * kVec - 1) / (kP * kVec), tiles = a.B * per;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t image = tile / per;
    t.pos = static_cast<int>(tile - image * per) * (kP * kVec) + t.lane * (kWide ? kVec : 1);
    float x[kC][kVec], r[kVec];
    Pack<T, kVec> rh[kC], rz[kC];
    Pack<Y, kVec> rr[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) t.template fetch<T>(a.h, image, i, rh[i]);
    if (a.z)
#pragma unroll
      for (int i = 0; i < kC; ++i) t.template fetch<T>(a.z, image, i, rz[i]);
    if (a.residual)
#pragma unroll
      for (int i = 0; i < kC; ++i) t.template fetch<Y>(a.residual, image, i, rr[i]);
#pragma unroll
    for (int i = 0; i < kC; ++i) t.template take<T>(rh[i], i, x[i]);
    if (a.w_post) unit(t, x, r, a.layer, a.eps, shared);
    const float* scale = a.scale ? a.scale + image / a.group * a.D : nullptr;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const float w = a.w_post ? t.channel_value(a.w_post, i) : 1.0f;
      const float b = a.b_post ? t.channel_value(a.b_post, i) : 0.0f;
      const float s = scale ? t.channel_value(scale, i) : 1.0f;
      float z[kVec], res[kVec];
      if (a.z) t.template take<T>(rz[i], i, z);
      if (a.residual) t.template take<Y>(rr[i], i, res);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float p = a.w_post ? fmaf(x[i][j], w, b) : x[i][j];
        if (a.z) p *= gate_value(z[j], sigmoid_f32(z[j]));
        if (scale) p *= s;
        if (a.residual) p += res[j];
        x[i][j] = p;
      }
      if (a.y) t.template store<Y>(a.y, image, i, x[i]);
    }
    if (a.w_pre) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[i][j] = t.in(j) && t.channel(i) < a.D ? x[i][j] : 0.0f;
      unit(t, x, r, a.layer, a.eps, shared);
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const float w = t.channel_value(a.w_pre, i);
        const float b = a.b_pre ? t.channel_value(a.b_pre, i) : 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[i][j] = fmaf(x[i][j], w, b);
        t.template store<T>(a.n, image, i, x[i]);
      }
    }
  }
}

// Adds a channel's sums over the 16 lanes of its positions and writes them.
template <int kThreads, int kC, int kVec, bool kWide>
__device__ __forceinline__ void write_sums(const Tile<kThreads, kC, kVec, kWide>& t, const float* x,
                                           float* out) {
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const float s = lane_sum<kP>(x[i]);
    if (t.lane == 0 && t.channel(i) < t.D) out[t.channel(i)] = s;
  }
}

template <typename T, typename Y, int kThreads, int kC, int kVec, bool kWide>
__global__ __launch_bounds__(kThreads) void k_norm_first_bwd(Args a) {
  __shared__ float2 shared[kThreads / 64 * kVec * kP];
  Tile<kThreads, kC, kVec, kWide> t;
  t.lane = threadIdx.x & (kP - 1);
  t.group = threadIdx.x / kP;
  t.D = a.D;
  t.L = a.L;
  const int64_t per = (a.L + kP * kVec - 1) / (kP * kVec), tiles = a.group * per;
  float dwp[kC] = {}, dbp[kC] = {}, dwn[kC] = {}, dbn[kC] = {};
  const int64_t part = blockIdx.x % a.blocks_per_group;
  const int64_t g0 = blockIdx.x / a.blocks_per_group * a.groups_per_block;
  const int64_t g1 = min(a.G, g0 + a.groups_per_block);
  for (int64_t g = g0; g < g1; ++g) {
    float dsc[kC] = {};
    const float* scale = a.scale ? a.scale + g * a.D : nullptr;
    for (int64_t tile = part; tile < tiles; tile += a.blocks_per_group) {
      const int64_t image = g * a.group + tile / per;
      t.pos = static_cast<int>(tile % per) * (kP * kVec) + t.lane * (kWide ? kVec : 1);
      float x[kC][kVec], d[kC][kVec], r[kVec];
      Pack<T, kVec> rh[kC], rz[kC];
      Pack<Y, kVec> rd[kC];
      if (a.w_pre) {
        Pack<Y, kVec> ry[kC];
        Pack<T, kVec> rn[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) t.template fetch<Y>(a.y, image, i, ry[i]);
#pragma unroll
        for (int i = 0; i < kC; ++i) t.template fetch<T>(a.dn, image, i, rn[i]);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          t.template take<Y>(ry[i], i, x[i]);
          t.template take<T>(rn[i], i, d[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
          for (int j = 0; j < kVec; ++j) d[i][j] = 0.0f;
      }
      if (a.w_pre) {
        unit(t, x, r, a.layer, a.eps, shared);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const float w = t.channel_value(a.w_pre, i);
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            dwn[i] = fmaf(d[i][j], x[i][j], dwn[i]);
            dbn[i] += d[i][j];
            d[i][j] *= w;
          }
        }
        through(t, d, x, r, a.layer, shared);
      }
      // only now, for the registers' sake
      if (a.dy)
#pragma unroll
        for (int i = 0; i < kC; ++i) t.template fetch<Y>(a.dy, image, i, rd[i]);
#pragma unroll
      for (int i = 0; i < kC; ++i) t.template fetch<T>(a.h, image, i, rh[i]);
      if (a.z)
#pragma unroll
        for (int i = 0; i < kC; ++i) t.template fetch<T>(a.z, image, i, rz[i]);
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        if (a.dy) {
          float y[kVec];
          t.template take<Y>(rd[i], i, y);
#pragma unroll
          for (int j = 0; j < kVec; ++j) d[i][j] += y[j];
        }
        if (a.dres) t.template store<Y>(a.dres, image, i, d[i]);
        t.template take<T>(rh[i], i, x[i]);
      }
      if (a.w_post) unit(t, x, r, a.layer, a.eps, shared);
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const float w = a.w_post ? t.channel_value(a.w_post, i) : 1.0f;
        const float b = a.b_post ? t.channel_value(a.b_post, i) : 0.0f;
        const float s = scale ? t.channel_value(scale, i) : 1.0f;
        float z[kVec], dz[kVec];
        if (a.z) t.template take<T>(rz[i], i, z);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float p = a.w_post ? fmaf(x[i][j], w, b) : x[i][j];
          float sg = 0.0f, gv = 1.0f;
          if (a.z) {
            sg = sigmoid_f32(z[j]);
            gv = gate_value(z[j], sg);
          }
          if (scale) {
            // positions past the end have d = 0
            dsc[i] = fmaf(d[i][j], a.z ? p * gv : p, dsc[i]);
            d[i][j] *= s;
          }
          if (a.z) {
            dz[j] = d[i][j] * p * gate_slope(z[j], sg);
            d[i][j] *= gv;
          }
          if (a.w_post) {
            dwp[i] = fmaf(d[i][j], x[i][j], dwp[i]);
            dbp[i] += d[i][j];
            d[i][j] *= w;
          }
        }
        if (a.z) t.template store<T>(a.dz, image, i, dz);
      }
      if (a.w_post) through(t, d, x, r, a.layer, shared);
#pragma unroll
      for (int i = 0; i < kC; ++i) t.template store<T>(a.dh, image, i, d[i]);
    }
    if (a.scale) write_sums(t, dsc, a.scale_parts + (g * a.blocks_per_group + part) * a.D);
  }
  float* out = a.parts + int64_t(blockIdx.x) * kSums * a.D;
  if (a.dw_post) write_sums(t, dwp, out);
  if (a.db_post) write_sums(t, dbp, out + a.D);
  if (a.dw_pre) write_sums(t, dwn, out + 2 * a.D);
  if (a.db_pre) write_sums(t, dbn, out + 3 * a.D);
}

// Positions of a thread; tiles are 16 times as wide.  A thread holds at most 32 values of a
// tensor (backward, with two tensors and the sums of its channels: 16) and 16 channels.
int vec_of(int D, bool bwd) {
  if (bwd) return D <= 128 ? 4 : (D <= 256 ? 2 : 1);
  return D <= 256 ? 4 : (D <= 512 ? 2 : 1);
}

template <typename T, typename Y, int kThreads, int kC, int kVec, bool kWide>
void forward(const Args& a, int64_t blocks, hipStream_t st) {
  hipLaunchKernelGGL((k_norm_first<T, Y, kThreads, kC, kVec, kWide>), dim3(static_cast<unsigned>(blocks)),
                     dim3(kThreads), 0, st, a);
}
template <typename T, typename Y, int kThreads, int kC, int kVec, bool kWide>
void backward(const Args& a, int64_t blocks, hipStream_t st) {
  hipLaunchKernelGGL((k_norm_first_bwd<T, Y, kThreads, kC, kVec, kWide>),
                     dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st, a);
}

// Widths by powers of two and one and a half times those, so that at most a third of a block's
// channels lie past the last one.  3.9e7 values (64 maps of 192 x 56 x 56), bfloat16 with an fp32
// residual stream, with powers of two alone and with the steps in between: forward 155 and 139 us
// at D = 96, 202 and 138 at 192, 216 and 197 at 384, 285 and 261 at 768; backward 312 and 285, 338
// and 312, 570 and 377, 1151 and 824.
template <typename T, typename Y, bool kWide>
int launch_channels(const Args& a, bool bwd, int64_t blocks, hipStream_t st) {
  if (bwd) {
    if (a.D <= 64) backward<T, Y, 256, 4, 4, kWide>(a, blocks, st);
    else if (a.D <= 96) backward<T, Y, 512, 3, 4, kWide>(a, blocks, st);
    else if (a.D <= 128) backward<T, Y, 512, 4, 4, kWide>(a, blocks, st);
    else if (a.D <= 192) backward<T, Y, 512, 6, 2, kWide>(a, blocks, st);
    else if (a.D <= 256) backward<T, Y, 512, 8, 2, kWide>(a, blocks, st);
    else if (a.D <= 384) backward<T, Y, 1024, 6, 1, kWide>(a, blocks, st);
    else if (a.D <= 512) backward<T, Y, 1024, 8, 1, kWide>(a, blocks, st);
    else if (a.D <= 768) backward<T, Y, 1024, 12, 1, kWide>(a, blocks, st);
    else backward<T, Y, 1024, 16, 1, kWide>(a, blocks, st);
  } else {
    if (a.D <= 64) forward<T, Y, 256, 4, 4, kWide>(a, blocks, st);
    else if (a.D <= 96) forward<T, Y, 512, 3, 4, kWide>(a, blocks, st);
    else if (a.D <= 128) forward<T, Y, 512, 4, 4, kWide>(a, blocks, st);
    else if (a.D <= 192) forward<T, Y, 512, 6, 4, kWide>(a, blocks, st);
    else if (a.D <= 256) forward<T, Y, 512, 8, 4, kWide>(a, blocks, st);
    else if (a.D <= 384) forward<T, Y, 1024, 6, 2, kWide>(a, blocks, st);
    else if (a.D <= 512) forward<T, Y, 1024, 8, 2, kWide>(a, blocks, st);
    else if (a.D <= 768) forward<T, Y, 1024, 12, 1, kWide>(a, blocks, st);
    else forward<T, Y, 1024, 16, 1, kWide>(a, blocks, st);
  }
  return static_cast<int>(hipGetLastError());
}

template <bool kWide>
int launch_types(const Args& a, int dtype, int ytype, bool bwd, int64_t blocks, hipStream_t st) {
  if (dtype == 0) return launch_channels<float, float, kWide>(a, bwd, blocks, st);
  if (ytype == 0) return launch_channels<uint16_t, float, kWide>(a, bwd, blocks, st);
  return launch_channels<uint16_t, uint16_t, kWide>(a, bwd, blocks, st);
}

}  // namespace

int64_t tiles_first(const Args& a, bool bwd) {  // of one group
  const int64_t width = kP * vec_of(a.D, bwd);
  return a.group * ((a.L + width - 1) / width);
}

int launch_norm_first(const Args& a, int dtype, int ytype, bool vec, bool bwd, int64_t blocks,
                      hipStream_t st) {
  if (!bwd) blocks = std::min<int64_t>(tiles_first(a, false) * a.G, 256 * 16);
  const bool wide = vec && a.L % vec_of(a.D, bwd) == 0;
  return wide ? launch_types<true>(a, dtype, ytype, bwd, blocks, st)
              : launch_types<false>(a, dtype, ytype, bwd, blocks, st);
}

}  // namespace norm
}  // namespace ss2d
