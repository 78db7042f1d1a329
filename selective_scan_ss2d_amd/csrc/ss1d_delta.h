// Shared pieces of the gated delta rule's kernels (gfx950): the arguments, the matrix
// operands and products, and the loads.
//
// The rule, per sequence and value head, with a (DK, DV) state S:
//   S <- e^g_t S;  u_t = beta_t (v_t - S^T k_t);  S <- S + k_t u_t^T;  o_t = scale S^T q_t.
// In chunks of 32 tokens, with G_i = g_1 + .. + g_i inside the chunk, S the state before it,
//   L_ij = e^(G_i - G_j) k_i.k_j (j < i),   P_ij = scale e^(G_i - G_j) q_i.k_j (j <= i),
//   r_i  = v_i - e^G_i S^T k_i,   (I + L diag(beta)) t = r,   u = beta t,
//   o_i  = scale e^G_i S^T q_i + (P u)_i,
//   S    <- e^G_32 S + sum_j e^(G_32 - G_j) k_j u_j^T.
// With N = (I + L diag(beta))^-1 L (strictly lower triangular, free of beta on the outside)
// t = r - N (beta r), and the backward's adjoint solve is w = y - N^T (beta y): the identity
// part is never rounded, and beta = 0 needs no care.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ss2d_device.h"
#include "ss2d_lanes.h"

namespace ss2d {
namespace delta {

constexpr int kC = 32;      // tokens per chunk: one 32 x 32 matrix tile
constexpr int kMaxDK = 128; // largest key width (the state's rows held by one wave)
constexpr int kMark = 64;   // tokens between the states a training forward keeps
constexpr int kGradWaves = 8;   // of a block that forms dq and dk

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Strides {  // in elements; the last axis has stride 1
  int64_t b, l, h;
};

struct Args {
  const void *q, *k, *v;       // (B, L, HK, DK), (B, L, HK, DK), (B, L, H, DV)
  const float *g, *beta;       // (B, L, H)
  const float* h0;             // (S, H, DK, DV) or NULL
  const int32_t* cu;           // (S + 1) offsets into the tokens of B = 1, or NULL
  void* o;                     // (B, L, H, DV)
  float* ht;                   // (S, H, DK, DV) or NULL
  Strides sq, sk, sv;
  int64_t S, L, T;             // sequences, tokens of a batch row, tokens in all
  int H, HK, rep, DK, DV;      // rep = H / HK value heads share a key head
  float scale;
  // scratch, per (chunk slot, head): matrix fragments and gates
  char* keys;                  // (slot, HK) records, see KeyRecord
  char* heads;                 // (slot, H) records, see HeadRecord
  int64_t slots;               // chunk slots
  int p_planes;                // bf16 terms kept of P
  // sequences cut into segments of `seglen` chunks (0: not cut), see span kernels; per
  // (segment slot, head): the state after the segment from a zero one (DK, DV), the state
  // before it (DK, DV), and the matrix that the segment applies to it, with its transpose if
  // a backward is to come (operand fragments, see matrix_plane)
  int64_t seglen, seg_slots;
  float *span_z, *starts;
  char *span_m, *span_t;
  // kept by a training forward
  float *marks, *ends;         // states before every 64 tokens and after the last
  float *ts, *os;              // t and o in fp32, (T, H, DV)
  // backward
  const void* dout;            // gradient of o, contiguous
  const float* dht;            // gradient of the end states, or NULL
  void *dq, *dk, *dv;
  float *dg, *dbeta, *dh0;     // dh0 may be NULL
  float* dmarks;               // gradients of the states after every 64 tokens
  float* dvs;                  // dv in fp32, (T, H, DV); for fp32 data dv itself
  float *pbeta, *pgate;        // per tile of 32 columns: w.t and do.o - dv.v of every token
  float* pdots;                // per 64 tokens, head and tile: <dS, S> after them
  int64_t marks_n;             // slots of 64 tokens
};

// ---- sequences and chunk slots -----------------------------------------------------------
struct Seq {
  int64_t row;   // first token among all tokens (rows of contiguous tensors)
  int64_t len;
};

// Offsets out of order or out of range are cut to [0, T], so that no address leaves the
// tensors whatever the offsets hold.
__device__ __forceinline__ Seq sequence(const Args& a, int64_t n) {
  if (!a.cu) return {n * a.L, a.L};
  int64_t s = a.cu[n], e = a.cu[n + 1];
  s = s < 0 ? 0 : (s > a.T ? a.T : s);
  e = e < s ? s : (e > a.T ? a.T : e);
  return {s, e - s};
}

// First slot of sequence n among slots of `unit` tokens, no two sequences sharing a slot:
// dense, n ceil(L / unit); packed, floor(start / unit) + n.
__device__ __forceinline__ int64_t first_slot(const Args& a, int64_t n, const Seq& s, int unit) {
  return a.cu ? s.row / unit + n : n * ((a.L + unit - 1) / unit);
}

// The sequence and index inside it of a slot; false for a slot that no sequence uses.
__device__ __forceinline__ bool find_slot(const Args& a, int64_t slot, int unit, int64_t* n,
                                          int64_t* index, Seq* s) {
  if (!a.cu) {
    const int64_t per = (a.L + unit - 1) / unit;
    *n = slot / per;
    *index = slot - *n * per;
    *s = sequence(a, *n);
    return *n < a.S;
  }
  int64_t lo = 0, hi = a.S;  // the last sequence whose first slot is not past `slot`
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (first_slot(a, mid, sequence(a, mid), unit) <= slot) lo = mid; else hi = mid;
  }
  *n = lo;
  *s = sequence(a, lo);
  *index = slot - first_slot(a, lo, *s, unit);
  return *index >= 0 && *index * unit < s->len;
}

// Part of a sequence: all of it, or segment `index` of it (slots of seglen chunks; segment 0
// exists for an empty sequence too).
struct Segment {
  int64_t n, index, slot;
  Seq seq;
  int64_t begin, end;  // chunks
  bool last;
};
__device__ __forceinline__ bool find_segment(const Args& a, int64_t slot, Segment* g) {
  if (a.seglen == 0) {
    g->n = slot;
    g->index = 0;
    g->slot = slot;
    g->seq = sequence(a, slot);
    g->begin = 0;
    g->end = (g->seq.len + kC - 1) / kC;
    g->last = true;
    return true;
  }
  const bool used = find_slot(a, slot, static_cast<int>(a.seglen * kC), &g->n, &g->index, &g->seq);
  const int64_t chunks = (g->seq.len + kC - 1) / kC;
  g->slot = slot;
  g->begin = g->index * a.seglen;
  g->end = min(chunks, g->begin + a.seglen);
  g->last = g->end == chunks;
  return used || (g->index == 0 && g->n < a.S);
}

// Element offset of token t of sequence n in a strided (B, L, H, .) tensor.
__device__ __forceinline__ int64_t token_at(const Args& a, const Strides& st, int64_t n,
                                            const Seq& s, int64_t t) {
  return a.cu ? (s.row + t) * st.l : n * st.b + t * st.l;
}

// ---- matrix operands -----------------------------------------------------------------------
// A tile of a product is 32 x 32 x 16.  Lane l holds 8 consecutive values of the contracted
// axis, 8 (l / 32) + 0..7, of row (left operand) or column (right operand) l % 32.  The
// result's lane holds column l % 32; its register r is row 8 (r / 4) + 4 (l / 32) + r % 4.
// Left operands are loaded with their rows in the order swap23 (bits 2 and 3 exchanged):
// then result register r is row 16 (r / 8) + 8 (l / 32) + r % 8 of the unpermuted order, and
// registers 8 s .. 8 s + 7 are the right operand of the next product's step s as they
// stand: states and solutions pass from one product to the next without leaving registers.
__device__ __forceinline__ int swap23(int i) {
  return (i & ~12) | ((i & 4) << 1) | ((i & 8) >> 1);
}
__device__ __forceinline__ int acc_row(int r, int half) { return 16 * (r >> 3) + 8 * half + (r & 7); }

// An operand as the data type stores it.  fp32 data use the fp32 matrix instructions.
template <typename T> struct Exact;
template <> struct Exact<uint16_t> { bf16x8 v; };
template <> struct Exact<float> { f32x8 v; };

// An fp32 operand.  For bfloat16 data it is a sum of P bfloat16 terms, each the rounding of
// what the terms before it leave: 3 terms hold 24 bits, i.e. the fp32 value, 2 terms 17.
// A product with an operand that is exact in bfloat16 then takes P matrix instructions, one
// of two fp32 operands the P (P + 1) / 2 pairs of terms that matter.
template <typename T, int P> struct Wide;
template <int P> struct Wide<uint16_t, P> { bf16x8 p[P]; };
template <int P> struct Wide<float, P> { f32x8 v; };

// Two values rounded to nearest bfloat16 and packed by one v_cvt_pk_bf16_f32.  The empty asm
// hides where the bits come from: the compiler otherwise converts each value once more, alone,
// to get at the rounded value.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 x = {lo, hi};
  uint32_t r = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  asm("" : "+v"(r));
  return r;
}
template <int P>
__device__ __forceinline__ void set_wide(Wide<uint16_t, P>& w, f32x8 x) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    u32x4 u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t both = pack_bf16(x[2 * j], x[2 * j + 1]);
      u[j] = both;
      if (i + 1 < P) {
        x[2 * j] -= __uint_as_float(both << 16);
        x[2 * j + 1] -= __uint_as_float(both & 0xffff0000u);
      }
    }
    w.p[i] = __builtin_bit_cast(bf16x8, u);
  }
}
template <int P>
__device__ __forceinline__ void set_wide(Wide<float, P>& w, f32x8 x) { w.v = x; }

template <int P>
__device__ __forceinline__ Wide<uint16_t, P> first_terms(const Wide<uint16_t, 3>& w) {
  Wide<uint16_t, P> x;
#pragma unroll
  for (int i = 0; i < P; ++i) x.p[i] = w.p[i];
  return x;
}
template <int P>
__device__ __forceinline__ Wide<float, P> first_terms(const Wide<float, 3>& w) { return {w.v}; }

__device__ __forceinline__ f32x8 part(const f32x16& x, int s) {
  f32x8 y;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[8 * s + i];
  return y;
}

__device__ __forceinline__ f32x16 mma16(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// Waits until the matrix instructions before it have written their results (at most 18 states):
// stands where the compiler counts short, see `settled`.
__device__ __forceinline__ void drained() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 1");
  __builtin_amdgcn_sched_barrier(0);
}
// fp32: one instruction contracts two values, one of each half of the wave.
__device__ __forceinline__ f32x16 mma8(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ f32x16 mma(const Exact<uint16_t>& a, const Exact<uint16_t>& b, f32x16 c) {
  return mma16(a.v, b.v, c);
}
template <int P>
__device__ __forceinline__ f32x16 mma(const Exact<uint16_t>& a, const Wide<uint16_t, P>& b, f32x16 c) {
#pragma unroll
  for (int j = P - 1; j >= 0; --j) c = mma16(a.v, b.p[j], c);
  return c;
}
template <int P>
__device__ __forceinline__ f32x16 mma(const Wide<uint16_t, P>& a, const Exact<uint16_t>& b, f32x16 c) {
#pragma unroll
  for (int j = P - 1; j >= 0; --j) c = mma16(a.p[j], b.v, c);
  return c;
}
template <int P, int R>
__device__ __forceinline__ f32x16 mma(const Wide<uint16_t, P>& a, const Wide<uint16_t, R>& b, f32x16 c) {
  constexpr int M = P > R ? P : R;
#pragma unroll
  for (int i = P - 1; i >= 0; --i)
#pragma unroll
    for (int j = R - 1; j >= 0; --j)
      if (i + j < M) c = mma16(a.p[i], b.p[j], c);
  return c;
}
__device__ __forceinline__ f32x16 mma(const Exact<float>& a, const Exact<float>& b, f32x16 c) {
  return mma8(a.v, b.v, c);
}
template <int P>
__device__ __forceinline__ f32x16 mma(const Exact<float>& a, const Wide<float, P>& b, f32x16 c) {
  return mma8(a.v, b.v, c);
}
template <int P>
__device__ __forceinline__ f32x16 mma(const Wide<float, P>& a, const Exact<float>& b, f32x16 c) {
  return mma8(a.v, b.v, c);
}
template <int P, int R>
__device__ __forceinline__ f32x16 mma(const Wide<float, P>& a, const Wide<float, R>& b, f32x16 c) {
  return mma8(a.v, b.v, c);
}

// Pointers into device memory, whose accesses need no look at the address space.
template <typename T> using Global = __attribute__((address_space(1))) T*;
template <typename T> __device__ __forceinline__ Global<T> global(T* p) { return (Global<T>)p; }

// ---- loads ---------------------------------------------------------------------------------
// 8 consecutive values of a row, columns c .. c + 7 of `width`; zero past the width or where
// `on` is false.  kAligned: every row starts on 16 bytes and the width is a multiple of 8.
template <bool kAligned>
__device__ __forceinline__ void load8(Exact<uint16_t>& x, const uint16_t* row, int c, int width,
                                      bool on) {
  if constexpr (kAligned) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (on && c < width) u = *reinterpret_cast<const uint4*>(row + c);
    x.v = __builtin_bit_cast(bf16x8, u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint16_t e = 0;
      if (on && c + i < width) e = row[c + i];
      x.v[i] = __builtin_bit_cast(__bf16, e);
    }
  }
}
template <bool kAligned>
__device__ __forceinline__ void load8(Exact<float>& x, const float* row, int c, int width, bool on) {
  if constexpr (kAligned) {
    f32x4 u = {0, 0, 0, 0}, w = {0, 0, 0, 0};
    if (on && c < width) {
      u = *reinterpret_cast<const f32x4*>(row + c);
      w = *reinterpret_cast<const f32x4*>(row + c + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) { x.v[i] = u[i]; x.v[4 + i] = w[i]; }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float e = 0.0f;
      if (on && c + i < width) e = row[c + i];
      x.v[i] = e;
    }
  }
}

__device__ __forceinline__ f32x16 load_gate(const float* gate, int half) {
  f32x16 x;
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(gate + 16 * s + 8 * half + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[8 * s + 4 * i + e] = u[e];
    }
  return x;
}

// Fragments in scratch: 16 bytes a lane, one plane of 1 KB after another.
constexpr int kPlane = 1024;
constexpr int kReadPast = 4 * kPlane;  // what Stage reads behind the last record at most
template <typename T> constexpr int exact_planes() { return sizeof(T) == 4 ? 2 : 1; }
template <typename T, int P> constexpr int wide_planes() { return sizeof(T) == 4 ? 2 : P; }

__device__ __forceinline__ void put_planes(char* at, int lane, const f32x8& v) {
  f32x4 u, w;
#pragma unroll
  for (int i = 0; i < 4; ++i) { u[i] = v[i]; w[i] = v[4 + i]; }
  reinterpret_cast<f32x4*>(at)[lane] = u;
  reinterpret_cast<f32x4*>(at + kPlane)[lane] = w;
}
__device__ __forceinline__ f32x8 get_planes(const char* at, int lane) {
  const f32x4 u = reinterpret_cast<const f32x4*>(at)[lane];
  const f32x4 w = reinterpret_cast<const f32x4*>(at + kPlane)[lane];
  f32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = u[i]; v[4 + i] = w[i]; }
  return v;
}
__device__ __forceinline__ void put(char* at, int lane, const Exact<uint16_t>& x) {
  reinterpret_cast<uint4*>(at)[lane] = __builtin_bit_cast(uint4, x.v);
}
__device__ __forceinline__ void put(char* at, int lane, const Exact<float>& x) {
  put_planes(at, lane, x.v);
}
__device__ __forceinline__ void get(Exact<uint16_t>& x, const char* at, int lane) {
  x.v = __builtin_bit_cast(bf16x8, reinterpret_cast<const uint4*>(at)[lane]);
}
__device__ __forceinline__ void get(Exact<float>& x, const char* at, int lane) {
  x.v = get_planes(at, lane);
}
template <int P>
__device__ __forceinline__ void put(char* at, int lane, const Wide<uint16_t, P>& x) {
#pragma unroll
  for (int i = 0; i < P; ++i)
    reinterpret_cast<uint4*>(at + i * kPlane)[lane] = __builtin_bit_cast(uint4, x.p[i]);
}
template <int P>
__device__ __forceinline__ void put(char* at, int lane, const Wide<float, P>& x) {
  put_planes(at, lane, x.v);
}
template <int P>
__device__ __forceinline__ void get(Wide<uint16_t, P>& x, const char* at, int lane) {
#pragma unroll
  for (int i = 0; i < P; ++i)
    x.p[i] = __builtin_bit_cast(bf16x8, reinterpret_cast<const uint4*>(at + i * kPlane)[lane]);
}
template <int P>
__device__ __forceinline__ void get(Wide<float, P>& x, const char* at, int lane) {
  x.v = get_planes(at, lane);
}

// A segment's (DK, DK) matrix in fp32: for each 32 rows the operands of 2 KT steps.
__host__ __device__ constexpr int64_t matrix_bytes(int kt) { return int64_t(4) * kt * kt * kPlane; }
__device__ __forceinline__ int64_t matrix_plane(int kt, int rows, int step) {
  return (int64_t(rows) * 2 * kt + step) * 2 * kPlane;
}

// One chunk's operands in scratch, in the order in which the sequential kernels take them:
// per key head K, K^T and Q (backward: Q^T), per value head N, a plane of gates (e^G,
// e^(G_32 - G), beta: 32 values each) and P (backward: N^T and P^T).
template <typename T, int KT> struct KeyRecord {
  static constexpr int kOperand = 2 * KT * exact_planes<T>();  // planes of one operand
  static constexpr int kPlanes = 3 * kOperand;
};
template <typename T, int P> struct HeadRecord {
  static constexpr int kN = 2 * wide_planes<T, 3>(), kP = 2 * wide_planes<T, P>();
  static constexpr int kGates = kN, kPStart = kN + 1, kPlanes = kN + 1 + kP;
};
__host__ __device__ constexpr int key_planes(bool f32, int kt) { return 3 * 2 * kt * (f32 ? 2 : 1); }
__host__ __device__ constexpr int head_planes(bool f32, int p) {
  return (f32 ? 4 : 6) + 2 * (f32 ? 2 : p) + 1;
}

// Brings the records of one chunk after another into LDS: fetch() starts the next chunk's loads
// into registers, which the chunk's products overlap; after the products and a barrier,
// commit() writes them.  (One buffer and two barriers: a second buffer would save one, but
// the LDS it takes keeps a second block off the CU, whose waves fill the first one's gaps.)  The block's kW waves share the planes; where those do not divide
// evenly the last ones are read (from the scratch behind the record) and not written.
// kState: only what the state's own recurrence takes (K, K^T, N and the gates).
template <typename T, int KT, int P, int kW, bool kState = false> struct Stage {
  using Key = KeyRecord<T, KT>;
  using Head = HeadRecord<T, P>;
  static constexpr int kKeyRead = kState ? 2 * Key::kOperand : Key::kPlanes;
  static constexpr int kHeadRead = kState ? Head::kN + 1 : Head::kPlanes;
  static constexpr int kPlanes = kKeyRead + kHeadRead;
  static constexpr int kKeys = (kKeyRead + kW - 1) / kW, kHeads = (kHeadRead + kW - 1) / kW;
  u32x4 x[kKeys + kHeads];
  Global<const char> key, head;       // this wave's first plane of the next chunk's records
  int64_t key_step, head_step;        // to the next chunk's (backward: the one before)
  int wave, lane;
  __device__ __forceinline__ void start(const Args& a, int64_t slot, int hv, int hk, int w, int l,
                                        int direction) {
    wave = w;
    lane = l;
    const int64_t kb = int64_t(Key::kPlanes) * kPlane,
                  hb = int64_t(head_planes(sizeof(T) == 4, a.p_planes)) * kPlane;
    key = global(static_cast<const char*>(a.keys)) + (slot * a.HK + hk) * kb + w * kPlane;
    head = global(static_cast<const char*>(a.heads)) + (slot * a.H + hv) * hb + w * kPlane;
    key_step = direction * a.HK * kb;
    head_step = direction * a.H * hb;
  }
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) x[i] = *(Global<const u32x4>)(key + i * kW * kPlane + 16u * lane);
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      x[kKeys + i] = *(Global<const u32x4>)(head + i * kW * kPlane + 16u * lane);
    key += key_step;
    head += head_step;
  }
  __device__ __forceinline__ void commit(char* buffer) const {
    char* to = buffer + wave * kPlane + 16 * lane;
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if ((i + 1) * kW <= kKeyRead || wave + i * kW < kKeyRead)
        *reinterpret_cast<u32x4*>(to + i * kW * kPlane) = x[i];
    to += kKeyRead * kPlane;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
      if ((i + 1) * kW <= kHeadRead || wave + i * kW < kHeadRead)
        *reinterpret_cast<u32x4*>(to + i * kW * kPlane) = x[kKeys + i];
  }
  // operand `which` (0 K, 1 K^T, 2 Q or Q^T), tile kt, step s
  static __device__ __forceinline__ const char* operand(const char* buffer, int which, int kt, int s) {
    return buffer + (which * Key::kOperand + (2 * kt + s) * exact_planes<T>()) * kPlane;
  }
  static __device__ __forceinline__ const char* n(const char* buffer, int s) {
    return buffer + (kKeyRead + s * wide_planes<T, 3>()) * kPlane;
  }
  static __device__ __forceinline__ const char* p(const char* buffer, int s) {
    return buffer + (kKeyRead + Head::kPStart + s * wide_planes<T, P>()) * kPlane;
  }
  static __device__ __forceinline__ const float* gates(const char* buffer) {
    return reinterpret_cast<const float*>(buffer + (kKeyRead + Head::kGates) * kPlane);
  }
};

// Orders a wave's own LDS accesses (its lanes exchange data; no other wave takes part).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- 32 x 32 tiles of matrices in memory -----------------------------------------------------
// A wave moves its tile in 16-byte pieces of rows and turns it in LDS of its own into the
// product's layout (a column per lane) and back: there the rows' distance is a constant, so
// the 16 accesses of a lane need no address arithmetic, which would otherwise cost more than
// the products.  The row pitch keeps the wave's halves, 8 rows apart, on different banks.
constexpr int row_base(int r) { return 16 * (r >> 3) + (r & 7); }  // acc_row of the lower half
template <typename T> constexpr int tile_pitch() { return sizeof(T) == 4 ? 144 : 80; }
constexpr int kTileBytes = 32 * 144;

// Whole tiles of aligned rows go through registers, loaded ahead; others (a sequence's last
// chunk, odd widths) element by element when they are wanted.
__device__ __forceinline__ bool aligned16(const void* base, uint32_t stride, int cols) {
  return ((reinterpret_cast<uintptr_t>(base) | stride) & 15) == 0 && cols >= 32;
}

template <typename T> struct Tile {
  static constexpr int kPieces = sizeof(T);              // 16-byte pieces per lane: 2 or 4
  static constexpr int kAcross = 2 * sizeof(T);          // pieces across a row
  static constexpr int kStep = 64 / kAcross;             // rows per access of the wave
  u32x4 x[kPieces];

  // Starts the loads of a whole tile, its rows `stride` bytes apart (base and stride uniform).
  __device__ __forceinline__ void fetch(const void* base, uint32_t stride, int lane) {
    const auto p = global(static_cast<const char*>(base));
    const uint32_t off = lane / kAcross * stride + lane % kAcross * 16;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      x[i] = *(Global<const u32x4>)(p + (uint64_t(i * kStep) * stride + off));
  }
  __device__ __forceinline__ void put(char* lds, int lane) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      *reinterpret_cast<u32x4*>(lds + (lane / kAcross + i * kStep) * tile_pitch<T>() +
                                lane % kAcross * 16) = x[i];
  }
  // The tile in the product's layout by way of `lds`: what fetch() brought where `whole`, else
  // `rows` rows (others are 0) and `cols` columns (others repeat the last) from `base`.
  __device__ __forceinline__ f32x16 columns(bool whole, const void* base, uint32_t stride, int rows,
                                            int cols, char* lds, int lane) const {
    wave_sync();
    if (whole) {
      put(lds, lane);
    } else {
      const auto p = global(static_cast<const char*>(base));
      const uint32_t c = lane & 31;
#pragma nounroll
      for (int i = lane >> 5; i < 32; i += 2) {
        T v = T(0);
        if (i < rows)
          v = *(Global<const T>)(p + (uint64_t(i) * stride + min(int(c), cols - 1) * sizeof(T)));
        *reinterpret_cast<T*>(lds + i * tile_pitch<T>() + c * sizeof(T)) = v;
      }
    }
    wave_sync();
    f32x16 v;
    const char* at = lds + 8 * (lane >> 5) * tile_pitch<T>() + (lane & 31) * sizeof(T);
#pragma unroll
    for (int r = 0; r < 16; ++r)
      v[r] = Elem<T>::load(reinterpret_cast<const T*>(at + row_base(r) * tile_pitch<T>()));
    return v;
  }
};

// Stores a tile in the product's layout: all of it where `whole`, else `rows` rows and `cols`
// columns (0: none).  column: that of this lane's values (lane % 32 by default).
template <typename T>
__device__ __forceinline__ void store_tile(const f32x16& v, void* base, uint32_t stride, bool whole,
                                           int rows, int cols, char* lds, int lane, int column = -1) {
  using X = Tile<T>;
  wave_sync();
  char* to = lds + 8 * (lane >> 5) * tile_pitch<T>() + (column < 0 ? lane & 31 : column) * sizeof(T);
#pragma unroll
  for (int r = 0; r < 16; ++r)
    *reinterpret_cast<T*>(to + row_base(r) * tile_pitch<T>()) = Elem<T>::from_f32(v[r]);
  wave_sync();
  const auto p = global(static_cast<char*>(base));
  if (whole) {
    const uint32_t off = lane / X::kAcross * stride + lane % X::kAcross * 16;
#pragma unroll
    for (int i = 0; i < X::kPieces; ++i)
      *(Global<u32x4>)(p + (uint64_t(i * X::kStep) * stride + off)) =
          *reinterpret_cast<const u32x4*>(lds + (lane / X::kAcross + i * X::kStep) * tile_pitch<T>() +
                                          lane % X::kAcross * 16);
  } else {
    const int c = lane & 31, end = min(rows, 32);
    if (c < cols)
#pragma nounroll
      for (int i = lane >> 5; i < end; i += 2)
        *(Global<T>)(p + (uint64_t(i) * stride + c * sizeof(T))) =
            *reinterpret_cast<const T*>(lds + i * tile_pitch<T>() + c * sizeof(T));
  }
}

// A wave's place: 32 columns (`tile`) of one sequence and head.  Columns past the last one
// repeat it, waves past the last tile repeat that tile: both compute and never store.
struct Place {
  int lane, wave, half, tile, hv, hk;
  int cols, store_cols;  // columns of the tile; those that this wave stores (0: none)
  int64_t head;          // of the state's tensors: n * H + hv
  bool in;               // this lane's column is stored
  Segment g;
};
// The block's unit is (segment, head, kW tiles); `width` columns make the tiles.
template <int kW>
__device__ __forceinline__ bool place(Place* p, const Args& a, int64_t unit, int width) {
  const int tiles = (width + 31) / 32, per = (tiles + kW - 1) / kW;
  p->lane = threadIdx.x & 63;
  p->wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  p->half = p->lane >> 5;
  const int64_t sh = unit / per, slot = sh / a.H;
  p->hv = static_cast<int>(sh - slot * a.H);
  p->hk = p->hv / a.rep;
  if (!find_segment(a, slot, &p->g)) return false;
  p->head = p->g.n * a.H + p->hv;
  const int tile = static_cast<int>(unit - sh * per) * kW + p->wave;
  p->tile = min(tile, tiles - 1);
  p->cols = min(32, width - 32 * p->tile);
  p->store_cols = tile < tiles ? p->cols : 0;
  p->in = (p->lane & 31) < p->store_cols;
  return true;
}

// The state's (DK, DV) columns of a wave, from `base` (its first column; NULL: zeros).
template <int KT>
__device__ __forceinline__ void load_state(f32x16* S, const float* base, const Args& a, const Place& w,
                                           char* lds) {
  const uint32_t stride = a.DV * 4u;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    S[kt] = f32x16{};
    const int rows = a.DK - 32 * kt;
    if (base == nullptr || rows <= 0) continue;
    const float* at = base + int64_t(32) * kt * a.DV;
    Tile<float> x;
    const bool whole = aligned16(at, stride, w.cols) && rows >= 32;
    if (whole) x.fetch(at, stride, w.lane);
    S[kt] = x.columns(whole, at, stride, rows, w.cols, lds, w.lane);
  }
}
template <typename T, int KT>
__device__ __forceinline__ void store_state(const f32x16* S, void* base, float factor, const Args& a,
                                            const Place& w, char* lds, int width = 0) {
  const uint32_t stride = (width ? width : a.DV) * sizeof(T);  // values of a row
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    const int rows = a.DK - 32 * kt;
    if (rows <= 0) continue;
    void* at = static_cast<char*>(base) + int64_t(32) * kt * stride;
    store_tile<T>(S[kt] * factor, at, stride, aligned16(at, stride, w.store_cols) && rows >= 32, rows,
                  w.store_cols, lds, w.lane);
  }
}

// A state under decay is held as S = factor * X with a common factor, so that a chunk's decay
// costs one multiplication instead of one per value; what is added to S is divided by the
// factor.  Before the factor falls under 2^-16 (growing decays: exceeds 1) it goes into X.
//
// The products before it have to be used up by then (`settled`): where a value that a matrix
// instruction wrote is first read behind a short conditional block, the compiler counts the wait
// states along that block alone and not along the jump past it, and the read comes too early.
__device__ __forceinline__ void settled(f32x16& x) { asm volatile("" : "+v"(x)); }
template <int KT>
__device__ __forceinline__ float decay_state(f32x16* X, float factor, float decay) {
  factor *= decay;
  if (!(factor >= 0x1p-16f && factor <= 1.0f)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) X[kt] *= factor;
    factor = 1.0f;
  }
  return factor;
}

// Log decays below this are 0 in fp32 either way; the bound keeps -inf out of differences.
// Prefix sums are kept in 64 bits and in units of log 2: a difference of far sums then is
// exact to fp32, and one v_exp_f32 (1 ulp) makes it a factor.
constexpr float kMinLog = -1000.0f;
constexpr double kLog2eWide = 1.4426950408889634074;
// (fmaxf would turn a NaN into the bound.)
__device__ __forceinline__ float bounded_log(float g) { return g < kMinLog ? kMinLog : g; }
__device__ __forceinline__ float decay_of(double diff) { return exp2_hw(static_cast<float>(diff)); }

int launch_prep(const Args& a, int dtype, bool aligned, bool backward, hipStream_t st);
int launch_scan(const Args& a, int dtype, bool save, hipStream_t st);
int launch_span(const Args& a, int dtype, hipStream_t st);
int launch_join(const Args& a, bool backward, hipStream_t st);
int launch_adjoint(const Args& a, int dtype, bool span, hipStream_t st);
int launch_grads(const Args& a, int dtype, bool aligned, hipStream_t st);
int launch_gate_grads(const Args& a, hipStream_t st);

}  // namespace delta
}  // namespace ss2d
