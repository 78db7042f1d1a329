// Sequences of a call in token order: B rows of L tokens, or packed ones named by S + 1 offsets
// into the tokens of one row, cut into units of a fixed length that are worked on at once.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ss2d {

// Element strides of one token to the next of a row, and of one row to the next.
struct RowStrides {
  int64_t b, l;
};

// unit u of a sequence's `len` tokens: dense rows hold ceil(L / len) units each; the units of
// packed sequence n start at unit offset[n] / len + n, which leaves enough for every sequence
// whatever the offsets are, and some units empty.
__host__ __device__ inline int64_t unit_count(int64_t L, int64_t S, int64_t T, bool packed,
                                              int64_t len) {
  return packed ? T / len + S : S * ((L + len - 1) / len);
}

struct Sequences {
  const int32_t* cu;   // S + 1 offsets, or NULL
  int64_t S, L, T;
};

// One sequence: row b of the tensors, tokens begin .. begin + len - 1 of it.
struct Sequence {
  int64_t n, b, begin, len;
};

__device__ __forceinline__ int64_t cut_offset(const Sequences& q, int64_t i) {
  const int64_t v = q.cu[i];
  return v < 0 ? 0 : (v > q.T ? q.T : v);
}

__device__ __forceinline__ Sequence sequence(const Sequences& q, int64_t n) {
  if (!q.cu) return {n, n, 0, q.L};
  const int64_t a = cut_offset(q, n), e = cut_offset(q, n + 1);
  return {n, 0, a, e > a ? e - a : 0};
}

// The first unit of a sequence.
__device__ __forceinline__ int64_t first_unit(const Sequences& q, const Sequence& s, int64_t len) {
  return q.cu ? s.begin / len + s.n : s.n * ((q.L + len - 1) / len);
}

// The sequence that a unit belongs to, and its number in it (which may lie past the sequence's
// end: an empty unit).  Offsets that do not ascend find some sequence.
__device__ __forceinline__ Sequence sequence_of(const Sequences& q, int64_t unit, int64_t len,
                                                int64_t* index) {
  if (!q.cu) {
    const int64_t per = (q.L + len - 1) / len;
    *index = unit % per;
    return sequence(q, unit / per);
  }
  int64_t lo = 0, hi = q.S;  // the last n with offset / len + n <= unit
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (cut_offset(q, mid) / len + mid <= unit) lo = mid;
    else hi = mid;
  }
  const Sequence s = sequence(q, lo);
  *index = unit - first_unit(q, s, len);
  if (*index < 0) *index = s.len / len + 1;  // offsets out of order: an empty unit
  return s;
}

// A value that is the same in every lane of a wave, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ Sequence uniform(const Sequence& s) {
  return {uniform(s.n), uniform(s.b), uniform(s.begin), uniform(s.len)};
}

}  // namespace ss2d
