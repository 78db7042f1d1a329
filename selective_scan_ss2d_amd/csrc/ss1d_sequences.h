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

// A value that the compiler takes for a new one, so that nothing derived from it leaves the loop.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Element `at` past a uniform pointer.  A load with the byte offset in 32 bits, extended beside it
// (`at` opaque, where the extension would be moved out of a loop), keeps the pointer in scalar
// registers and one vector register for the lane.
template <typename T> __device__ __forceinline__ const T& element(const T* p, uint32_t at) {
  return *reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + at * uint32_t(sizeof(T)));
}
template <typename T> __device__ __forceinline__ T& element(T* p, uint32_t at) {
  return *reinterpret_cast<T*>(reinterpret_cast<char*>(p) + at * uint32_t(sizeof(T)));
}

// The rows of a step and the slots that they name.  Padding rows name a slot outside 0 .. count - 1.
// Rows that name one slot are further tokens of one sequence, in row order: the first of them does
// them all, so that no two waves hold the same state.
struct Slots {
  const int32_t* at;  // (rows) or NULL: row b has slot b
  int rows;
  int64_t count;
};

// For rows first .. first + n - 1 (n <= 32) of a block, in bit i of `seen`: [0] an earlier row names
// row first + i's slot, [1] a later one does.  Every thread of the block takes part.
__device__ __forceinline__ void find_repeats(const Slots& s, int first, int n, uint32_t* seen) {
  if (threadIdx.x < 2) seen[threadIdx.x] = 0;
  if (!s.at) return;
  const int lane = threadIdx.x & 63;
  const int mine = s.at[min(first + (lane < n ? lane : 0), s.rows - 1)];
  __syncthreads();
  for (int i = threadIdx.x; i < s.rows; i += blockDim.x) {
    const int v = s.at[i];
    uint32_t before = 0, behind = 0;
    for (int r = 0; r < n; ++r) {
      const bool same = v == __builtin_amdgcn_readlane(mine, r);
      before |= same && i < first + r ? 1u << r : 0u;
      behind |= same && i > first + r ? 1u << r : 0u;
    }
    if (before) atomicOr(&seen[0], before);
    if (behind) atomicOr(&seen[1], behind);
  }
  __syncthreads();
}

// The slot of row first + i, -1 for a row to leave alone.
__device__ __forceinline__ int slot_of(const Slots& s, int first, int i, const uint32_t* seen) {
  if (!s.at) return first + i;
  const int slot = __builtin_amdgcn_readfirstlane(s.at[first + i]);
  const bool left = slot < 0 || slot >= s.count || (__builtin_amdgcn_readfirstlane(seen[0]) >> i & 1);
  return left ? -1 : slot;
}

// The next row behind b that names the slot, `rows` if there is none.
__device__ __forceinline__ int next_of(const Slots& s, int b, int slot) {
  const int lane = threadIdx.x & 63;
  for (int base = b + 1; base < s.rows; base += 64) {
    const int i = base + lane;
    const uint64_t hit = __ballot(i < s.rows && s.at[i < s.rows ? i : b] == slot);
    if (hit) return base + __ffsll(static_cast<unsigned long long>(hit)) - 1;
  }
  return s.rows;
}

}  // namespace ss2d
