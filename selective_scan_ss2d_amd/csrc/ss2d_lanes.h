// Values of other lanes of a wave without LDS permutes: DPP moves inside rows of 16 lanes, the
// row and half-wave swaps across them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ss2d {

template <int kCtrl> __device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, true));
}

// The v of lane ^ kXor inside its row: quad permutations, a rotation by 8, and for 4 the mirrors
// of 8 and of 4 lanes one after the other.
template <int kXor> __device__ __forceinline__ float from_lane(float v) {
  static_assert(kXor == 1 || kXor == 2 || kXor == 4 || kXor == 8, "lanes of one row");
  if constexpr (kXor == 1) return dpp_move<0xB1>(v);
  else if constexpr (kXor == 2) return dpp_move<0x4E>(v);
  else if constexpr (kXor == 4) return dpp_move<0x1B>(dpp_move<0x141>(v));
  else return dpp_move<0x128>(v);
}

// The swaps: rows 1 and 3 of a against rows 0 and 2 of b, the upper half of a against the lower
// half of b.
__device__ __forceinline__ void swap_rows(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

// v plus the v of lane ^ kXor.
template <int kXor> __device__ __forceinline__ float add_across(float v) {
  if constexpr (kXor < 16) {
    return v + from_lane<kXor>(v);
  } else {
    float w = v;
    if constexpr (kXor == 16) swap_rows(v, w);
    else swap_halves(v, w);
    return v + w;
  }
}

// Sum over kLanes adjacent lanes (a power of two), or over every kFirst-th of them, in all.
template <int kLanes, int kFirst = 1> __device__ __forceinline__ float lane_sum(float v) {
  if constexpr (kFirst <= 1 && kLanes > 1) v = add_across<1>(v);
  if constexpr (kFirst <= 2 && kLanes > 2) v = add_across<2>(v);
  if constexpr (kFirst <= 4 && kLanes > 4) v = add_across<4>(v);
  if constexpr (kFirst <= 8 && kLanes > 8) v = add_across<8>(v);
  if constexpr (kFirst <= 16 && kLanes > 16) v = add_across<16>(v);
  if constexpr (kFirst <= 32 && kLanes > 32) v = add_across<32>(v);
  return v;
}

}  // namespace ss2d
