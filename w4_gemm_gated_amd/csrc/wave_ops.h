// Running sums and reductions over the 64 lanes of a wave, by moves between lanes within the
// vector unit (a step takes a few cycles; through the LDS crossbar, as a shuffle goes, more
// than a hundred).  All lanes of the wave must be active.
#pragma once

#include "device_common.h"

namespace spear {

// v of another lane: CTRL 0x111, 0x112, 0x114, 0x118 of the one 1, 2, 4, 8 before it in
// the row of sixteen, 0x142 and 0x143 of the last of the row, and of the half, before it.
// `none` where there is no such lane, or the row is not one of ROWS.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T moved(T v, T none) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v), CTRL,
                                                             ROWS, 0xF, false));
  } else {
    typedef int two_t __attribute__((ext_vector_type(2)));
    const two_t x = __builtin_bit_cast(two_t, v), n = __builtin_bit_cast(two_t, none);
    const two_t r = {__builtin_amdgcn_update_dpp(n[0], x[0], CTRL, ROWS, 0xF, false),
                     __builtin_amdgcn_update_dpp(n[1], x[1], CTRL, ROWS, 0xF, false)};
    return __builtin_bit_cast(T, r);
  }
}

// f over the lanes up to and with this one; `none`: f(x, none) = x.
template <typename T, typename F>
__device__ __forceinline__ T wave_run(T v, T none, F f) {
  v = f(v, moved<0x111, 0xF>(v, none));
  v = f(v, moved<0x112, 0xF>(v, none));
  v = f(v, moved<0x114, 0xF>(v, none));
  v = f(v, moved<0x118, 0xF>(v, none));
  v = f(v, moved<0x142, 0xA>(v, none));
  return f(v, moved<0x143, 0xC>(v, none));
}
template <typename T>
__device__ __forceinline__ T wave_run(T v) {
  return wave_run(v, (T)0, [](T a, T b) { return a + b; });
}

// f over groups of 8, 16 or 32 neighbouring lanes, in each of them.
template <int LANES, typename T, typename F>
__device__ __forceinline__ T lanes_all(T v, F f) {
  static_assert(LANES == 8 || LANES == 16 || LANES == 32, "within a half of the wave");
  v = f(v, moved<0xB1, 0xF>(v, v));       // the lane one apart, two apart, ..
  v = f(v, moved<0x4E, 0xF>(v, v));
  v = f(v, moved<0x141, 0xF>(v, v));      // .. the other four of eight, the other eight of sixteen
  if constexpr (LANES > 8) v = f(v, moved<0x140, 0xF>(v, v));
  if constexpr (LANES > 16) v = f(v, (T)__shfl_xor(v, 16));
  return v;
}

// A lane's value, in every lane.
template <typename T>
__device__ __forceinline__ T of_lane(T v, int lane) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  } else {
    typedef int two_t __attribute__((ext_vector_type(2)));
    const two_t x = __builtin_bit_cast(two_t, v);
    const two_t r = {__builtin_amdgcn_readlane(x[0], lane), __builtin_amdgcn_readlane(x[1], lane)};
    return __builtin_bit_cast(T, r);
  }
}

// f over all lanes, in every lane.
template <typename T, typename F>
__device__ __forceinline__ T wave_all(T v, T none, F f) {
  return of_lane(wave_run(v, none, f), kWave - 1);
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
  return of_lane(wave_run(v), kWave - 1);
}
template <typename T>
__device__ __forceinline__ T wave_max(T v, T none) {
  return wave_all(v, none, [](T a, T b) { return a > b ? a : b; });
}

}  // namespace spear
