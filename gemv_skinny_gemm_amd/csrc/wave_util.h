// wave_util.h - sums and maxima over a wave by lane moves, no shared memory.
#ifndef SKINNY_WAVE_UTIL_H
#define SKINNY_WAVE_UTIL_H

#include <hip/hip_runtime.h>

namespace skinny_wave {

typedef unsigned long long u64;

// The value of the lane that CTRL names within a row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ unsigned from_lane(unsigned x) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ u64 from_lane(u64 x) {
  return (u64)from_lane<CTRL>((unsigned)x) | (u64)from_lane<CTRL>((unsigned)(x >> 32)) << 32;
}
// A lane's value and that of the lane OFF (16 or 32) away, in either order.
struct Pair {
  u64 a, b;
};
template <int OFF>
__device__ __forceinline__ auto swapped(unsigned x) {
  if constexpr (OFF == 16) return __builtin_amdgcn_permlane16_swap(x, x, false, false);
  else return __builtin_amdgcn_permlane32_swap(x, x, false, false);
}
template <int OFF>
__device__ __forceinline__ Pair across(u64 x) {
  const auto lo = swapped<OFF>((unsigned)x), hi = swapped<OFF>((unsigned)(x >> 32));
  const unsigned l0 = lo[0], l1 = lo[1], h0 = hi[0], h1 = hi[1];
  return Pair{(u64)l0 | (u64)h0 << 32, (u64)l1 | (u64)h1 << 32};
}

template <typename T>
__device__ __forceinline__ u64 bits(T x) { return __builtin_bit_cast(u64, x); }

// Sums over runs of 2, 4, 8 and 16 neighbouring lanes, in all of them: neighbours,
// pairs, then mirrored halves and rows, whose lanes agree by then.
template <int N>
__device__ __forceinline__ double lanes_sum(double x) {
  if constexpr (N > 1) x += __builtin_bit_cast(double, from_lane<0xb1>(bits(x)));    // quad_perm 1 0 3 2
  if constexpr (N > 2) x += __builtin_bit_cast(double, from_lane<0x4e>(bits(x)));    // quad_perm 2 3 0 1
  if constexpr (N > 4) x += __builtin_bit_cast(double, from_lane<0x141>(bits(x)));   // row_half_mirror
  if constexpr (N > 8) x += __builtin_bit_cast(double, from_lane<0x140>(bits(x)));   // row_mirror
  return x;
}
// Over the wave, in every lane.
__device__ __forceinline__ double wave_sum(double x) {
  x = lanes_sum<16>(x);
  const Pair p = across<16>(bits(x));
  x = __builtin_bit_cast(double, p.a) + __builtin_bit_cast(double, p.b);
  const Pair q = across<32>(bits(x));
  return __builtin_bit_cast(double, q.a) + __builtin_bit_cast(double, q.b);
}
__device__ __forceinline__ unsigned wave_max(unsigned x) {
  x = max(x, from_lane<0xb1>(x));
  x = max(x, from_lane<0x4e>(x));
  x = max(x, from_lane<0x141>(x));
  x = max(x, from_lane<0x140>(x));
  const auto p = swapped<16>(x);
  const unsigned a = p[0], b = p[1];
  const auto q = swapped<32>(max(a, b));
  const unsigned c = q[0], d = q[1];
  return max(c, d);
}
}  // namespace skinny_wave

#endif  // SKINNY_WAVE_UTIL_H
