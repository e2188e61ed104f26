// Sums of the scan's decays, in 64 bits, shared by its forms.
#pragma once

#include <type_traits>

#include "sk_scan.hpp"

namespace sk {

// From the lane that the DPP control CTRL names (MASK: the rows that it writes), 0
// where there is none.
template <int CTRL, int MASK = 0xF>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, MASK, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, MASK, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum of the lanes up to this one: of a row of 16, of the wave.
__device__ __forceinline__ double row_prefix(double x) {
  x += dpp_d<0x111>(x);                          // row_shr:1, 2, 4, 8
  x += dpp_d<0x112>(x);
  x += dpp_d<0x114>(x);
  x += dpp_d<0x118>(x);
  return x;
}
__device__ __forceinline__ double wave_prefix(double x) {
  x = row_prefix(x);
  x += dpp_d<0x142, 0xA>(x);                     // row_bcast:15, 31
  x += dpp_d<0x143, 0xC>(x);
  return x;
}
// A lane's value, in every lane.
template <int LANE>
__device__ __forceinline__ double lane_d(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, LANE), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), LANE);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_last(double x) { return lane_d<63>(x); }

// 2^x in fp32 of an exponent in 64 bits: of what rounding it leaves, to first order.
__device__ __forceinline__ float exp2_of(double x) {
  const float f = (float)x, e = __builtin_amdgcn_exp2f(f);
  return fmaf(e, (float)(x - (double)f) * 0.693147182f, e);
}
constexpr double LOG2E = 1.4426950408889634;

}  // namespace sk
