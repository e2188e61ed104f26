// 16-byte vectors of activations as fp32 values, and the activations, shared by
// the output norm and the short convolution.
#pragma once

#include "sk_serve_device.hpp"

namespace sk {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename T> struct Vec { static constexpr int N = 16 / (int)sizeof(T); };

// 16 bytes, past the caches' keeping or not; as fp32 values, and back.
template <bool PAST>
__device__ __forceinline__ u32x4 read16(const void* p) {
  const u32x4* at = reinterpret_cast<const u32x4*>(p);
  return PAST ? __builtin_nontemporal_load(at) : *at;
}
__device__ __forceinline__ void unpack(const u32x4& w, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const u32x4& w, float (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(w[e]);
}
__device__ __forceinline__ u32x4 pack(const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {                  // (one instruction: to nearest even)
    const bf16x2 v = {(__bf16)x[2 * e], (__bf16)x[2 * e + 1]};
    w[e] = __builtin_bit_cast(uint32_t, v);
  }
  return w;
}
__device__ __forceinline__ u32x4 pack(const float (&x)[4]) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(x[e]);
  return w;
}

// Sum over aligned groups of L lanes (L a power of two up to 64).
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (L <= 8) return low_lane_sum<L>(x);
  x = row16_sum(x);
  if constexpr (L >= 32) x += __shfl_xor(x, 16);
  if constexpr (L >= 64) x += __shfl_xor(x, 32);
  return x;
}

// act: 0 none, 1 SiLU, 2 sigmoid.  In fp32, of exp(-|x|), which does not overflow:
// 2^t of the rounded t = -|x| log2(e) and, to first order, of what the rounding
// left, over 1 + that by a reciprocal put right once: some units of 2^-24 of the
// result.  In bf16 the exponential instruction alone, whose rounded argument puts
// it off by 2^-24 |x| of itself, and the reciprocal instruction (2^-23) are far
// below half a step (2^-8) wherever the result is over 2^-118 (below -87 it becomes
// 0).  16384 x 32 groups of 128: fp32, gated 134 us, centred without a gate 92, as with
// the short form (with expf and an exact quotient 134 and 100); bf16, gated, 66 with
// the short form and 67 with this, centred without a gate 53 and 61.
template <typename T>
__device__ __forceinline__ float activation(float x, int act) {
  if (act == 0) return x;
  float s;
  if constexpr (sizeof(T) == 4) {
    constexpr float L = 1.44269502f, L_REST = 1.92596303e-8f, LN2 = 0.693147182f;
    const float a = fabsf(x) > 128.f ? 128.f : fabsf(x);      // (the rest of an infinity would be a NaN)
    const float t = -L * a, rest = fmaf(a, -L_REST, fmaf(a, -L, -t));
    const float f = __builtin_amdgcn_exp2f(t), e = fmaf(f, rest * LN2, f), d = 1.f + e;
    const float r = __builtin_amdgcn_rcpf(d);
    s = (x < 0.f ? e : 1.f) * fmaf(fmaf(-d, r, 1.f), r, r);
  } else {
    s = __builtin_amdgcn_rcpf(1.f + __expf(-x));
  }
  return act == 1 ? x * s : s;
}

}  // namespace sk
