// Group norm of rows whose channels come last, with an activation:
//   x' = x * act(z) where the gate comes first, else x
//   n  = (x' - mean) / sqrt(var + eps) over each group of `width` channels
//        (mean 0 and var = mean of squares unless centred)
//   y  = n * weight + bias, times act(z) where the gate comes after, or
//        act(y) where there is no gate.
// Bound by memory: x (and z) read once, y written once (16384 x 32 groups of 128
// in bf16, call behind call: 403 MB in 65.5 us, 6.1 TB/s).  A lane keeps its
// 16-byte vectors of a group in registers, so the variance is that of the
// held values about their mean (two passes over registers, one over memory),
// and a thread keeps its channels' weights while it goes from row to row.
// Statistics are summed in 32 bits.
#include "sk_serve_device.hpp"

namespace sk {
namespace {

constexpr int NORM_THREADS = 256;

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

// LPG: lanes of a group (256: the whole workgroup, through LDS), VPL: vectors
// of a lane.  Thread position in a row: group * LPG + lane; `tpr` = groups *
// LPG threads make a row where that is at most the workgroup, otherwise
// blockIdx.y selects the part of the row.
template <typename T, int LPG, int VPL, bool PAST>
__global__ void __launch_bounds__(NORM_THREADS) group_norm_kernel(NormParams p) {
  constexpr int N = Vec<T>::N;
  __shared__ float s_part[4];
  const int tid = threadIdx.x, tpr = p.groups * LPG;
  const int rpw = tpr < NORM_THREADS ? NORM_THREADS / tpr : 1;       // rows of a workgroup
  const int rl = tpr < NORM_THREADS ? tid / tpr : 0;
  const int pos = tpr < NORM_THREADS ? tid - rl * tpr : (int)blockIdx.y * NORM_THREADS + tid;
  const int g = pos / LPG, ln = pos - g * LPG;
  const int nvec = p.width / N;
  // (every lane of a group shares g and rl, so a group is in or out whole;
  // the lanes that are out take no part in the others' sums)
  const bool in = rl < rpw && g < p.groups;
  if (LPG < NORM_THREADS && !in) return;
  float w[VPL][N], b[VPL][N];
#pragma unroll
  for (int u = 0; u < VPL; ++u) {
    const int c = ln + LPG * u;
#pragma unroll
    for (int e = 0; e < N; ++e) { w[u][e] = 1.f; b[u][e] = 0.f; }
    if (c < nvec) {
      const int64_t at = (int64_t)g * p.wgs + c * N;
      if (p.weight) ldn<N>(p.weight + at, w[u]);
      if (p.bias) ldn<N>(p.bias + at, b[u]);
    }
  }
  const float inv_n = 1.f / (float)p.width;
  const T* X = reinterpret_cast<const T*>(p.x) + (int64_t)g * p.width;
  const T* Z = reinterpret_cast<const T*>(p.gate) + (int64_t)g * p.width;
  T* Y = reinterpret_cast<T*>(p.y) + (int64_t)g * p.width;
  auto sum = [&](float x) -> float {
    if constexpr (LPG < NORM_THREADS) {
      return group_sum<LPG>(x);
    } else {
      x = group_sum<64>(x);
      __syncthreads();
      if ((tid & 63) == 0) s_part[tid >> 6] = x;
      __syncthreads();
      return s_part[0] + s_part[1] + s_part[2] + s_part[3];
    }
  };
  int64_t lo = p.first ? *p.first : 0, end = p.end ? *p.end : p.rows;
  lo = lo > 0 ? lo : 0;
  end = end < p.rows ? end : p.rows;
  for (int64_t row = lo + (int64_t)blockIdx.x * rpw + rl; row < end; row += (int64_t)gridDim.x * rpw) {
    float x[VPL][N], z[VPL][N];
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      const int c = ln + LPG * u;
#pragma unroll
      for (int e = 0; e < N; ++e) x[u][e] = z[u][e] = 0.f;
      if (c < nvec) {
        unpack(read16<PAST>(X + row * p.xs + c * N), x[u]);
        if (p.gate) unpack(read16<PAST>(Z + row * p.zs + c * N), z[u]);
      }
    }
    if (p.gate && p.gate_first) {
#pragma unroll
      for (int u = 0; u < VPL; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) x[u][e] *= (ln + LPG * u < nvec) ? activation<T>(z[u][e], p.act) : 0.f;
    }
    float mean = 0.f;
    if (p.centred) {
      float a = 0.f;
#pragma unroll
      for (int u = 0; u < VPL; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) a += x[u][e];
      mean = sum(a) * inv_n;
    }
    float a = 0.f;
#pragma unroll
    for (int u = 0; u < VPL; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = x[u][e] - mean;
        x[u][e] = d;
        a += (ln + LPG * u < nvec) ? d * d : 0.f;
      }
    const float rs = 1.f / sqrtf(sum(a) * inv_n + p.eps);
#pragma unroll
    for (int u = 0; u < VPL; ++u) {
      const int c = ln + LPG * u;
      if (c < nvec) {
        float y[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          y[e] = x[u][e] * rs * w[u][e] + b[u][e];
          if (!p.gate) y[e] = activation<T>(y[e], p.act);
          else if (!p.gate_first) y[e] *= activation<T>(z[u][e], p.act);
        }
        u32x4* at = reinterpret_cast<u32x4*>(Y + row * p.ys + c * N);
        if (PAST) __builtin_nontemporal_store(pack(y), at);
        else *at = pack(y);
      }
    }
  }
}

template <typename T, int LPG, int VPL>
int launch(const NormParams& p, hipStream_t st) {
  const int64_t tpr = (int64_t)p.groups * LPG;
  const int64_t rpw = tpr < NORM_THREADS ? NORM_THREADS / tpr : 1;
  const int64_t parts = tpr < NORM_THREADS ? 1 : (tpr + NORM_THREADS - 1) / NORM_THREADS;
  int64_t rows = (p.rows + rpw - 1) / rpw;
  // 64 workgroups for each of the 256 CUs, and further rows in turn (16384 x 32
  // groups of 128, 403 MB: 16 a CU 77.3 us, 32 70.6, 64 65.5, 128 67.8, one for
  // every row 67.7).  Where the output is beyond the 32 MiB of the L2s, it is
  // stored and the inputs are read past them (74.7 and 65.5 us).
  const int64_t most = (16384 + parts - 1) / parts;
  if (rows > most) rows = most;
  const bool past = p.rows > (32 << 20) / ((int64_t)p.groups * p.width * (int)sizeof(T));
  const dim3 grid((unsigned)rows, (unsigned)parts), block(NORM_THREADS);
  if (past) hipLaunchKernelGGL((group_norm_kernel<T, LPG, VPL, true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((group_norm_kernel<T, LPG, VPL, false>), grid, block, 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <typename T>
int launch_type(const NormParams& p, hipStream_t st) {
  const int nvec = p.width / Vec<T>::N;
  if (nvec <= 1) return launch<T, 1, 1>(p, st);
  if (nvec <= 2) return launch<T, 2, 1>(p, st);
  if (nvec <= 4) return launch<T, 4, 1>(p, st);
  if (nvec <= 8) return launch<T, 8, 1>(p, st);
  if (nvec <= 16) return launch<T, 16, 1>(p, st);
  if (nvec <= 32) return launch<T, 32, 1>(p, st);
  if (nvec <= 64) return launch<T, 64, 1>(p, st);
  if (nvec <= 128) return launch<T, 64, 2>(p, st);
  if (nvec <= 256) return launch<T, 64, 4>(p, st);
  if (nvec <= 512) return launch<T, NORM_THREADS, 2>(p, st);
  if (nvec <= 1024) return launch<T, NORM_THREADS, 4>(p, st);
  return launch<T, NORM_THREADS, 8>(p, st);
}

}  // namespace

int launch_group_norm(int dtype, const NormParams& p, hipStream_t st) {
  return dtype == DT_F32 ? launch_type<float>(p, st) : launch_type<bf16>(p, st);
}

}  // namespace sk
