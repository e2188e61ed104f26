// The state cache: states quantised as they are written to slots, and read
// back.  A block is 32 consecutive values of a state row (along dv); with
// m = 127 (8 bits) or 7 (4 bits),
//   scale = max|x| / m,  code = round to nearest even (x / scale),
//   value = code * scale.
// A block whose largest magnitude is under 2^-100 is stored as zeros (its
// scale would leave the normal range); a block that holds an infinity or a
// NaN gets the scale NaN and reads back as NaN.
//
// Both directions are bound by memory: 4 bytes a value on the state's side,
// bits / 8 + 1/8 on the cache's (128 sequences of 32 heads of 128 x 128 in 8 bits:
// 344 MB in 66 us to the cache, 5.2 TB/s, and 352 MB in 58 us back, 6.0; 96 of 128
// heads of 128 x 64 in 4 bits: 466 MB in 92 us and 479 MB in 78).
#include "sk_serve_device.hpp"

namespace sk {
namespace {

constexpr int QB = 32;                     // values that share a scale
constexpr int SAVE_THREADS = 256;
// Up to this many tiles are saved by several workgroups each.  Measured, a
// workgroup a tile and split (us): 128 x 128 in 8 bits, 32 tiles 5.4 and 3.3, 512
// 10.9 and 10.3, 1024 18.4 and 19.1, 4096 64 and 69; 64 x 64, 32 tiles 3.4 and 3.1, 512
// 4.5 and 4.2, 2048 9.8 and 10.3.
constexpr int kSplitSave = 512;

// 1.5 * 2^23: a sum with it is rounded to a whole number (to nearest even), which
// is then the low bits of the sum.
constexpr float WHOLE = 12582912.f;

// round(x / s) to nearest even, exactly, as WHOLE + code, from c, the rounded
// product with s's reciprocal: c is off by at most one, and its remainder, a
// multiple of the smaller operand's unit that is at most about s, is exact in one
// fma.
__device__ __forceinline__ float exact_code(float x, float s, float c) {
  const float r = fmaf(-c, s, x), half = 0.5f * s;
  const bool odd = ((int)c & 1) != 0;
  if (r > half || (r == half && odd)) c += 1.f;
  else if (r < -half || (r == -half && odd)) c -= 1.f;
  return c + WHOLE;
}

// max over the four lanes of a quad, NaN-keeping (integer maximum of the
// magnitudes' bits: NaN sorts above infinity).
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false);
  x = x > y ? x : y;
  y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false);
  return x > y ? x : y;
}

// One workgroup per (entry, head), or PARTS of them where there are few tiles: a
// lane takes 8 consecutive values, so a block is a quad of lanes and a wave
// reads 2 KiB in a row.
template <int DK, int DV, int BITS, int PARTS>
__global__ void __launch_bounds__(SAVE_THREADS) state_save_kernel(CacheParams p) {
  constexpr int ALL = DK * DV / 8, ITEMS = ALL / PARTS, U = (ITEMS + SAVE_THREADS - 1) / SAVE_THREADS;
  static_assert(ALL % PARTS == 0 && ITEMS % 4 == 0, "whole blocks");
  const int i = blockIdx.x / p.H, h = blockIdx.x - i * p.H, tid = threadIdx.x;
  const int b = p.seqs[i], slot = p.slot[i];
  const bool in = b >= 0 && b < p.B;
  const int first = (int)blockIdx.y * ITEMS * 8;
  const float* S = p.S + ((size_t)b * p.H + h) * DK * DV + first;
  float x[U][8];                             // (in flight over the checks)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + SAVE_THREADS * u;
    if (in && (ITEMS % SAVE_THREADS == 0 || c < ITEMS)) {
      float a[4], d[4];
      ldn_nt<4>(S + 8 * c, a);
      ldn_nt<4>(S + 8 * c + 4, d);
#pragma unroll
      for (int e = 0; e < 4; ++e) { x[u][e] = a[e]; x[u][4 + e] = d[e]; }
    }
  }
  int bad = 0;
  if (!in) bad = ERRBIT_SEQ;
  else if (slot < 0 || slot >= p.slots || listed_before(p.slot, i, slot)) bad = ERRBIT_SLOT;
  else if (p.count[(size_t)b * p.H + h] != 0) bad = ERRBIT_COUNT;
  if (bad) {
    if (tid == 0) atomicOr(p.err, bad);
    return;
  }
  const size_t tile = (size_t)slot * p.H + h;
  float* scale = p.scale + tile * (DK * DV / QB) + first / QB;
  char* codes = reinterpret_cast<char*>(p.codes) + tile * (DK * DV * BITS / 8) + first * BITS / 8;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = tid + SAVE_THREADS * u;
    if (ITEMS % SAVE_THREADS == 0 || c < ITEMS) {    // (whole quads: ITEMS is a multiple of 4)
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t a = __float_as_uint(x[u][e]) & 0x7fffffffu;
        m = m > a ? m : a;
      }
      m = quad_max(m);
      const float amax = __uint_as_float(m);
      const bool finite = m < 0x7f800000u, live = finite && amax >= 0x1p-100f;
      // (127 times the scale of the largest fp32 value, rounded up, would pass it)
      const float of = BITS == 8 ? fminf(amax / 127.f, 0x1.0204060000000p+121f) : amax / 7.f;
      const float s = live ? of : (finite ? 0.f : __uint_as_float(0x7fc00000u));
      const float inv = live ? 1.f / s : 0.f;
      // The product with the rounded reciprocal is off by at most 2^-24 of a
      // quotient up to 127, 8e-6: a code is right where the product is no nearer
      // than 2e-5 to a half.  The others (4e-5 of them) are put right with their
      // wave's eight values.
      uint32_t q[8];
      float near = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float w = fmaf(x[u][e], inv, WHOLE);
        near = fmaxf(near, fabsf(fmaf(x[u][e], inv, -(w - WHOLE))));
        q[e] = __float_as_uint(w);
      }
      if (__any(near > 0.49998f)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (live) q[e] = __float_as_uint(exact_code(x[u][e], s, __uint_as_float(q[e]) - WHOLE));
      }
      if constexpr (BITS == 8) {
        auto four = [&](int e) {               // their low bytes
          const uint32_t a = __builtin_amdgcn_perm(q[e + 1], q[e], 0x0c0c0400u);
          const uint32_t b = __builtin_amdgcn_perm(q[e + 3], q[e + 2], 0x04000c0cu);
          return live ? a | b : 0u;
        };
        reinterpret_cast<uint2*>(codes)[c] = make_uint2(four(0), four(4));
      } else {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= (q[e] & 15) << (4 * e);
        reinterpret_cast<uint32_t*>(codes)[c] = live ? w : 0;
      }
      if ((tid & 3) == 0) scale[c >> 2] = s;
    }
  }
}

// One workgroup per (entry, head), a wave per 32 columns: a row's block of
// those columns has one scale.  The codes come as 16-byte chunks through
// LDS, and the tile is held in the flush's register layout, from which the
// sketch needs no further pass over the state.
template <int DK, int DV, int BITS, typename UT>
__global__ void __launch_bounds__(DV * 2) state_load_kernel(CacheParams p) {
  constexpr int NT = DV * 2, MB = DK / 16, BYTES = DK * DV * BITS / 8, CH = BYTES / 16;
  constexpr int NS = DK * DV / QB, SROW = DV / QB;
  __shared__ __align__(16) unsigned char s_codes[BYTES];
  __shared__ __align__(16) float s_scale[NS];
  const int i = blockIdx.x / p.H, h = blockIdx.x - i * p.H, tid = threadIdx.x;
  const int b = p.seqs[i], slot = p.slot[i];
  int bad = 0;
  if (slot < 0 || slot >= p.slots) bad = ERRBIT_SLOT;
  else if (b < 0 || b >= p.B || listed_before(p.seqs, i, b)) bad = ERRBIT_SEQ;
  if (bad) {
    if (tid == 0) atomicOr(p.err, bad);
    return;
  }
  const size_t tile = (size_t)slot * p.H + h;
  const uint4* codes = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p.codes) + tile * BYTES);
  const float4* scale = reinterpret_cast<const float4*>(p.scale + tile * NS);
  for (int c = tid; c < CH; c += NT) reinterpret_cast<uint4*>(s_codes)[c] = codes[c];
  for (int c = tid; c < NS / 4; c += NT) reinterpret_cast<float4*>(s_scale)[c] = scale[c];
  __syncthreads();

  const int lane = tid & 63, cg = lane & 15, rg = lane >> 4, wv = tid >> 6;
  const int col0 = 32 * wv, col = col0 + 2 * cg;
  float s[MB][2][4];
  float* Sg = p.S + ((size_t)b * p.H + h) * DK * DV + col;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int m = 16 * mb + 4 * rg + v;
      const float sc = s_scale[m * SROW + wv];
      int q0, q1;
      if constexpr (BITS == 8) {
        const int w = *reinterpret_cast<const uint16_t*>(s_codes + m * DV + col);
        q0 = (int)(int8_t)(w & 255);
        q1 = (int)(int8_t)(w >> 8);
      } else {
        const int w = s_codes[(m * DV + col) / 2];
        q0 = (w << 28) >> 28;
        q1 = (w << 24) >> 28;
      }
      const float x[2] = {(float)q0 * sc, (float)q1 * sc};
      s[mb][0][v] = x[0];
      s[mb][1][v] = x[1];
      stn_nt<2>(Sg + (size_t)m * DV, x);
    }
  if (p.prime) sketch_tile<DK, DV, UT, 2>(p.sk, s, b, h, col0, lane);
  if (tid == 0) p.count[(size_t)b * p.H + h] = 0;
}

template <int DK, int DV, int PARTS>
void launch_save(const CacheParams& p, hipStream_t st) {
  const dim3 grid(p.n * p.H, PARTS);
  if (p.bits == 8)
    hipLaunchKernelGGL((state_save_kernel<DK, DV, 8, PARTS>), grid, dim3(SAVE_THREADS), 0, st, p);
  else
    hipLaunchKernelGGL((state_save_kernel<DK, DV, 4, PARTS>), grid, dim3(SAVE_THREADS), 0, st, p);
}

template <int DK, int DV>
int save_shape(const CacheParams& p, hipStream_t st) {
  constexpr int PARTS = DK * DV >= 8 * SAVE_THREADS ? DK * DV / (8 * SAVE_THREADS) : 1;
  if (p.n * p.H <= kSplitSave)
    launch_save<DK, DV, PARTS>(p, st);
  else
    launch_save<DK, DV, 1>(p, st);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <int DK, int DV, typename UT>
int load_shape(const CacheParams& p, hipStream_t st) {
  const dim3 grid(p.n * p.H), block(DV * 2);
  if (p.bits == 8)
    hipLaunchKernelGGL((state_load_kernel<DK, DV, 8, UT>), grid, block, 0, st, p);
  else
    hipLaunchKernelGGL((state_load_kernel<DK, DV, 4, UT>), grid, block, 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_state_save(int dk, int dv, const CacheParams& p, hipStream_t st) {
  if (dk == 16 && dv == 32) return save_shape<16, 32>(p, st);
  if (dk == 64 && dv == 64) return save_shape<64, 64>(p, st);
  if (dk == 128 && dv == 64) return save_shape<128, 64>(p, st);
  if (dk == 128 && dv == 128) return save_shape<128, 128>(p, st);
  return -2;
}

int launch_state_load(int dk, int dv, int sketch, const CacheParams& p, hipStream_t st) {
  const bool f = sketch == DT_F32;
  if (dk == 16 && dv == 32) return f ? load_shape<16, 32, float>(p, st) : load_shape<16, 32, bf16>(p, st);
  if (dk == 64 && dv == 64) return f ? load_shape<64, 64, float>(p, st) : load_shape<64, 64, bf16>(p, st);
  if (dk == 128 && dv == 64) return f ? load_shape<128, 64, float>(p, st) : load_shape<128, 64, bf16>(p, st);
  if (dk == 128 && dv == 128) return f ? load_shape<128, 128, float>(p, st) : load_shape<128, 128, bf16>(p, st);
  return -2;
}

}  // namespace sk
