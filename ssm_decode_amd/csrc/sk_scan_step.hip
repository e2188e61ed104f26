// Prompts through the selective state space scan, one token at a time:
//   S <- a S + k (dt v)^T,  a = exp(-dt exp(A_h)),  o = S^T q.
// One workgroup per (prompt, head); a wave holds 16 or 32 columns of the tile, all
// of its rows, in registers for the whole prompt (rows and columns of S never
// mix but in the output's sum over rows).
//
// A prompt of a few tokens is bound by its state's traffic (4 dk dv bytes in and
// out), a longer one by the chain from token to token, so long ones take the
// chunked form.
#include "sk_scan.hpp"
#include "sk_serve_device.hpp"

namespace sk {
namespace {

constexpr int TB = 16;    // tokens staged at a time

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void put16(float* dst, const u32x4& r, const bf16*) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const u32x4 x = {r[2 * e] << 16, r[2 * e] & 0xffff0000u, r[2 * e + 1] << 16, r[2 * e + 1] & 0xffff0000u};
    reinterpret_cast<u32x4*>(dst)[e] = x;
  }
}
__device__ __forceinline__ void put16(float* dst, const u32x4& r, const float*) { *reinterpret_cast<u32x4*>(dst) = r; }

// Rows of D elements of up to TB tokens: global -> registers -> LDS as fp32.
template <int D, int NT, typename AT>
struct Rows {
  static constexpr int N = 16 / (int)sizeof(AT), CPR = D / N, U = (TB * CPR + NT - 1) / NT;
  u32x4 r[U];
  __device__ __forceinline__ void load(const AT* base, int64_t stride, int nt) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + NT * u, t = c / CPR;
      r[u] = u32x4{0, 0, 0, 0};
      if (t < nt) r[u] = *reinterpret_cast<const u32x4*>(base + t * stride + (c - t * CPR) * N);
    }
  }
  __device__ __forceinline__ void stage(float* lds, int nt) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + NT * u, t = c / CPR;
      if (t < nt) put16(lds + t * D + (c - t * CPR) * N, r[u], (const AT*)nullptr);
    }
  }
};

// NCC: columns of a lane: two in bf16 (8-byte loads and stores of the state), one
// in fp32.
template <typename AT> constexpr int lane_columns() { return sizeof(AT) == 2 ? 2 : 1; }

template <int DK, int DV, typename AT, int NCC = lane_columns<AT>()>
__global__ void __launch_bounds__(DV * 4 / NCC) scan_step_kernel(ScanParams p) {
  constexpr int NT = DV * 4 / NCC, MB = DK / 16;
  __shared__ __align__(16) float s_k[TB * DK], s_q[TB * DK], s_v[TB * DV], s_ad[2 * TB];

  const int i = blockIdx.x / p.H, h = blockIdx.x - i * p.H, g = h / (p.H / p.G);
  const int s0 = p.start[i], len = p.start[i + 1] - s0;
  // (a longer prompt belongs to the chunked form's launch; so that a refused
  // list is reported, the first prompt's workgroups go on to the checks)
  if (i > 0 && (unsigned)len > (unsigned)p.len_hi) return;
  const int b = p.seqs ? p.seqs[i] : i;
  const bool in = b >= 0 && b < p.B;

  const int tid = threadIdx.x, lane = tid & 63, cg = lane & 15, rg = lane >> 4;
  const int col0 = 16 * NCC * (tid >> 6), col = col0 + NCC * cg;
  float* Sg = p.S + ((size_t)(in ? b : 0) * p.H + h) * DK * DV + (size_t)(4 * rg) * DV + col;

  // the state's loads are in flight over the checks and the tokens' first loads
  float s[MB][NCC][4];
  if (in && (!p.has_state || p.has_state[i] != 0)) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float* at = Sg + (size_t)(16 * mb + v) * DV;
        if constexpr (NCC == 2) {
          float x[2];
          ldn_nt<2>(at, x);
          s[mb][0][v] = x[0];
          s[mb][1][v] = x[1];
        } else {
          s[mb][0][v] = *at;
        }
      }
  } else {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int c = 0; c < NCC; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) s[mb][c][v] = 0.f;
  }
  if (!prompt_ok(p, i, h, b) || len > p.len_hi) return;

  const AT* kp = reinterpret_cast<const AT*>(p.k) + s0 * p.ks + (int64_t)g * DK;
  const AT* qp = reinterpret_cast<const AT*>(p.q) + s0 * p.qs + (int64_t)g * DK;
  const AT* vp = reinterpret_cast<const AT*>(p.v) + s0 * p.vs + (int64_t)h * DV;
  const AT* dp = reinterpret_cast<const AT*>(p.gate) + s0 * p.gs + h;
  AT* op = reinterpret_cast<AT*>(p.o) + s0 * p.os + (int64_t)h * DV + col;
  const float rate = expf(p.A[h]);

  Rows<DK, NT, AT> rk, rq;
  Rows<DV, NT, AT> rv;
  float d = 0.f;
  auto fetch = [&](int t0, int nt) {
    rk.load(kp + t0 * p.ks, p.ks, nt);
    rq.load(qp + t0 * p.qs, p.qs, nt);
    rv.load(vp + t0 * p.vs, p.vs, nt);
    if (tid < nt) d = ld(dp + (t0 + tid) * p.gs);
  };
  int nt = len < TB ? len : TB;
  fetch(0, nt);

  for (int t0 = 0; t0 < len; t0 += TB) {
    rk.stage(s_k, nt);
    rq.stage(s_q, nt);
    rv.stage(s_v, nt);
    if (tid < nt) {
      s_ad[2 * tid] = expf(-d * rate);
      s_ad[2 * tid + 1] = d;
    }
    __syncthreads();
    const int now = nt, left = len - t0 - TB;
    if (left > 0) {                        // the next block's loads, in flight over this one
      nt = left < TB ? left : TB;
      fetch(t0 + TB, nt);
    }
#pragma unroll 1
    for (int j = 0; j < now; ++j) {
      float u[NCC];
      ldn<NCC>(s_v + j * DV + col, u);
      const float a = s_ad[2 * j], dt = s_ad[2 * j + 1];
#pragma unroll
      for (int c = 0; c < NCC; ++c) u[c] *= dt;
      float o[NCC];
#pragma unroll
      for (int c = 0; c < NCC; ++c) o[c] = 0.f;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        float kk[4], qq[4];
        ld4(s_k + j * DK + 16 * mb + 4 * rg, kk);
        ld4(s_q + j * DK + 16 * mb + 4 * rg, qq);
#pragma unroll
        for (int c = 0; c < NCC; ++c)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            s[mb][c][v] = a * s[mb][c][v] + kk[v] * u[c];
            o[c] += s[mb][c][v] * qq[v];
          }
      }
#pragma unroll
      for (int c = 0; c < NCC; ++c) o[c] = row_groups_sum(o[c]);
      if (rg == 0) stn<NCC>(op + (t0 + j) * p.os, o);
    }
    __syncthreads();
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float* at = Sg + (size_t)(16 * mb + v) * DV;
      if constexpr (NCC == 2) {
        const float x[2] = {s[mb][0][v], s[mb][1][v]};
        stn_nt<2>(at, x);
      } else {
        *at = s[mb][0][v];
      }
    }
  if (p.prime) sketch_tile<DK, DV, AT, NCC>(p.sk, s, b, h, col0, lane);
}

template <int DK, int DV>
int launch_shape(int act, const ScanParams& p, hipStream_t st) {
  const dim3 grid(p.nseq * p.H);
  if (act == DT_F32)
    hipLaunchKernelGGL((scan_step_kernel<DK, DV, float>), grid, dim3(DV * 4 / lane_columns<float>()), 0, st, p);
  else
    hipLaunchKernelGGL((scan_step_kernel<DK, DV, bf16>), grid, dim3(DV * 4 / lane_columns<bf16>()), 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_scan_step(int dk, int dv, int act, const ScanParams& p, hipStream_t st) {
  if (dk == 16 && dv == 32) return launch_shape<16, 32>(act, p, st);
  if (dk == 64 && dv == 64) return launch_shape<64, 64>(act, p, st);
  if (dk == 128 && dv == 64) return launch_shape<128, 64>(act, p, st);
  if (dk == 128 && dv == 128) return launch_shape<128, 128>(act, p, st);
  return -2;
}

}  // namespace sk
