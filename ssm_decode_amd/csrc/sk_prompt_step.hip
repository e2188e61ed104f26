// Prompts through the gated delta rule, one token at a time:
//   u = beta (v - alpha S^T k),  S <- alpha S + k u^T,  o = S^T q.
// One workgroup per (prompt, head); a wave holds 16 or 32 columns of the tile,
// all of its rows, in registers for the whole prompt (the columns of S never mix,
// so the waves of a tile meet only where the tokens are staged).
//
// A prompt of a few tokens is bound by its state's traffic (4 dk dv bytes in
// and out; 256 sequences of 32 heads of 128 x 128 by one token: 1.1 GB in 206 us,
// 5.3 TB/s), a longer one by the chain from token to token, so long ones take the
// chunked form (not dk = 16, whose tokens are short).
#include "sk_serve_device.hpp"

namespace sk {
namespace {

constexpr int TB = 16;    // tokens staged at a time

template <typename AT> struct Chunk16 { static constexpr int N = 16 / (int)sizeof(AT); };

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void put_chunk(float* dst, const u32x4& r, const bf16*) {
  const u32x4 a = {r[0] << 16, r[0] & 0xffff0000u, r[1] << 16, r[1] & 0xffff0000u};
  const u32x4 b = {r[2] << 16, r[2] & 0xffff0000u, r[3] << 16, r[3] & 0xffff0000u};
  reinterpret_cast<u32x4*>(dst)[0] = a;
  reinterpret_cast<u32x4*>(dst)[1] = b;
}
__device__ __forceinline__ void put_chunk(float* dst, const u32x4& r, const float*) {
  *reinterpret_cast<u32x4*>(dst) = r;
}

// Rows of D elements of up to TB tokens: global -> registers -> LDS as fp32.
template <int D, int NT, typename AT>
struct Rows {
  static constexpr int N = Chunk16<AT>::N, CPR = D / N, U = (TB * CPR + NT - 1) / NT;
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
      if (t < nt) put_chunk(lds + t * D + (c - t * CPR) * N, r[u], (const AT*)nullptr);
    }
  }
};

// NCC: columns of a lane.  Two in bf16 (8-byte loads and stores of the state);
// one in fp32, where the chain from token to token weighs more: half the
// arithmetic of a token, with its key and value read from LDS one token ahead
// (64 x 64 tiles, 0.36 us a token against 0.5 with two columns).
template <typename AT> constexpr int lane_columns() { return sizeof(AT) == 2 ? 2 : 1; }

template <int DK, int DV, typename AT, int NCC = lane_columns<AT>()>
__global__ void __launch_bounds__(DV * 4 / NCC) prompt_step_kernel(PromptParams p) {
  constexpr int NT = DV * 4 / NCC, MB = DK / 16;
  constexpr bool AHEAD = NCC == 1;
  __shared__ __align__(16) float s_k[TB * DK], s_q[TB * DK], s_v[TB * DV], s_ab[2 * TB];

  const int i = blockIdx.x / p.H, h = blockIdx.x - i * p.H;
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

  const AT* kp = reinterpret_cast<const AT*>(p.k) + s0 * p.ks + (int64_t)h * DK;
  const AT* qp = reinterpret_cast<const AT*>(p.q) + s0 * p.qs + (int64_t)h * DK;
  const AT* vp = reinterpret_cast<const AT*>(p.v) + s0 * p.vs + (int64_t)h * DV;
  const float* ap = p.gate + s0 * p.gs + h;
  const float* bp = p.beta + s0 * p.bs + h;
  AT* op = reinterpret_cast<AT*>(p.o) + s0 * p.os + (int64_t)h * DV + col;

  Rows<DK, NT, AT> rk, rq;
  Rows<DV, NT, AT> rv;
  float ab = 0.f;
  auto fetch = [&](int t0, int nt) {
    rk.load(kp + t0 * p.ks, p.ks, nt);
    rq.load(qp + t0 * p.qs, p.qs, nt);
    rv.load(vp + t0 * p.vs, p.vs, nt);
    if (tid < TB) {
      if (tid < nt) ab = ap[(t0 + tid) * p.gs];
    } else if (tid < 2 * TB && tid - TB < nt) {
      ab = bp[(t0 + tid - TB) * p.bs];
    }
  };
  int nt = len < TB ? len : TB;
  fetch(0, nt);

  for (int t0 = 0; t0 < len; t0 += TB) {
    rk.stage(s_k, nt);
    rq.stage(s_q, nt);
    rv.stage(s_v, nt);
    if (tid < 2 * TB) s_ab[tid] = ab;
    __syncthreads();
    const int now = nt, left = len - t0 - TB;
    if (left > 0) {                        // the next block's loads, in flight over this one
      nt = left < TB ? left : TB;
      fetch(t0 + TB, nt);
    }
    float kk[MB][4], vv[NCC], al, be;
    auto token = [&](int j) {                // a token's key, value and factors
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) ld4(s_k + j * DK + 16 * mb + 4 * rg, kk[mb]);
      ldn<NCC>(s_v + j * DV + col, vv);
      al = s_ab[j];
      be = s_ab[TB + j];
    };
    if (AHEAD) token(0);
#pragma unroll 1
    for (int j = 0; j < now; ++j) {
      if (!AHEAD) token(j);
      float qq[MB][4];
      auto query = [&]() {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) ld4(s_q + j * DK + 16 * mb + 4 * rg, qq[mb]);
      };
      if (AHEAD) query();
      float u[NCC];
#pragma unroll
      for (int c = 0; c < NCC; ++c) {
        float a = 0.f;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int v = 0; v < 4; ++v) a += s[mb][c][v] * kk[mb][v];
        u[c] = be * (vv[c] - al * row_groups_sum(a));
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int c = 0; c < NCC; ++c)
#pragma unroll
          for (int v = 0; v < 4; ++v) s[mb][c][v] = al * s[mb][c][v] + kk[mb][v] * u[c];
      if (AHEAD && j + 1 < now) token(j + 1);        // in flight over this token's output
      if (!AHEAD) query();
      float o[NCC];
#pragma unroll
      for (int c = 0; c < NCC; ++c) {
        float a = 0.f;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int v = 0; v < 4; ++v) a += s[mb][c][v] * qq[mb][v];
        o[c] = row_groups_sum(a);
      }
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
int launch_shape(int act, const PromptParams& p, hipStream_t st) {
  const dim3 grid(p.nseq * p.H);
  if (act == DT_F32)
    hipLaunchKernelGGL((prompt_step_kernel<DK, DV, float>), grid, dim3(DV * 4 / lane_columns<float>()), 0, st, p);
  else
    hipLaunchKernelGGL((prompt_step_kernel<DK, DV, bf16>), grid, dim3(DV * 4 / lane_columns<bf16>()), 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_prompt_step(int dk, int dv, int act, const PromptParams& p, hipStream_t st) {
  if (dk == 16 && dv == 32) return launch_shape<16, 32>(act, p, st);
  if (dk == 64 && dv == 64) return launch_shape<64, 64>(act, p, st);
  if (dk == 128 && dv == 64) return launch_shape<128, 64>(act, p, st);
  if (dk == 128 && dv == 128) return launch_shape<128, 128>(act, p, st);
  return -2;
}

}  // namespace sk
