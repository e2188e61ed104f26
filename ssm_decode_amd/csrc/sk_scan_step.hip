// Prompts through the selective state space scan, one token at a time:
//   S <- a S + k (dt v)^T,  a = exp(-dt exp(A_h)),  o = S^T q.
// One workgroup per (prompt, head); a wave holds 16 or 32 columns of the tile, all
// of its rows, in registers for the whole prompt (rows and columns of S never
// mix but in the output's sum over rows).
//
// The state is held as S = g S', g in (1, 2], and the logarithms of the decays are summed in 64
// bits: with x their sum to the base 2, negated, g is 2^(1 - (x - floor x)), and where
// floor x grows S' is scaled by that many powers of two, exactly.  So
//   S' <- S' + k (dt v / g)^T,  o = g (S'^T q),
// and no decay rounds the state.  (Each rounded, and its product with the state, steps
// that are alike err to one side: 16000 tokens of dt = 3e-4 put the state off by 8e-5 of itself.)
//
// A prompt of a few tokens is bound by its state's traffic (4 dk dv bytes in and
// out; 256 sequences of 128 heads of 128 x 64 by one token: 2.1 GB in 371 us, 5.7 TB/s), a
// longer one by the chain from token to token, so long ones take the chunked form, or,
// where there is none (fp32, dk = 16) and tiles are few, go in segments as the chunked
// form's: without outputs first, each from a zero state, then each from the state
// before it.
#include "sk_prompt_chunk.hpp"
#include "sk_scan_device.hpp"

namespace sk {
namespace {

constexpr int TB = 16;    // tokens staged at a time
constexpr int DTB = 64;   // .. and their decays: a lane each of one wave

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
  __device__ __forceinline__ void stage(float* lds) const {      // (zeros behind the end)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = threadIdx.x + NT * u, t = c / CPR;
      if (t < TB) put16(lds + t * D + (c - t * CPR) * N, r[u], (const AT*)nullptr);
    }
  }
};

// NCC: columns of a lane: two in bf16 (8-byte loads and stores of the state), one
// in fp32.
template <typename AT> constexpr int lane_columns() { return sizeof(AT) == 2 ? 2 : 1; }

// Tokens under way at once: nothing but the state goes from one to the next.  bf16: one,
// whose registers leave three waves a SIMD.  fp32: two where waves are few, in segments and
// for small heads (us, one and two: 8 prompts of 512 tokens with 16 heads of 64 x 64 67
// and 65, 32 of them, whole, 146 and 141; 8 with 16 heads of 128 x 64 125 and 116, 2 with
// 64 heads 106 and 107), else one (64 prompts of 200 tokens with 64 heads of 128 x 64 556
// and 604; 16 with heads of 128 x 128 274 and 364).
template <int DK, int DV, typename AT, bool SEG>
constexpr int tokens_at_once() { return sizeof(AT) == 4 && (SEG || DK * DV <= 64 * 64) ? 2 : 1; }

// (64 prompts of 5 tokens with 128 heads of 128 x 64 in fp32: 123 us, 136 with three waves)
template <int DK, int DV, typename AT, bool SEG>
constexpr int MIN_WAVES = sizeof(AT) == 4 && DK == 128 && DV == 64 && !SEG ? 4 : 1;

// A decay of less than 2^-1024 a token is zero (an infinite step would leave no sum).
constexpr double FORGOTTEN = 1024.;

// OUT: with outputs.  SEG: one workgroup per (segment, head); the first segment
// leaves the state that its prompt starts from in the last one's place, as in the
// chunked form.
template <int DK, int DV, typename AT, bool OUT, bool SEG, int NCC = lane_columns<AT>()>
__global__ void __launch_bounds__(DV * 4 / NCC, (MIN_WAVES<DK, DV, AT, SEG>)) scan_step_kernel(ScanParams p) {
  constexpr int NT = DV * 4 / NCC, MB = DK / 16, T = tokens_at_once<DK, DV, AT, SEG>();
  __shared__ __align__(16) float s_k[TB * DK], s_q[OUT ? TB * DK : 1], s_v[TB * DV], s_ad[4 * DTB];

  const int slot = blockIdx.x / p.H, h = blockIdx.x - slot * p.H, g = h / (p.H / p.G);
  int i = slot, rank = 0, seg = 0, segs = 1;
  if (SEG) {
    // (a refused list may have no prompt that any launch comes to: it is reported here)
    if (slot == 0) prompt_ok(p, 0, h, p.seqs ? p.seqs[0] : 0);
    i = slot_prompt(p, slot, p.seg_shift, &rank);
    if (i < 0) return;
  }
  int s0 = p.start[i], len = p.start[i + 1] - s0;
  // (a longer prompt belongs to the chunked form's launch; so that a refused
  // list is reported, the first prompt's workgroups go on to the checks)
  if (!SEG && i > 0 && (unsigned)len > (unsigned)p.len_hi) return;
  if (SEG) {
    seg = slot - first_slot(s0, rank, p.seg_shift);
    const int64_t from = (int64_t)seg << p.seg_shift;
    if (from >= len && seg > 0) return;
    segs = (int)(((int64_t)len + (1 << p.seg_shift) - 1) >> p.seg_shift);
    s0 += (int)from;
    len = len - from <= (1 << p.seg_shift) ? len - (int)from : 1 << p.seg_shift;
  }
  const bool last = seg + 1 >= segs;
  if (!OUT && last) return;
  const int b = p.seqs ? p.seqs[i] : i;
  const bool in = b >= 0 && b < p.B;

  const int tid = threadIdx.x, lane = tid & 63, cg = lane & 15, rg = lane >> 4;
  const int col0 = 16 * NCC * (tid >> 6), col = col0 + NCC * cg;
  float* Sg = p.S + ((size_t)(in ? b : 0) * p.H + h) * DK * DV + (size_t)(4 * rg) * DV + col;

  auto seg_at = [&](int at) { return p.seg + ((size_t)at * p.H + h) * DK * DV + (size_t)(4 * rg) * DV + col; };

  // (a wrong list has segments anywhere: nothing is read for one)
  if (SEG && !prompt_ok(p, i, h, b)) return;
  // the state's loads are in flight over the checks and the tokens' first loads
  float s[MB][NCC][4];
  const float* from = Sg;
  bool read = in && (!p.has_state || p.has_state[i] != 0);
  if (SEG) {
    if (seg > 0) {
      from = seg_at(slot - 1);
      read = OUT;
    } else if (OUT && !last) {
      from = seg_at(slot + segs - 1);
      read = true;
    }
  }
  if (read) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float* at = from + (size_t)(16 * mb + v) * DV;
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
  if (!SEG && (!prompt_ok(p, i, h, b) || len > p.len_hi)) return;
  auto write = [&](float* to) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float* at = to + (size_t)(16 * mb + v) * DV;
        if constexpr (NCC == 2) {
          const float x[2] = {s[mb][0][v], s[mb][1][v]};
          stn_nt<2>(at, x);
        } else {
          *at = s[mb][0][v];
        }
      }
  };
  if (SEG && !OUT && seg == 0) write(seg_at(slot + segs - 1));

  const AT* kp = reinterpret_cast<const AT*>(p.k) + s0 * p.ks + (int64_t)g * DK;
  const AT* qp = reinterpret_cast<const AT*>(p.q) + s0 * p.qs + (int64_t)g * DK;
  const AT* vp = reinterpret_cast<const AT*>(p.v) + s0 * p.vs + (int64_t)h * DV;
  const AT* dp = reinterpret_cast<const AT*>(p.gate) + s0 * p.gs + h;
  AT* op = reinterpret_cast<AT*>(p.o) + s0 * p.os + (int64_t)h * DV + col;
  // (finite also where exp(A) is not, so that a step of zero takes nothing)
  const float rate_log = p.A[h];
  const double rate = (double)expf(rate_log > 88.f ? 88.f : rate_log) * LOG2E;

  Rows<DK, NT, AT> rk, rq;
  Rows<DV, NT, AT> rv;
  float d = 0.f, g_last = 1.f;
  double frac = 0., gone = 0.;                   // x - floor x and floor x, of the tokens staged so far
  auto fetch = [&](int t0, int nt) {
    rk.load(kp + t0 * p.ks, p.ks, nt);
    if (OUT) rq.load(qp + t0 * p.qs, p.qs, nt);
    rv.load(vp + t0 * p.vs, p.vs, nt);
  };
  auto fetch_dt = [&](int t0) {                  // (behind the end nothing happens)
    d = tid < DTB && t0 + tid < len ? ld(dp + (t0 + tid) * p.gs) : 0.f;
  };
  int nt = len < TB ? len : TB;
  fetch(0, nt);
  fetch_dt(0);

  for (int t0 = 0; t0 < len; t0 += TB) {
    rk.stage(s_k);
    if (OUT) rq.stage(s_q);
    rv.stage(s_v);
    const float* s_now = s_ad + 4 * (t0 % DTB);
    if (t0 % DTB == 0 && tid < DTB) {
      double x = (double)d * rate;
      x = x > FORGOTTEN ? FORGOTTEN : x;
      const double at = frac + wave_prefix(x), whole = floor(at), part = at - whole;
      const double from = dpp_d<0x138>(whole), before = tid > 0 ? from : t0 > 0 ? 0. : -1.;
      // (wave_shr:1, in which all lanes take part; the first token's S' is half of S)
      const int drop = part == part ? (int)(whole - before) : 0;
      const f32x4s ad = {d * exp2_of(part - 1.), exp2_of(1. - part), ldexpf(1.f, -drop),
                         __uint_as_float((uint32_t)(__ballot(drop != 0) >> (tid & -TB)))};
      reinterpret_cast<f32x4s*>(s_ad)[tid] = ad;
      frac = wave_last(part);
      gone += wave_last(whole);
      fetch_dt(t0 + DTB);
    }
    __syncthreads();
    const int now = nt, left = len - t0 - TB;
    if (left > 0) {                        // the next block's loads, in flight over this one
      nt = left < TB ? left : TB;
      fetch(t0 + TB, nt);
    }
    g_last = s_now[4 * (TB - 1) + 1];
    const uint32_t drops = __builtin_amdgcn_readfirstlane(__float_as_uint(s_now[3]));
#pragma unroll 1
    for (int j0 = 0; j0 < now; j0 += T) {
      float u[T][NCC], o[T][NCC], o2[T][NCC], g[T], drop[T];       // (drop: the power of two that S' is scaled by)
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float x[4];
        ldn<NCC>(s_v + (j0 + t) * DV + col, u[t]);
        ld4(s_now + 4 * (j0 + t), x);
        g[t] = x[1];
        drop[t] = x[2];
#pragma unroll
        for (int c = 0; c < NCC; ++c) {
          u[t][c] *= x[0];
          o[t][c] = o2[t][c] = 0.f;
        }
      }
      if (drops >> j0 & 1) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int c = 0; c < NCC; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) s[mb][c][v] *= drop[0];
      }
      // row block mb of S' for token t, and its part of the output
      auto update = [&](int mb, int t, const float (&kk)[4], const float (&qq)[4]) {
#pragma unroll
        for (int c = 0; c < NCC; ++c)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (t > 0) s[mb][c][v] *= drop[t];
            s[mb][c][v] += kk[v] * u[t][c];
            if (OUT) (v & 1 ? o2 : o)[t][c] += s[mb][c][v] * qq[v];
          }
      };
      auto read = [&](int mb, int t, float (&kk)[4], float (&qq)[4]) {
        ld4(s_k + (j0 + t) * DK + 16 * mb + 4 * rg, kk);
        if (OUT) ld4(s_q + (j0 + t) * DK + 16 * mb + 4 * rg, qq);
      };
      if constexpr (T > 1) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int t = 0; t < T; ++t) {
            float kk[4], qq[4];
            read(mb, t, kk, qq);
            update(mb, t, kk, qq);
          }
      } else {                                   // (one token: the next row blocks' are read ahead)
        constexpr int N = sizeof(AT) == 2 ? 2 : 3;
        float kk[N][4], qq[N][4];
#pragma unroll
        for (int mb = 0; mb < N - 1 && mb < MB; ++mb) read(mb, 0, kk[mb], qq[mb]);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const int far = mb + N - 1;
          if (far < MB) read(far, 0, kk[far % N], qq[far % N]);
          update(mb, 0, kk[mb % N], qq[mb % N]);
        }
      }
      if (!OUT) continue;
#pragma unroll
      for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int c = 0; c < NCC; ++c) o[t][c] = g[t] * row_groups_sum(o[t][c] + o2[t][c]);
        if (rg == 0 && j0 + t < now) stn<NCC>(op + (t0 + j0 + t) * p.os, o[t]);
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int c = 0; c < NCC; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) s[mb][c][v] *= g_last;
  if (!OUT) {
    write(seg_at(slot));
    if (tid == 0) p.seg_decay[(size_t)slot * p.H + h] = exp2_of(-(gone + frac));
    return;
  }
  if (!last) return;                             // (the state behind a segment is known already)
  write(Sg);
  if (p.prime) sketch_tile<DK, DV, AT, NCC>(p.sk, s, b, h, col0, lane);
}

template <int DK, int DV, typename AT>
int launch_type(const ScanParams& p, hipStream_t st) {
  const dim3 block(DV * 4 / lane_columns<AT>());
  if (p.nchunked > 0 && p.seg_shift) {           // (p.nchunked: all prompts, in segments)
    const dim3 grid(p.nsegs * p.H);
    hipLaunchKernelGGL((scan_step_kernel<DK, DV, AT, false, true>), grid, block, 0, st, p);
    if (int rc = launch_scan_join(DK, DV, p, st)) return rc;
    hipLaunchKernelGGL((scan_step_kernel<DK, DV, AT, true, true>), grid, block, 0, st, p);
  } else {
    hipLaunchKernelGGL((scan_step_kernel<DK, DV, AT, true, false>), dim3(p.nseq * p.H), block, 0, st, p);
  }
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <int DK, int DV>
int launch_shape(int act, const ScanParams& p, hipStream_t st) {
  return act == DT_F32 ? launch_type<DK, DV, float>(p, st) : launch_type<DK, DV, bf16>(p, st);
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
