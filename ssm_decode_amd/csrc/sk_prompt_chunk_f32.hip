// Prompts with fp32 activations, chunk after chunk (sk_prompt_chunk.hpp has the
// mathematics and the launch before this one).
//
// One workgroup of four waves per (prompt, head, 64 columns); a wave holds 16
// columns of the state, all rows, as tiles of v_mfma_f32_16x16x4_f32: lane
// (hi = lane / 16, n = lane % 16) has rows 4 hi + r of column n.  A tile is the
// B operand of the next product as it stands, with K-step r over rows 4 k + r, so
// nothing moves between K S, T R, P U and K^T U; the A operands are runs of
// four columns from LDS (of K^T, single values: four rows of 16 in 64 banks).
//
// Bound by the matrix instructions: 2 (3 dk dv + 40 dv) 64 operations a chunk
// beside the triangles, of 32 cycles for 2048.  K and T, P are in LDS twice, Q
// once (its next copy starts when the chunk's outputs have it behind them), V
// comes to registers a chunk ahead.
#include "sk_prompt_chunk.hpp"

namespace sk {
namespace {

constexpr int NW = 4;                            // waves of a workgroup
constexpr int WRUNS = (CHUNK_WORK_F32 + PROMPT_WORK_OVER) / 1024, RUNS = (WRUNS + NW - 1) / NW;
static_assert((CHUNK_WORK_F32 + PROMPT_WORK_OVER) % 1024 == 0, "runs");

template <int DK>
struct F32Lds {
  static constexpr int K = 0, KBYTES = PC * DK * 4;
  static constexpr int Q = K + 2 * KBYTES;
  static constexpr int W = Q + KBYTES, WBYTES = WRUNS * 1024;
  static constexpr int BYTES = W + 2 * WBYTES;
  static_assert(BYTES <= 160 * 1024, "LDS of a CU");
};

__device__ __forceinline__ f32x4s mm4(float a, float b, f32x4s c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <int DK, int DV>
__global__ void __launch_bounds__(64 * NW, 1) prompt_chunk_f32_kernel(PromptParams p) {
  using L = F32Lds<DK>;
  constexpr int PPR = DK / 4, MB = DK / 16, TB = PC / 16, PARTS = DV / (16 * NW);
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, hi = lane >> 4;
  // (the parts of a tile on one XCD, as in bf16)
  const int part = blockIdx.x / 8 % PARTS, tile = blockIdx.x / (8 * PARTS) * 8 + blockIdx.x % 8;
  if (tile >= p.nchunked * p.H) return;
  const int h = tile % p.H;
  int rank = 0;
  const int i = chunked_prompt(p, tile / p.H, &rank);
  if (i < 0) return;
  const int s0 = p.start[i], len = p.start[i + 1] - s0;
  const int b = p.seqs ? p.seqs[i] : i;
  if (!prompt_ok(p, i, h, b)) return;

  const int c0 = part * NW * 16 + wv * 16;       // the wave's first column
  const float* kp = reinterpret_cast<const float*>(p.k) + s0 * p.ks + (int64_t)h * DK;
  const float* qp = reinterpret_cast<const float*>(p.q) + s0 * p.qs + (int64_t)h * DK;
  const float* vp = reinterpret_cast<const float*>(p.v) + s0 * p.vs + (int64_t)h * DV + c0 + n;
  float* op = reinterpret_cast<float*>(p.o) + s0 * p.os + (int64_t)h * DV + c0 + n;
  const unsigned char* wp = reinterpret_cast<const unsigned char*>(p.work) +
                            ((size_t)first_slot(s0, rank, 6) * p.H + h) * CHUNK_WORK_F32;
  const uint32_t lds0 = lds_address(smem);

  // 64 rows of K or Q from token t0 on; 16-byte pieces swizzled by row.  A unit
  // is 64 pieces; rows behind the prompt's end repeat its last one (their beta
  // in T is 0, their columns of P meet only zeros).
  auto piece = [](int row, int pc) { return row * PPR + (pc ^ (row & 15)); };
  auto copy_rows = [&](const float* base, int64_t stride, int t0, uint32_t lds) {
    constexpr int RPU = 64 / PPR;                // rows of a unit
    const int end = len - t0 < PC ? len - t0 - 1 : PC - 1;
#pragma unroll
    for (int v = 0; v < PPR / NW; ++v) {
      const int u = NW * v + wv, row0 = u * RPU, from = row0 < end ? row0 : end;      // (uniform)
      const int row = row0 + lane / PPR, left = (row < end ? row : end) - from;
      copy16(base + (t0 + from) * stride, (uint32_t)(left * stride * 4) + (uint32_t)((lane % PPR) ^ (row & 15)) * 16,
             lds + u * 1024);
    }
  };
  auto copy_work = [&](int t0, uint32_t lds) {   // (the last wave's runs end with the workspace)
    const int run0 = wv * RUNS < WRUNS - RUNS ? wv * RUNS : WRUNS - RUNS;
    const unsigned char* w = wp + (size_t)(t0 / PC) * p.H * CHUNK_WORK_F32 + run0 * 1024;
#pragma unroll
    for (int u = 0; u < RUNS; ++u) copy16(w + u * 1024, lane * 16, lds + (run0 + u) * 1024);
  };
  float vv[TB][4];
  auto load_v = [&](int t0) {
    const int end = len - t0 < PC ? len - t0 - 1 : PC - 1;
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * tb + 4 * hi + r;
        vv[tb][r] = vp[(t0 + (row < end ? row : end)) * p.vs];
      }
  };
  if (len > 0) {
    copy_rows(kp, p.ks, 0, lds0 + L::K);
    copy_rows(qp, p.qs, 0, lds0 + L::Q);
    copy_work(0, lds0 + L::W);
    load_v(0);
  }

  float* Sg = p.S + ((size_t)b * p.H + h) * DK * DV + (size_t)(4 * hi) * DV + c0 + n;
  f32x4s S[MB];
  {
    const bool read = !p.has_state || p.has_state[i] != 0;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[mb][r] = read ? Sg[(size_t)(16 * mb + r) * DV] : 0.f;
  }

  int buf = 0;
  for (int t0 = 0; t0 < len; t0 += PC, buf ^= 1) {
    // this wave's copies for the chunk have landed, then everybody's; and
    // everybody has read the other buffers
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const bool more = len - t0 > PC;
    if (more) {
      copy_rows(kp, p.ks, t0 + PC, lds0 + L::K + (buf ^ 1) * L::KBYTES);
      copy_work(t0 + PC, lds0 + L::W + (buf ^ 1) * L::WBYTES);
    }
    const float* s_k = reinterpret_cast<const float*>(smem + L::K + buf * L::KBYTES);
    const float* s_q = reinterpret_cast<const float*>(smem + L::Q);
    const float* s_w = reinterpret_cast<const float*>(smem + L::W + buf * L::WBYTES);
    const float* s_g = s_w + 2 * F32_TILES * 256;
    const f32x4s zero = {0.f, 0.f, 0.f, 0.f};
    f32x4s R[TB], O[TB], U[TB];
    // K S and Q S
    auto times_state = [&](const float* m, f32x4s (&out)[TB]) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) out[tb] = zero;
#pragma unroll
      for (int kb = 0; kb < MB; ++kb) {
        float a[TB][4];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) ld4(m + piece(16 * tb + n, 4 * kb + hi) * 4, a[tb]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int tb = 0; tb < TB; ++tb) out[tb] = mm4(a[tb][r], S[kb][r], out[tb]);
      }
    };
    times_state(s_q, O);
    __syncthreads();                             // everybody has read Q
    if (more) copy_rows(qp, p.qs, t0 + PC, lds0 + L::Q);
    times_state(s_k, R);
    float g[TB][4];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      ld4(s_g + 16 * tb + 4 * hi, g[tb]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        R[tb][r] = vv[tb][r] - g[tb][r] * R[tb][r];
        O[tb][r] *= g[tb][r];
      }
    }
    if (more) load_v(t0 + PC);
    // U = T R, O += P U: tile (tb, kb) is the (tb (tb + 1) / 2 + kb)-th
    auto triangle = [&](const float* m, const f32x4s (&in)[TB], f32x4s (&out)[TB]) {
#pragma unroll
      for (int kb = 0; kb < TB; ++kb) {
        float a[TB][4];
#pragma unroll
        for (int tb = kb; tb < TB; ++tb) ld4(m + (tb * (tb + 1) / 2 + kb) * 256 + lane * 4, a[tb]);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int tb = kb; tb < TB; ++tb) out[tb] = mm4(a[tb][r], in[kb][r], out[tb]);
      }
    };
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) U[tb] = zero;
    triangle(s_w, R, U);
    triangle(s_w + F32_TILES * 256, U, O);
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * tb + 4 * hi + r;
        if (t0 + row < len) op[(t0 + row) * p.os] = O[tb][r];
      }
    // S = g_C S + K^T (D_C U)
    const float gC = s_g[PC - 1];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      float d[4];
      ld4(s_g + PC + 16 * tb + 4 * hi, d);
#pragma unroll
      for (int r = 0; r < 4; ++r) U[tb][r] *= d[r];
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[mb][r] *= gC;
#pragma unroll
    for (int kb = 0; kb < TB; ++kb)
#pragma unroll
      for (int m0 = 0; m0 < MB; m0 += 4) {
        float a[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            a[m][r] = s_k[piece(16 * kb + 4 * hi + r, 4 * (m0 + m) + (n >> 2)) * 4 + (n & 3)];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int m = 0; m < 4; ++m) S[m0 + m] = mm4(a[m][r], U[kb][r], S[m0 + m]);
      }
  }

  float s[MB][1][4];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[mb][0][r] = S[mb][r];
      Sg[(size_t)(16 * mb + r) * DV] = S[mb][r];
    }
  if (p.prime) sketch_tile<DK, DV, float, 1>(p.sk, s, b, h, c0, lane);
}

template <int DK, int DV>
int launch(const PromptParams& p, hipStream_t st) {
  const unsigned tiles = (unsigned)p.nchunked * p.H;
  constexpr unsigned PARTS = DV / (16 * NW);
  hipLaunchKernelGGL((prompt_chunk_f32_kernel<DK, DV>), dim3((tiles + 7) / 8 * 8 * PARTS), dim3(64 * NW),
                     (F32Lds<DK>::BYTES), st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_prompt_chunks_f32(int dk, int dv, const PromptParams& p, hipStream_t st) {
  if (dk == 64 && dv == 64) return launch<64, 64>(p, st);
  if (dk == 128 && dv == 64) return launch<128, 64>(p, st);
  if (dk == 128 && dv == 128) return launch<128, 128>(p, st);
  return -2;
}

}  // namespace sk
