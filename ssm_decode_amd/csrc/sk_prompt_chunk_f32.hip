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
// Bound by the matrix instructions: 64 x 64, 272 a wave and chunk at 32 cycles, 3.6
// of the 5.3 us that a chunk takes (47 us for 8; branches between the products and
// outputs stored in their own chunk took 11 more).  K and T, P are in LDS twice, Q
// once (its next copy starts when the chunk's outputs have it behind them), V
// comes to registers a chunk ahead.
#include <type_traits>

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

template <int DK, int DV>
__global__ void __launch_bounds__(64 * NW, 2) prompt_chunk_f32_kernel(PromptParams p) {
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
  const float* vp = reinterpret_cast<const float*>(p.v) + s0 * p.vs + (int64_t)h * DV + c0;      // (all uniform)
  float* op = reinterpret_cast<float*>(p.o) + s0 * p.os + (int64_t)h * DV + c0;
  const unsigned char* wp = reinterpret_cast<const unsigned char*>(p.work) +
                            ((size_t)first_slot(s0, rank, 6) * p.H + h) * CHUNK_WORK_F32;
  const uint32_t lds0 = lds_address(smem);

  // 64 rows of K or Q; 16-byte pieces swizzled by row.  A unit is 64 pieces.  In a
  // whole chunk a lane's offset from the unit's first row is the same in all of
  // a wave's units but for the swizzle, whose period is 16 rows.
  constexpr int RPU = 64 / PPR, KU = PPR / NW;   // rows of a unit, a wave's units
  auto swz = [&](int v) { return (uint32_t)((lane % PPR) ^ (((NW * v + wv) * RPU + lane / PPR) & 15)) * 16; };
  constexpr int PERIOD = 16 / (NW * RPU) > 0 ? 16 / (NW * RPU) : 1;
  const uint32_t krow = (uint32_t)(lane / PPR * p.ks * 4), qrow = (uint32_t)(lane / PPR * p.qs * 4);
  uint32_t sw[PERIOD];
#pragma unroll
  for (int v = 0; v < PERIOD; ++v) sw[v] = swz(v);
  const float *kc = kp + wv * RPU * p.ks, *qc = qp + wv * RPU * p.qs, *vc = vp;      // (uniform, of the next chunk)
  const int run0 = (wv * RUNS < WRUNS - RUNS ? wv * RUNS : WRUNS - RUNS) * 1024;     // (the last wave's runs end with the workspace)
  const unsigned char* wc = wp + run0;
  auto copy_k = [&](int v, uint32_t lds) { copy16(kc + v * NW * RPU * p.ks, krow + sw[v % PERIOD], lds + (NW * v + wv) * 1024); };
  auto copy_q = [&](int v, uint32_t lds) { copy16(qc + v * NW * RPU * p.qs, qrow + sw[v % PERIOD], lds + (NW * v + wv) * 1024); };
  auto copy_w = [&](int u, uint32_t lds) { copy16(wc + u * 1024, lane * 16, lds + run0 + u * 1024); };
  auto next_chunk = [&]() {
    kc += PC * p.ks;
    qc += PC * p.qs;
    vc += PC * p.vs;
    wc += (size_t)p.H * CHUNK_WORK_F32;
  };
  // .. and of a chunk that may be the prompt's last: rows behind its end repeat
  // its last one (their beta in T is 0, their columns of P meet only zeros)
  auto copy_rows = [&](const float* base, int64_t stride, int t0, uint32_t lds) {
    const int end = len - t0 < PC ? len - t0 - 1 : PC - 1;
#pragma unroll 1
    for (int v = 0; v < KU; ++v) {
      const int u = NW * v + wv, row0 = u * RPU, from = row0 < end ? row0 : end;      // (uniform)
      const int row = row0 + lane / PPR, left = (row < end ? row : end) - from;
      copy16(base + (t0 + from) * stride, (uint32_t)(left * stride * 4) + swz(v), lds + u * 1024);
    }
  };
  const uint32_t vo = (uint32_t)(4 * hi * p.vs + n) * 4;
  float vv[TB][4];
  auto load_v = [&](int tb) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      vv[tb][r] = *reinterpret_cast<const float*>(reinterpret_cast<const char*>(vc + (16 * tb + r) * p.vs) + vo);
  };
  auto load_v_last = [&](int t0) {
    const int end = len - t0 < PC ? len - t0 - 1 : PC - 1;
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * tb + 4 * hi + r;
        vv[tb][r] = vp[(t0 + (row < end ? row : end)) * p.vs + n];
      }
  };
  auto copy_last = [&](int t0, int buf) {        // (K, T and P)
    copy_rows(kp, p.ks, t0, lds0 + L::K + buf * L::KBYTES);
#pragma unroll
    for (int u = 0; u < RUNS; ++u) copy_w(u, lds0 + L::W + buf * L::WBYTES);
  };
  if (len > 0) {
    copy_last(0, 0);
    copy_rows(qp, p.qs, 0, lds0 + L::Q);
    load_v_last(0);
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

  // a chunk's outputs leave in the next chunk's time (the wait at its start
  // would wait for them too)
  float out[TB][4];
  const uint32_t oo = (uint32_t)(4 * hi * p.os + n) * 4;
  auto store_out = [&](int t0, int tb, int cnt) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (cnt >= PC || 16 * tb + 4 * hi + r < cnt)
        *reinterpret_cast<float*>(reinterpret_cast<char*>(op + (t0 + 16 * tb + r) * p.os) + oo) = out[tb][r];
  };

  // A lane's byte offsets into rows of K or Q: of four columns 16 kb + 4 hi .. of
  // row 16 tb + n (kb % 4 = m), and of column 16 mb + n of row 16 kb + 4 hi + r
  // (mb % 4 = m).  The swizzle leaves the rest of both indices to constants.
  constexpr int ROWB = DK * 4;
  uint32_t by_row[4], by_col[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    by_row[m] = n * ROWB + (4 * (m ^ (n >> 2)) + (hi ^ (n & 3))) * 16;
#pragma unroll
    for (int r = 0; r < 4; ++r) by_col[m][r] = (4 * hi + r) * ROWB + (4 * (m ^ hi) + ((n >> 2) ^ r)) * 16 + (n & 3) * 4;
  }

  // (as in bf16: columns where R is no finite number)
  int since = NEVER;
  int t0 = 0, buf = 0;
  // one chunk; `more`: a whole one follows.  Steps of up to 16 matrix
  // instructions, in each the reads of the next one's A operands.
  auto chunk = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;
    // this wave's copies for the chunk have landed, then everybody's; and
    // everybody has read the other buffers.  (V's loads too: the compiler, which
    // does not know of the copies, would wait for the next chunk's with them.)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) asm volatile("" : "+v"(vv[tb][r]));
    __syncthreads();
    const unsigned char *s_k = smem + L::K + buf * L::KBYTES, *s_q = smem + L::Q;
    const float* s_w = reinterpret_cast<const float*>(smem + L::W + buf * L::WBYTES);
    const float* s_g = s_w + 2 * F32_TILES * 256;
    const uint32_t knext = lds0 + L::K + (buf ^ 1) * L::KBYTES, wnext = lds0 + L::W + (buf ^ 1) * L::WBYTES;
    const bool tail = !MORE && len - t0 > PC;    // the prompt's end follows
    const f32x4s zero = {0.f, 0.f, 0.f, 0.f};

    float a[2][4][4], g[TB][4], d[TB][4];
    auto load_rows = [&](const unsigned char* s, int kb, int at) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb)
        ld4(reinterpret_cast<const float*>(s + by_row[kb & 3] + (kb >> 2) * 256 + tb * 16 * ROWB), a[at & 1][tb]);
    };
    // column kb of a triangle: tile (tb, kb) is the (tb (tb + 1) / 2 + kb)-th
    auto load_tri = [&](const float* m, int kb, int at) {
#pragma unroll
      for (int tb = kb; tb < TB; ++tb) ld4(m + (tb * (tb + 1) / 2 + kb) * 256 + lane * 4, a[at & 1][tb]);
    };
    auto load_kt = [&](int kb, int m0, int at) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          a[at & 1][m][r] = *reinterpret_cast<const float*>(s_k + by_col[m][r] + m0 * 64 + kb * 16 * ROWB);
    };
    auto times = [&](int at, const f32x4s& in, f32x4s* out, int from) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int m = from; m < 4; ++m) out[m] = mm4(a[at & 1][m][r], in[r], out[m]);
    };
    f32x4s R[TB], O[TB], U[TB];
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) R[tb] = O[tb] = U[tb] = zero;
    load_rows(s_k, 0, 0);
    next_chunk();
    __builtin_amdgcn_sched_barrier(0);
    if (tail) copy_last(t0 + PC, buf ^ 1);
    // K S
#pragma unroll
    for (int kb = 0; kb < MB; ++kb) {
      if (kb + 1 < MB) load_rows(s_k, kb + 1, kb + 1);
      else load_rows(s_q, 0, MB);
      if (kb < TB) ld4(s_g + 16 * kb + 4 * hi, g[kb]);
      times(kb, S[kb], R, 0);
      region<16, 1, 2>();
      if (MORE) {
#pragma unroll
        for (int u = kb * KU / MB; u < (kb + 1) * KU / MB; ++u) copy_k(u, knext);
#pragma unroll
        for (int u = kb * RUNS / MB; u < (kb + 1) * RUNS / MB; ++u) copy_w(u, wnext);
      }
    }
    // Q S;  R = V - g (K S) meanwhile
    int low = 16;
#pragma unroll
    for (int kb = 0; kb < MB; ++kb) {
      if (kb + 1 < MB) load_rows(s_q, kb + 1, kb + 1);
      else load_tri(s_w, 0, MB);
      if (kb < TB) {
        ld4(s_g + PC + 16 * kb + 4 * hi, d[kb]);
#pragma unroll
        for (int r = 3, l = 16; r >= 0; --r) {
          const float x = vv[kb][r] - g[kb][r] * R[kb][r];
          const bool ok = finite(x);
          l = ok ? l : 4 * kb + r;
          R[kb][r] = ok ? x : 0.f;
          if (r == 0) low = min(low, l);
        }
      }
      times(kb, S[kb], O, 0);
      region<16, 1, 2>();
    }
    if (t0 > 0) {
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) store_out(t0 - PC, tb, PC);
    }
    const float gC = column_poison(low < 16, s_g[PC - 1]);
    since = low < 16 && since == NEVER ? t0 + 16 * (low >> 2) + 4 * hi + (low & 3) : since;
    __syncthreads();                             // everybody has read Q
    if (tail) {
      copy_rows(qp, p.qs, t0 + PC, lds0 + L::Q);
      load_v_last(t0 + PC);
    }
    // U = T R;  S = g_C S and O = g O meanwhile
    constexpr int STEPS = 1 + MB / 4;            // of the last part, for each block of tokens
#pragma unroll
    for (int kb = 0; kb < TB; ++kb) {
      if (kb + 1 < TB) load_tri(s_w, kb + 1, kb + 1);
      else load_tri(s_w + F32_TILES * 256, 0, TB);
      times(kb, R[kb], U, kb);
#pragma unroll
      for (int r = 0; r < 4; ++r) O[kb][r] *= g[kb][r];
#pragma unroll
      for (int mb = kb * MB / TB; mb < (kb + 1) * MB / TB; ++mb)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[mb][r] *= gC;
      region<4 * (TB - 1), 1, 4>();
      if (MORE) {
#pragma unroll
        for (int u = kb * KU / TB; u < (kb + 1) * KU / TB; ++u) copy_q(u, lds0 + L::Q);
        load_v(kb);
      }
    }
    // O += P U;  S += K^T (D_C U)
#pragma unroll
    for (int kb = 0; kb < TB; ++kb) {
      load_kt(kb, 0, kb * STEPS + 1);
      times(kb * STEPS, U[kb], O, kb);
#pragma unroll
      for (int r = 0; r < 4; ++r) U[kb][r] *= d[kb][r];
      region<16, 2, 2>();
#pragma unroll
      for (int m0 = 0; m0 < MB; m0 += 4) {
        const int at = kb * STEPS + 1 + m0 / 4;
        if (m0 + 4 < MB) load_kt(kb, m0 + 4, at + 1);
        else if (kb + 1 < TB) load_tri(s_w + F32_TILES * 256, kb + 1, at + 1);
        times(at, U[kb], S + m0, 0);
        region<16, 1, 2>();
      }
    }
#pragma unroll
    for (int tb = 0; tb < TB; ++tb)
#pragma unroll
      for (int r = 0; r < 4; ++r) out[tb][r] = O[tb][r];
    t0 += PC;
    buf ^= 1;
  };
  while (len - t0 >= 2 * PC) chunk(std::true_type{});
  while (t0 < len) chunk(std::false_type{});
  if (len > 0) {
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) store_out(t0 - PC, tb, len - (t0 - PC));
  }

  if (__any(since != NEVER)) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int first = column_first(since);
    for (int64_t t = (int64_t)first + hi; t < len; t += 4) op[t * p.os + n] = __builtin_nanf("");
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
