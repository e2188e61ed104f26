// The two launches of the chunked form (see sk_prompt_chunk.hpp).
#include "sk_prompt_chunk.hpp"

namespace sk {
namespace {

// ------------------------------------------------------------ T and P
// One workgroup of four waves per (chunk slot, head).  K K^T and Q K^T on the
// bf16 matrix cores (exact products, fp32 sums); the unit triangular inverse
// by substitution in 16 x 16 blocks, joined to 32 and 64 by fp32 products.
constexpr int LS = PC + 4;                       // row stride of the fp32 matrices in LDS

template <int DK, int CW>
__global__ void __launch_bounds__(256) prompt_prep_kernel(PromptParams p) {
  constexpr int KB = PC * DK * 2;                // bytes of K or Q in LDS
  constexpr int MB = PC * LS * 4;                // bytes of A or P in LDS
  constexpr int BIG = 2 * KB > 2 * MB ? 2 * KB : 2 * MB;
  __shared__ __align__(16) unsigned char s_big[BIG];   // K and Q, then A (T in its place) and P
  __shared__ float s_al[PC], s_be[PC], s_pre[PC], s_suf[PC], s_blk[4], s_din[PC * 17];
  float* s_A = reinterpret_cast<float*>(s_big);
  float* s_P = reinterpret_cast<float*>(s_big + MB);

  const int slot = blockIdx.x / p.H, h = blockIdx.x - slot * p.H;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  // the last prompt whose first slot is not behind this one
  int i = -1;
  for (int j0 = 0; j0 < p.nseq; j0 += 64) {
    const int j = j0 + lane;
    const unsigned long long m = __ballot(j < p.nseq && first_slot(p.start[j < p.nseq ? j : 0], j) <= slot);
    if (m) i = j0 + 63 - __clzll(m);
  }
  if (i < 0) return;
  const int s0 = p.start[i], s1 = p.start[i + 1];
  if (s0 < 0 || s1 < s0 || s1 > p.tokens) return;      // (reported by the other launch)
  const int c0 = (slot - first_slot(s0, i)) * PC, len = s1 - s0;
  if (c0 >= len || len <= p.len_lo) return;
  const int nt = len - c0 < PC ? len - c0 : PC;
  const int64_t tok = (int64_t)s0 + c0;

  // K and Q, rows of DK with their 16-byte pieces swizzled, zeros behind nt
  constexpr int PPR = DK / 8;
  auto piece = [](int row, int pc) { return row * PPR + (pc ^ ((PPR == 16 ? row : row >> 1) & (PPR - 1))); };
  u32x4* s_k = reinterpret_cast<u32x4*>(s_big);
  u32x4* s_q = reinterpret_cast<u32x4*>(s_big + KB);
  const bf16* kp = reinterpret_cast<const bf16*>(p.k) + tok * p.ks + (int64_t)h * DK;
  const bf16* qp = reinterpret_cast<const bf16*>(p.q) + tok * p.qs + (int64_t)h * DK;
#pragma unroll
  for (int u = 0; u < PC * PPR / 256; ++u) {
    const int c = tid + 256 * u, row = c / PPR, pc = c % PPR;
    u32x4 a = u32x4{0, 0, 0, 0}, b = a;
    if (row < nt) {
      a = *reinterpret_cast<const u32x4*>(kp + row * p.ks + pc * 8);
      b = *reinterpret_cast<const u32x4*>(qp + row * p.qs + pc * 8);
    }
    s_k[piece(row, pc)] = a;
    s_q[piece(row, pc)] = b;
  }
  if (tid < PC) {
    s_al[tid] = tid < nt ? p.gate[(tok + tid) * p.gs + h] : 1.f;
    s_be[tid] = tid < nt ? p.beta[(tok + tid) * p.bs + h] : 0.f;
  }
  __syncthreads();

  // decays: within blocks of 16 (D_ij for i, j of a block), from a block's
  // start up to i, after j up to its end, and over whole blocks
  if (wv == 0) {
    const int b = lane >> 4, jl = lane & 15;
    float d = 1.f, pre = s_al[16 * b];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const float a = s_al[16 * b + t];
      if (t > jl) d *= a;
      s_din[(16 * b + t) * 17 + jl] = t >= jl ? d : 0.f;
      if (t > 0 && t <= jl) pre *= a;
    }
    s_suf[lane] = d;
    s_pre[lane] = pre;
    if (jl == 15) s_blk[b] = pre;
  }
  __syncthreads();

  // tiles (ti, tj), tj <= ti, of K K^T and Q K^T
  f32x4s ak[3], aq[3];
  const int cg = lane & 15, g = lane >> 4;
  auto tile_of = [](int t, int* ti, int* tj) {
    *ti = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    *tj = t - *ti * (*ti + 1) / 2;
  };
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    const int t = wv + 4 * n;
    ak[n] = aq[n] = f32x4s{0.f, 0.f, 0.f, 0.f};
    if (t < 10) {                                       // uniform over the wave
      int ti, tj;
      tile_of(t, &ti, &tj);
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const bf16x8 fk = as_frag(s_k[piece(16 * ti + cg, 4 * s + g)]);
        const bf16x8 fq = as_frag(s_q[piece(16 * ti + cg, 4 * s + g)]);
        const bf16x8 fb = as_frag(s_k[piece(16 * tj + cg, 4 * s + g)]);
        ak[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fk, fb, ak[n], 0, 0, 0);
        aq[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq, fb, aq[n], 0, 0, 0);
      }
    }
  }
  __syncthreads();                                      // K and Q are read: A and P over them
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    const int t = wv + 4 * n;
    if (t < 10) {
      int ti, tj;
      tile_of(t, &ti, &tj);
      float mid = 1.f;
      for (int b = tj + 1; b < ti; ++b) mid *= s_blk[b];
      const int j = 16 * tj + cg;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int ii = 16 * ti + 4 * g + r;
        const float D = ti == tj ? s_din[ii * 17 + cg] : s_pre[ii] * mid * s_suf[j];
        // (selected, not multiplied by a zero: nothing above the diagonal may
        // reach the sums)
        s_A[ii * LS + j] = j < ii ? s_be[ii] * D * ak[n][r] : 0.f;
        s_P[ii * LS + j] = j <= ii ? D * aq[n][r] : 0.f;
      }
    }
  }
  // the 16 x 16 blocks above the diagonal that fragments cover: (0, 1), (2, 3)
  for (int c = tid; c < 2 * 256; c += 256) {
    const int b = c >> 8, r = (c >> 4) & 15, cc = c & 15;
    s_A[(32 * b + r) * LS + 32 * b + 16 + cc] = 0.f;
    s_P[(32 * b + r) * LS + 32 * b + 16 + cc] = 0.f;
  }
  __syncthreads();

  // inverses of the four diagonal blocks: lane = (block, column), by rows
  float x[16];
  if (wv == 0) {
    const float* A = s_A + (16 * g) * LS + 16 * g;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float a = r == cg ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < r; j += 4) {
        float row[4];
        ld4(A + r * LS + j, row);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < r) a -= row[e] * x[j + e];
      }
      x[r] = a;
    }
    wave_lds_sync();
#pragma unroll
    for (int r = 0; r < 16; ++r) s_A[(16 * g + r) * LS + 16 * g + cg] = x[r];
  }
  __syncthreads();
  // T_21 = -T_22 (A_21 T_11): products of 16 x 16 blocks.  The result of one
  // (rows 4 g + r of column cg) is the next one's B operand with K-step r over
  // rows {4 k + r}, so A operands are read at column 4 g + r.
  auto mul16 = [&](const float* a, const f32x4s& b, f32x4s acc) {       // a: LDS block, b: registers
    float row[4];
    ld4(a + cg * LS + 4 * g, row);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(row[r], b[r], acc, 0, 0, 0);
    return acc;
  };
  auto load16 = [&](const float* b) {                                   // rows 4 g + r of column cg
    f32x4s v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = b[(4 * g + r) * LS + cg];
    return v;
  };
  auto store16 = [&](float* b, const f32x4s& v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) b[(4 * g + r) * LS + cg] = -v[r];
  };
  const f32x4s zero = {0.f, 0.f, 0.f, 0.f};
  auto blk = [&](int bi, int bj) { return s_A + 16 * bi * LS + 16 * bj; };
  if (wv < 2) {
    const int b = 2 * wv;
    const f32x4s X = mul16(blk(b + 1, b), load16(blk(b, b)), zero);
    const f32x4s Y = mul16(blk(b + 1, b + 1), X, zero);
    wave_lds_sync();
    store16(blk(b + 1, b), Y);
  }
  __syncthreads();
  {
    const int bi = wv >> 1, bj = wv & 1;                 // of the 32 x 32 block below the diagonal
    f32x4s X0 = mul16(blk(2, bj), load16(blk(bj, bj)), zero);
    f32x4s X1 = mul16(blk(3, bj), load16(blk(bj, bj)), zero);
    if (bj == 0) {
      const f32x4s t10 = load16(blk(1, 0));
      X0 = mul16(blk(2, 1), t10, X0);
      X1 = mul16(blk(3, 1), t10, X1);
    }
    f32x4s Y = mul16(blk(2 + bi, 2), X0, zero);
    if (bi == 1) Y = mul16(blk(3, 3), X1, Y);
    __syncthreads();
    store16(blk(2 + bi, bj), Y);
  }
  __syncthreads();

  // fragments of T diag(beta) and P, and the row factors
  unsigned char* W = reinterpret_cast<unsigned char*>(p.work) + ((size_t)slot * p.H + h) * CHUNK_WORK_BYTES;
  for (int c = tid; c < FRAGS * 64; c += 256) {
    const int f = c >> 6, ln = c & 63, pair = f >> 1;
    const int rb = pair > 0, kb = pair == 2;
    int row, k;
    frag_at<CW>(ln, f & 1, &row, &k);
    row += 32 * rb;
    k += 32 * kb;
    float t[8], v[8], a4[4];
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      ld4(s_A + row * LS + k + e, a4);
#pragma unroll
      for (int d = 0; d < 4; ++d) t[e + d] = a4[d] * s_be[k + e + d];
      ld4(s_P + row * LS + k + e, a4);
#pragma unroll
      for (int d = 0; d < 4; ++d) v[e + d] = a4[d];
    }
    bf16x8 ts[3], ps[2];
    split8<3>(t, ts);
    split8<2>(v, ps);
#pragma unroll
    for (int n = 0; n < 3; ++n)
      *reinterpret_cast<bf16x8*>(W + (f * 3 + n) * FRAG_BYTES + ln * 16) = ts[n];
#pragma unroll
    for (int n = 0; n < 2; ++n)
      *reinterpret_cast<bf16x8*>(W + T_BYTES + (f * 2 + n) * FRAG_BYTES + ln * 16) = ps[n];
  }
  if (tid < PC) {
    const int b = tid >> 4;
    float pre = s_pre[tid], suf = s_suf[tid];
    for (int n = 0; n < b; ++n) pre *= s_blk[n];
    for (int n = b + 1; n < 4; ++n) suf *= s_blk[n];
    float* G = reinterpret_cast<float*>(W + T_BYTES + P_BYTES);
    G[tid] = pre;
    G[PC + tid] = suf;
  }
}

// ------------------------------------------------------ chunk after chunk
// One workgroup of four waves per (prompt, head, part of the columns); a wave
// holds CW columns of the state, all rows, in registers.  K, Q, K^T, T and P
// are staged in LDS for the four waves; the next chunk's loads are in flight
// over the present one.
template <int DK, int DV, int CW>
struct ChunkLds {
  static constexpr int VC = 4 * CW;              // columns of the workgroup
  static constexpr int K = 0;
  static constexpr int Q = K + PC * DK * 2;
  static constexpr int KT = Q + PC * DK * 2;
  static constexpr int V = KT + PC * DK * 2;     // wave after wave: [64][CW], then the outputs
  static constexpr int W = V + PC * VC * 2;      // a chunk's workspace as it is
  static constexpr int BYTES = W + CHUNK_WORK_BYTES;
};

template <int DK, int DV, int CW>
__global__ void __launch_bounds__(256, 1) prompt_chunk_kernel(PromptParams p) {
  using M = Mf<CW>;
  using L = ChunkLds<DK, DV, CW>;
  typedef typename M::Acc Acc;
  constexpr int VC = L::VC, PARTS = DV / VC, PPR = DK / 8, NB = M::NB, DB = DK / 32;
  constexpr int AR = NB / M::TILES;              // registers of a tile
  __shared__ __align__(16) unsigned char smem[L::BYTES];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  int bid = blockIdx.x;
  const int part = bid % PARTS;
  bid /= PARTS;
  const int i = bid / p.H, h = bid - i * p.H;
  if ((int64_t)p.start[i + 1] - p.start[i] <= p.len_lo) return;
  const PromptTile pt = prompt_tile(p, i, h);
  if (!pt.ok) return;

  const int n = lane % M::MT, hi = lane / M::MT;           // column, part of the k axis
  const int col = part * VC + wv * CW + n;
  float* Sg = p.S + ((size_t)pt.b * p.H + h) * DK * DV + col;

  // the state, block after block of 32 rows
  Acc S[DB][M::TILES];
  const bool cont = !p.has_state || p.has_state[i] != 0;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < NB; ++r)
      S[db][r / AR][r % AR] = cont ? Sg[(size_t)(32 * db + M::index(lane, r)) * DV] : 0.f;

  // staging: a thread takes eight columns of four consecutive tokens of K (so
  // that it can write K^T in runs of four tokens), any pieces of the rest
  const bf16* kp = reinterpret_cast<const bf16*>(p.k) + pt.s0 * p.ks + (int64_t)h * DK;
  const bf16* qp = reinterpret_cast<const bf16*>(p.q) + pt.s0 * p.qs + (int64_t)h * DK;
  const bf16* vp = reinterpret_cast<const bf16*>(p.v) + pt.s0 * p.vs + (int64_t)h * DV + part * VC + wv * CW;
  bf16* op = reinterpret_cast<bf16*>(p.o) + pt.s0 * p.os + (int64_t)h * DV + part * VC + wv * CW;
  const unsigned char* wp = reinterpret_cast<const unsigned char*>(p.work) +
                            ((size_t)first_slot(pt.s0, i) * p.H + h) * CHUNK_WORK_BYTES;
  constexpr int KT4 = PC * PPR / 4 / 256 > 0 ? PC * PPR / 4 / 256 : 1;   // groups of four tokens a thread
  constexpr int QU = PC * PPR / 256;
  constexpr int VPR = CW / 8, VU = PC * VPR / 64;                         // pieces of a row, of a lane
  constexpr int WU = (CHUNK_WORK_BYTES / 16 + 255) / 256;
  constexpr bool KALL = PC * PPR / 4 >= 256;
  u32x4 rk[KT4][4], rq[QU], rv[VU], rw[WU];
  const u32x4 none = u32x4{0, 0, 0, 0};
  auto fetch = [&](int t0, int nt) {
#pragma unroll
    for (int u = 0; u < KT4; ++u) {
      const int c = tid + 256 * u, t4 = c / PPR * 4, pc = c % PPR;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rk[u][e] = none;
        if ((KALL || t4 < PC) && t4 + e < nt)
          rk[u][e] = *reinterpret_cast<const u32x4*>(kp + (t0 + t4 + e) * p.ks + pc * 8);
      }
    }
#pragma unroll
    for (int u = 0; u < QU; ++u) {
      const int c = tid + 256 * u, t = c / PPR, pc = c % PPR;
      rq[u] = none;
      if (t < nt) rq[u] = *reinterpret_cast<const u32x4*>(qp + (t0 + t) * p.qs + pc * 8);
    }
#pragma unroll
    for (int u = 0; u < VU; ++u) {
      const int c = lane + 64 * u, t = c / VPR, pc = c % VPR;
      rv[u] = none;
      if (t < nt) rv[u] = *reinterpret_cast<const u32x4*>(vp + (t0 + t) * p.vs + pc * 8);
    }
    const u32x4* w = reinterpret_cast<const u32x4*>(wp + (size_t)(t0 / PC) * p.H * CHUNK_WORK_BYTES);
#pragma unroll
    for (int u = 0; u < WU; ++u) {
      const int c = tid + 256 * u;
      rw[u] = w[c < CHUNK_WORK_BYTES / 16 ? c : 0];
    }
  };
  u32x4* s_k = reinterpret_cast<u32x4*>(smem + L::K);
  u32x4* s_q = reinterpret_cast<u32x4*>(smem + L::Q);
  unsigned char* s_kt = smem + L::KT;
  bf16* s_v = reinterpret_cast<bf16*>(smem + L::V) + wv * PC * CW;
  u32x4* s_w = reinterpret_cast<u32x4*>(smem + L::W);
  const float* s_g = reinterpret_cast<const float*>(smem + L::W + T_BYTES + P_BYTES);
  auto piece = [](int row, int pc) {
    return row * PPR + (pc ^ ((PPR == 16 ? M::swizzle(row) : M::swizzle(row) >> 1) & (PPR - 1)));
  };
  // K^T rows of 64 tokens (128 bytes, eight pieces): swizzled so that both the
  // writes (rows eight apart) and the reads (neighbouring rows) spread
  auto kt_piece = [](int d, int pc) { return d * 8 + (pc ^ (((d >> 1) ^ (d >> 4)) & 7)); };
  auto stage = [&]() {
#pragma unroll
    for (int u = 0; u < KT4; ++u) {
      const int c = tid + 256 * u, t4 = c / PPR * 4, pc = c % PPR;
      if (KALL || t4 < PC) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s_k[piece(t4 + e, pc)] = rk[u][e];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          auto word = [&](int a) {
            const u32x4& x = rk[u][a];
            return e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w;
          };
          const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
          const uint2 w = make_uint2(__builtin_amdgcn_perm(word(1), word(0), sel),
                                     __builtin_amdgcn_perm(word(3), word(2), sel));
          *reinterpret_cast<uint2*>(s_kt + kt_piece(8 * pc + e, t4 >> 3) * 16 + (t4 & 4) * 2) = w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < QU; ++u) {
      const int c = tid + 256 * u;
      s_q[piece(c / PPR, c % PPR)] = rq[u];
    }
#pragma unroll
    for (int u = 0; u < VU; ++u) reinterpret_cast<u32x4*>(s_v)[lane + 64 * u] = rv[u];
#pragma unroll
    for (int u = 0; u < WU; ++u) {
      const int c = tid + 256 * u;
      if (c < CHUNK_WORK_BYTES / 16) s_w[c] = rw[u];
    }
  };

  int arow[2], ak[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) frag_at<CW>(lane, f, &arow[f], &ak[f]);
  // fragment f of block (rb, kb) of a row-major operand
  auto frag_k = [&](const u32x4* s, int rb, int kb, int f) { return as_frag(s[piece(32 * rb + arow[f], (32 * kb + ak[f]) >> 3)]); };
  auto frag_kt = [&](int rb, int kb, int f) {
    return as_frag(reinterpret_cast<const u32x4*>(s_kt)[kt_piece(32 * rb + arow[f], (32 * kb + ak[f]) >> 3)]);
  };
  auto frag_t = [&](int f, int term) { return as_frag(s_w[(f * 3 + term) * 64 + lane]); };
  auto frag_p = [&](int f, int term) { return as_frag(s_w[T_BYTES / 16 + (f * 2 + term) * 64 + lane]); };
  auto block8 = [&](const Acc (&a)[M::TILES], int s, float (&x)[8]) {    // the B operand of step s
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = a[(8 * s + e) / AR][(8 * s + e) % AR];
  };

  int nt = pt.len < PC ? pt.len : PC;
  fetch(0, nt);
  for (int t0 = 0; t0 < pt.len; t0 += PC) {
    stage();
    __syncthreads();
    const int now = nt, left = pt.len - t0 - PC;
    if (left > 0) {
      nt = left < PC ? left : PC;
      fetch(t0 + PC, nt);
    }

    // K S and Q S
    Acc R[2][M::TILES], O[2][M::TILES];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int t = 0; t < M::TILES; ++t)
#pragma unroll
        for (int r = 0; r < AR; ++r) R[rb][t][r] = O[rb][t][r] = 0.f;
#pragma unroll
    for (int kb = 0; kb < DB; ++kb)
#pragma unroll
      for (int s = 0; s < M::STEPS; ++s) {
        float x[8];
        bf16x8 b[3];
        block8(S[kb], s, x);
        split8<3>(x, b);
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < M::TILES; ++t) {
            const int f = M::TILES == 2 ? t : s;
            const bf16x8 fk = frag_k(s_k, rb, kb, f), fq = frag_k(s_q, rb, kb, f);
            R[rb][t] = M::mm(fk, b[0], R[rb][t]);
            O[rb][t] = M::mm(fq, b[0], O[rb][t]);
            R[rb][t] = M::mm(fk, b[1], R[rb][t]);
            O[rb][t] = M::mm(fq, b[1], O[rb][t]);
            R[rb][t] = M::mm(fk, b[2], R[rb][t]);
          }
      }
    // R = V - g (K S);  O = g (Q S)
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int r = 0; r < NB; ++r) {
        const int t = 32 * rb + M::index(lane, r);
        const float gam = s_g[t];
        R[rb][r / AR][r % AR] = to_f32(s_v[t * CW + n]) - gam * R[rb][r / AR][r % AR];
        O[rb][r / AR][r % AR] *= gam;
      }
    // U = T R
    Acc U[2][M::TILES];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int t = 0; t < M::TILES; ++t)
#pragma unroll
        for (int r = 0; r < AR; ++r) U[rb][t][r] = 0.f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int s = 0; s < M::STEPS; ++s) {
        float x[8];
        bf16x8 b[3];
        block8(R[kb], s, x);
        split8<3>(x, b);
#pragma unroll
        for (int rb = kb; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < M::TILES; ++t) {
            const int f = (rb + kb) * 2 + (M::TILES == 2 ? t : s);
            const bf16x8 a0 = frag_t(f, 0), a1 = frag_t(f, 1), a2 = frag_t(f, 2);
            U[rb][t] = M::mm(a0, b[2], U[rb][t]);
            U[rb][t] = M::mm(a2, b[0], U[rb][t]);
            U[rb][t] = M::mm(a1, b[1], U[rb][t]);
            U[rb][t] = M::mm(a0, b[1], U[rb][t]);
            U[rb][t] = M::mm(a1, b[0], U[rb][t]);
            U[rb][t] = M::mm(a0, b[0], U[rb][t]);
          }
      }
    // O += P U;  S = g_C S + K^T (D_C U)
    const float gC = s_g[PC - 1];
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int t = 0; t < M::TILES; ++t)
#pragma unroll
        for (int r = 0; r < AR; ++r) S[db][t][r] *= gC;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int s = 0; s < M::STEPS; ++s) {
        float x[8];
        bf16x8 b2[2], b[3];
        block8(U[kb], s, x);
        split8<2>(x, b2);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= s_g[PC + 32 * kb + M::index(lane, 8 * s + e)];
        split8<3>(x, b);
#pragma unroll
        for (int rb = kb; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < M::TILES; ++t) {
            const int f = (rb + kb) * 2 + (M::TILES == 2 ? t : s);
            const bf16x8 a0 = frag_p(f, 0), a1 = frag_p(f, 1);
            O[rb][t] = M::mm(a0, b2[1], O[rb][t]);
            O[rb][t] = M::mm(a1, b2[0], O[rb][t]);
            O[rb][t] = M::mm(a0, b2[0], O[rb][t]);
          }
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int t = 0; t < M::TILES; ++t) {
            const bf16x8 a = frag_kt(db, kb, M::TILES == 2 ? t : s);
            S[db][t] = M::mm(a, b[2], S[db][t]);
            S[db][t] = M::mm(a, b[1], S[db][t]);
            S[db][t] = M::mm(a, b[0], S[db][t]);
          }
      }
    // the outputs leave through the wave's own part of LDS as whole rows
    wave_lds_sync();
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int r = 0; r < NB; ++r)
        s_v[(32 * rb + M::index(lane, r)) * CW + n] = f32_to_bf16(O[rb][r / AR][r % AR]);
    wave_lds_sync();
#pragma unroll
    for (int u = 0; u < VU; ++u) {
      const int c = lane + 64 * u, t = c / VPR, pc = c % VPR;
      if (t < now) *reinterpret_cast<u32x4*>(op + (t0 + t) * p.os + pc * 8) = reinterpret_cast<const u32x4*>(s_v)[c];
    }
    __syncthreads();                             // every wave has read this chunk's operands
  }

#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < NB; ++r) Sg[(size_t)(32 * db + M::index(lane, r)) * DV] = S[db][r / AR][r % AR];
  if (!p.prime) return;
  const int off = p.sk.off[h], rank = p.sk.off[h + 1] - off;
  if (rank == 0) {                               // a dense-fallback head: the state copy
    int slot = 0;
    while (slot + 1 < p.sk.ndense && p.sk.dense_list[slot] != h) ++slot;
    bf16* C = reinterpret_cast<bf16*>(p.sk.Sc) + ((size_t)pt.b * p.sk.ndense + slot) * DK * DV + col;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < NB; ++r)
        C[(size_t)(32 * db + M::index(lane, r)) * DV] = f32_to_bf16(S[db][r / AR][r % AR]);
    return;
  }
  bf16* Ug = reinterpret_cast<bf16*>(p.sk.U) + ((size_t)pt.b * p.sk.R + off) * DV + col;
  for (int j = 0; j < rank; ++j) {               // u_j = S^T p_j
    const float* P = p.sk.Pt + (size_t)(off + j) * DK + 8 * hi;
    float a = 0.f;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int s = 0; s < M::STEPS; ++s) {
        float x[8], w[8];
        block8(S[db], s, x);
        ldn<8>(P + 32 * db + M::KS * s, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) a += x[e] * w[e];
      }
    if (M::MT == 16) a += __shfl_xor(a, 16);
    a += __shfl_xor(a, 32);
    if (hi == 0) Ug[(size_t)j * DV] = f32_to_bf16(a);
  }
}

template <int DK, int DV, int CW>
int launch(const PromptParams& p, hipStream_t st) {
  using L = ChunkLds<DK, DV, CW>;
  hipLaunchKernelGGL((prompt_prep_kernel<DK, CW>), dim3((unsigned)p.nslots * p.H), dim3(256), 0, st, p);
  hipLaunchKernelGGL((prompt_chunk_kernel<DK, DV, CW>), dim3((unsigned)p.nseq * p.H * (DV / L::VC)), dim3(256), 0,
                     st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_prompt_chunks(int dk, int dv, const PromptParams& p, hipStream_t st) {
  if (dk == 64 && dv == 64) return launch<64, 64, 16>(p, st);
  if (dk == 128 && dv == 64) return launch<128, 64, 16>(p, st);
  if (dk == 128 && dv == 128) return launch<128, 128, 32>(p, st);
  return -2;
}

}  // namespace sk
