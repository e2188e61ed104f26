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
// holds CW columns of the state, all rows, in registers.  K, Q, V, T and P
// are in LDS twice: the next chunk's copy, straight from memory, is in flight
// over the present chunk.  K^T comes from K by transposing reads.
template <int DK, int CW, int BUFS>
struct ChunkLds {
  static constexpr int VC = 4 * CW;              // columns of the workgroup
  static constexpr int K = 0;
  static constexpr int Q = K + PC * DK * 2;
  static constexpr int V = Q + PC * DK * 2;      // wave after wave: [64][CW], then the outputs [CW][64]
  static constexpr int W = V + PC * VC * 2;      // a chunk's workspace as it is
  static constexpr int BUF = W + (CHUNK_WORK_BYTES + 1023) / 1024 * 1024;
  static constexpr int BYTES = BUFS * BUF;
  static_assert(BYTES <= BUFS * 80 * 1024, "two workgroups of one buffer, or one of two, on a CU");
};

// 16 bytes of each active lane from memory to LDS at lds + 16 * lane, in
// flight until the wave's next wait for its memory counter.  (The compiler
// would have every LDS read wait for a copy that it knows of, also where the
// two are in different buffers.)
__device__ __forceinline__ void copy16(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(reinterpret_cast<uint64_t>(g)),
               "s"(lds)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// Within each 16 lanes, lane i gives the address of four values: 4 rows (i / 4)
// of 16 (4 (i % 4) ..); it receives column i of the four rows.
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x4 read_tr(const void* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
      (__attribute__((address_space(3))) bf16x4*)const_cast<void*>(p));
}
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Asks for a step's instructions in the order: a matrix instruction, LDS reads
// (of the next step's fragments), vector work (the next step's split), and so
// on.  One wave's vector work runs in the shadow of its matrix instructions
// only where it stands between them.
template <int MFMAS, int READS, int VALU>
__device__ __forceinline__ void interleave() {
  if constexpr (MFMAS > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    interleave<MFMAS - 1, READS, VALU>();
  }
}

template <int DK, int DV, int CW, int BUFS>
__global__ void __launch_bounds__(256, 3 - BUFS) prompt_chunk_kernel(PromptParams p) {
  using M = Mf<CW>;
  using L = ChunkLds<DK, CW, BUFS>;
  typedef typename M::Acc Acc;
  constexpr int VC = L::VC, PARTS = DV / VC, PPR = DK / 8, NB = M::NB, DB = DK / 32;
  constexpr int AR = NB / M::TILES;              // registers of a tile
  constexpr int PIPE = BUFS - 1;                 // one wave a SIMD: it overlaps its own steps
  __shared__ __align__(1024) unsigned char smem[L::BYTES];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  // (the parts of a tile are a multiple of nseq * H workgroups apart: mostly
  // on the same XCD, whose cache then serves the K, Q, T and P that they share)
  const int tiles = p.nseq * p.H, part = blockIdx.x / tiles, tile = blockIdx.x - part * tiles;
  const int i = tile / p.H, h = tile - i * p.H;
  if ((int64_t)p.start[i + 1] - p.start[i] <= p.len_lo) return;
  const PromptTile pt = prompt_tile(p, i, h);
  if (!pt.ok) return;

  const int n = lane % M::MT, hi = lane / M::MT;           // column, part of the k axis
  const int col = part * VC + wv * CW + n;
  float* Sg = p.S + ((size_t)pt.b * p.H + h) * DK * DV + col;

  const bf16* kp = reinterpret_cast<const bf16*>(p.k) + pt.s0 * p.ks + (int64_t)h * DK;
  const bf16* qp = reinterpret_cast<const bf16*>(p.q) + pt.s0 * p.qs + (int64_t)h * DK;
  const bf16* vp = reinterpret_cast<const bf16*>(p.v) + pt.s0 * p.vs + (int64_t)h * DV + part * VC + wv * CW;
  bf16* op = reinterpret_cast<bf16*>(p.o) + pt.s0 * p.os + (int64_t)h * DV + part * VC + wv * CW;
  const unsigned char* wp = reinterpret_cast<const unsigned char*>(p.work) +
                            ((size_t)first_slot(pt.s0, i) * p.H + h) * CHUNK_WORK_BYTES;

  // rows of K and Q with their 16-byte pieces swizzled
  auto swz = [](int row) { return (PPR == 16 ? M::swizzle(row) : M::swizzle(row) >> 1) & (PPR - 1); };
  auto piece = [&](int row, int pc) { return row * PPR + (pc ^ swz(row)); };
  // A chunk's copies, in units of 64 pieces that the waves share out.  Rows
  // behind the prompt's end repeat its last: their beta in T is 0, their
  // columns of P meet only zeros, and their outputs are not stored.
  const uint32_t lds0 = lds_address(smem);
  constexpr int VPR = CW / 8, KU = PPR / 4, KROWS = 256 / PPR, VROWS = 64 / VPR;
  constexpr int WFULL = CHUNK_WORK_BYTES / 16 / 64, WREST = CHUNK_WORK_BYTES / 16 % 64;
  const int krow = (wv * 64 + lane) / PPR, kpc = lane % PPR, vrow = lane / VPR;
  const unsigned char* wp0 = wp + lane * 16 + wv * 1024;
  auto copies = [&](int t0, int nt, int buf) {
    const uint32_t l0 = lds0 + buf * L::BUF;
    if (nt == PC) {                                        // uniform: a whole chunk
      const bf16* kc = kp + (t0 + krow) * p.ks;
      const bf16* qc = qp + (t0 + krow) * p.qs;
      const bf16* vc = vp + (t0 + vrow) * p.vs + (lane % VPR) * 8;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int pc = (kpc ^ swz(krow + KROWS * u)) * 8;
        copy16(kc + (u * KROWS * p.ks + pc), l0 + L::K + (4 * u + wv) * 1024);
        copy16(qc + (u * KROWS * p.qs + pc), l0 + L::Q + (4 * u + wv) * 1024);
      }
#pragma unroll
      for (int u = 0; u < VPR; ++u)
        copy16(vc + u * VROWS * p.vs, l0 + L::V + wv * PC * CW * 2 + u * 1024);
    } else {
#pragma unroll 1
      for (int u = 0; u < KU; ++u) {
        const int row = krow + KROWS * u, pc = (kpc ^ swz(row)) * 8;
        const int64_t t = t0 + (row < nt ? row : nt - 1);
        copy16(kp + t * p.ks + pc, l0 + L::K + (4 * u + wv) * 1024);
        copy16(qp + t * p.qs + pc, l0 + L::Q + (4 * u + wv) * 1024);
      }
#pragma unroll 1
      for (int u = 0; u < VPR; ++u) {
        const int row = vrow + VROWS * u;
        const int64_t t = t0 + (row < nt ? row : nt - 1);
        copy16(vp + t * p.vs + (lane % VPR) * 8, l0 + L::V + wv * PC * CW * 2 + u * 1024);
      }
    }
    const unsigned char* w = wp0 + (size_t)(t0 / PC) * p.H * CHUNK_WORK_BYTES;
#pragma unroll
    for (int u = 0; u < WFULL / 4; ++u) copy16(w + u * 4096, l0 + L::W + (4 * u + wv) * 1024);
    constexpr int U = WFULL / 4 * 4;
    if (U + wv < WFULL || (U + wv == WFULL && lane < WREST)) copy16(w + U * 1024, l0 + L::W + (U + wv) * 1024);
  };
  int nt = pt.len < PC ? pt.len : PC;
  if (pt.len > 0) copies(0, nt, 0);

  // the state, block after block of 32 rows
  Acc S[DB][M::TILES];
  const bool cont = !p.has_state || p.has_state[i] != 0;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < NB; ++r)
      S[db][r / AR][r % AR] = cont ? Sg[(size_t)(32 * db + M::index(lane, r)) * DV] : 0.f;

  int arow[2], ak[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) frag_at<CW>(lane, f, &arow[f], &ak[f]);
  const unsigned char* sb = smem;                // the present chunk's buffer
  // fragment f of block (rb, kb) of K or Q
  auto frag_k = [&](int at, int rb, int kb, int f) {
    return as_frag(reinterpret_cast<const u32x4*>(sb + at)[piece(32 * rb + arow[f], (32 * kb + ak[f]) >> 3)]);
  };
  // of K^T: eight tokens from 32 kb + ak of the rows that the lane's group of 16
  // gives the addresses of: lane i those of tokens i / 4 and i / 4 + 4
  const int ti = (lane & 15) >> 2, tc = 4 * (lane & 3), tg = M::MT == 32 ? lane & 16 : 0;
  auto frag_kt = [&](int rb, int kb, int f) {
    const int d = 32 * rb + M::row(tg + tc, M::TILES == 2 ? f : 0), t = 32 * kb + ak[f] + ti;
    const unsigned char* s = sb + L::K + (d & 7) * 2;
    return join(read_tr(s + piece(t, d >> 3) * 16), read_tr(s + piece(t + 4, d >> 3) * 16));
  };
  auto frag_t = [&](int f, int term) { return as_frag(reinterpret_cast<const u32x4*>(sb + L::W)[(f * 3 + term) * 64 + lane]); };
  auto frag_p = [&](int f, int term) {
    return as_frag(reinterpret_cast<const u32x4*>(sb + L::W + T_BYTES)[(f * 2 + term) * 64 + lane]);
  };
  auto block8 = [&](const Acc (&a)[M::TILES], int s, float (&x)[8]) {    // the B operand of step s
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = a[(8 * s + e) / AR][(8 * s + e) % AR];
  };
  // the wave's outputs of a chunk, as whole rows: lane's 8 columns of OU tokens
  constexpr int OU = NB / 8 * 2, OG = CW / 8;    // OG column groups, 4 / OG groups of 16 tokens at a time
  u32x4 out[OU];
  const int og = (lane >> 4) % OG, ot = (lane >> 4) / OG * 16 + (lane & 15);
  bf16* op0 = op + ot * p.os + og * 8;
  auto store_out = [&](int t0, int cnt) {
#pragma unroll
    for (int u = 0; u < OU; ++u) {
      if (ot + u * (64 / OG) < cnt)
        *reinterpret_cast<u32x4*>(op0 + (int64_t)t0 * p.os + u * (64 / OG) * p.os) = out[u];
    }
  };

  int t0 = 0;
  for (int buf = 0; t0 < pt.len; t0 += PC, buf ^= PIPE) {
    // this wave's copies for the chunk have landed, then everybody's; with two
    // buffers, everybody has read the other
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    sb = smem + buf * L::BUF;
    if (t0 > 0) store_out(t0 - PC, PC);
    const int left = pt.len - t0 - PC;
    nt = left < PC ? left : PC;
    if (PIPE && left > 0) copies(t0 + PC, nt, buf ^ 1);
    const float* s_g = reinterpret_cast<const float*>(sb + L::W + T_BYTES + P_BYTES);
    unsigned char* s_v = smem + buf * L::BUF + L::V + wv * PC * CW * 2;

    // Each step of a product (KS values of its k axis) has its A fragments read
    // from LDS and its B operand split during the step before, so that neither
    // LDS latency nor vector work stands between two steps' matrix
    // instructions; the barriers keep the compiler from undoing that.
    constexpr int NF = M::TILES, J1 = DB * M::STEPS, J2 = 2 * M::STEPS;
    Acc R[2][NF], O[2][NF], U[2][NF];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int t = 0; t < NF; ++t)
#pragma unroll
        for (int r = 0; r < AR; ++r) R[rb][t][r] = O[rb][t][r] = U[rb][t][r] = 0.f;
    bf16x8 ft[BUFS][2][NF][3];                              // T fragments: [step parity][rb][tile][value]
    bf16x8 b[BUFS][3];
    auto load_t = [&](int j) {
      const int kb = j / M::STEPS, sp = j % M::STEPS;
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int t = 0; t < NF; ++t)
          if (rb >= kb) {
#pragma unroll
            for (int v = 0; v < 3; ++v) ft[j & PIPE][rb][t][v] = frag_t((rb + kb) * 2 + (NF == 2 ? t : sp), v);
          }
    };
    {  // K S and Q S
      bf16x8 fk[BUFS][2][NF], fq[BUFS][2][NF];
      auto load_kq = [&](int j) {
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < NF; ++t) {
            fk[j & PIPE][rb][t] = frag_k(L::K, rb, j / M::STEPS, NF == 2 ? t : j % M::STEPS);
            fq[j & PIPE][rb][t] = frag_k(L::Q, rb, j / M::STEPS, NF == 2 ? t : j % M::STEPS);
          }
      };
      auto split_s = [&](int j) {
        float x[8];
        block8(S[j / M::STEPS], j % M::STEPS, x);
        split8<3>(x, b[j & PIPE]);
      };
      if (PIPE) {
        load_kq(0);
        split_s(0);
      }
#pragma unroll
      for (int j = 0; j < J1; ++j) {
        if (j + PIPE < J1) {
          load_kq(j + PIPE);
          split_s(j + PIPE);
        } else {
          load_t(0);
        }
#pragma unroll
        for (int v = 0; v < 3; ++v)
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int t = 0; t < NF; ++t) {
              R[rb][t] = M::mm(fk[j & PIPE][rb][t], b[j & PIPE][v], R[rb][t]);
              if (v < 2) O[rb][t] = M::mm(fq[j & PIPE][rb][t], b[j & PIPE][v], O[rb][t]);
            }
        if constexpr (PIPE) {
          interleave<10 * NF, 1, (NF == 1 ? 6 : 3)>();
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    // R = V - g (K S);  O = g (Q S)
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int s8 = 0; s8 < NB / 8; ++s8) {
        // V's column n, eight tokens: as K^T, from rows of CW values
        const int tk = 32 * rb + M::index(lane, 8 * s8);
        const unsigned char* sv = s_v + ((tk + ti) * CW + tg + tc) * 2;
        const bf16x8 v8 = join(read_tr(sv), read_tr(sv + 4 * CW * 2));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = 8 * s8 + e;
          const float gam = s_g[tk + e];
          R[rb][r / AR][r % AR] = (float)v8[e] - gam * R[rb][r / AR][r % AR];
          O[rb][r / AR][r % AR] *= gam;
        }
      }
    const float gC = s_g[PC - 1];
    bf16x8 fp[BUFS][2][NF][2], fs[BUFS][DB][NF];
    auto load_ps = [&](int j) {
      const int kb = j / M::STEPS, sp = j % M::STEPS;
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int t = 0; t < NF; ++t)
          if (rb >= kb) {
#pragma unroll
            for (int v = 0; v < 2; ++v) fp[j & PIPE][rb][t][v] = frag_p((rb + kb) * 2 + (NF == 2 ? t : sp), v);
          }
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int t = 0; t < NF; ++t) fs[j & PIPE][db][t] = frag_kt(db, kb, NF == 2 ? t : sp);
    };
    {  // U = T R;  S = g_C S meanwhile
      auto split_r = [&](int j) {
        float x[8];
        block8(R[j / M::STEPS], j % M::STEPS, x);
        split8<3>(x, b[j & PIPE]);
      };
      if (PIPE) split_r(0);
#pragma unroll
      for (int j = 0; j < J2; ++j) {
        if (j + PIPE < J2) {
          load_t(j + PIPE);
          split_r(j + PIPE);
        } else {
          load_ps(0);
        }
        const int kb = j / M::STEPS;
        constexpr int TA[6] = {0, 2, 1, 0, 1, 0}, TB[6] = {2, 0, 1, 1, 0, 0};   // the smaller products first
#pragma unroll
        for (int v = 0; v < 6; ++v)
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int t = 0; t < NF; ++t)
              if (rb >= kb) U[rb][t] = M::mm(ft[j & PIPE][rb][t][TA[v]], b[j & PIPE][TB[v]], U[rb][t]);
#pragma unroll
        for (int db = j * DB / J2; db < (j + 1) * DB / J2; ++db)
#pragma unroll
          for (int t = 0; t < NF; ++t)
#pragma unroll
            for (int r = 0; r < AR; ++r) S[db][t][r] *= gC;
        if constexpr (PIPE) {
          if (kb == 0) interleave<12 * NF, 1, (NF == 1 ? 6 : 4)>();
          else interleave<6 * NF, 2, (NF == 1 ? 9 : 6)>();
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    {  // O += P U;  S += K^T (D_C U)
      bf16x8 c[BUFS][2];
      auto split_u = [&](int j) {
        float x[8];
        block8(U[j / M::STEPS], j % M::STEPS, x);
        split8<2>(x, c[j & PIPE]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= s_g[PC + 32 * (j / M::STEPS) + M::index(lane, 8 * (j % M::STEPS) + e)];
        split8<3>(x, b[j & PIPE]);
      };
      if (PIPE) split_u(0);
#pragma unroll
      for (int j = 0; j < J2; ++j) {
        if (j + PIPE < J2) {
          load_ps(j + PIPE);
          split_u(j + PIPE);
        }
        const int kb = j / M::STEPS;
        constexpr int PA[3] = {0, 1, 0}, PB[3] = {1, 0, 0};
#pragma unroll
        for (int v = 0; v < 3; ++v) {
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int t = 0; t < NF; ++t)
              if (rb >= kb) O[rb][t] = M::mm(fp[j & PIPE][rb][t][PA[v]], c[j & PIPE][PB[v]], O[rb][t]);
        }
#pragma unroll
        for (int v = 2; v >= 0; --v)
#pragma unroll
          for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int t = 0; t < NF; ++t) S[db][t] = M::mm(fs[j & PIPE][db][t], b[j & PIPE][v], S[db][t]);
        if constexpr (PIPE) if (j + 1 < J2) {
          interleave<(3 * DB + 3) * NF, 1, (NF == 1 ? 6 : 4)>();
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    // the outputs, columns of 64 tokens (eight swizzled pieces), over the wave's
    // part of V, and back as rows of eight columns by transposing reads
    wave_lds_sync();
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int s8 = 0; s8 < NB / 8; ++s8) {
        bf16x8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = (__bf16)O[rb][(8 * s8 + e) / AR][(8 * s8 + e) % AR];
        const int pc = (32 * rb + M::index(lane, 8 * s8)) >> 3;
        *reinterpret_cast<bf16x8*>(s_v + n * 128 + (pc ^ (n & 7)) * 16) = w;
      }
    wave_lds_sync();
#pragma unroll
    for (int u = 0; u < OU; ++u) {
      // lane i of a group: column 8 og + i / 4 (and + 4), tokens 4 (i % 4) ..
      const int t = (lane >> 4) / OG * 16 + u * (64 / OG) + tc, c = 8 * og + ti;
      auto at = [&](int cc) { return s_v + cc * 128 + ((t >> 3) ^ (cc & 7)) * 16 + (t & 7) * 2; };
      out[u] = __builtin_bit_cast(u32x4, join(read_tr(at(c)), read_tr(at(c + 4))));
    }
    wave_lds_sync();
    if (!PIPE && left > 0) {                     // one buffer: everybody has read it
      __syncthreads();
      copies(t0 + PC, nt, 0);
    }
  }
  if (pt.len > 0) store_out(t0 - PC, pt.len - (t0 - PC));

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

template <int DK, int DV, int CW, int BUFS>
int launch(const PromptParams& p, hipStream_t st) {
  hipLaunchKernelGGL((prompt_prep_kernel<DK, CW>), dim3((unsigned)p.nslots * p.H), dim3(256), 0, st, p);
  hipLaunchKernelGGL((prompt_chunk_kernel<DK, DV, CW, BUFS>), dim3((unsigned)p.nseq * p.H * (DV / (4 * CW))), dim3(256),
                     0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_prompt_chunks(int dk, int dv, const PromptParams& p, hipStream_t st) {
  const bool few = p.nseq * p.H <= 256;
  if (dk == 64 && dv == 64) return few ? launch<64, 64, 16, 2>(p, st) : launch<64, 64, 16, 1>(p, st);
  if (dk == 128 && dv == 64) return few ? launch<128, 64, 16, 2>(p, st) : launch<128, 64, 16, 1>(p, st);
  if (dk == 128 && dv == 128) return few ? launch<128, 128, 16, 2>(p, st) : launch<128, 128, 32, 1>(p, st);
  return -2;
}

}  // namespace sk
