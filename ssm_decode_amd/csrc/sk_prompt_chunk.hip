// The launches of the chunked form: T and P of every chunk, then, for bf16
// activations, the chunks in order (sk_prompt_chunk.hpp has the mathematics).
#include <type_traits>

#include "sk_prompt_chunk.hpp"

namespace sk {
namespace {

// ------------------------------------------------------------ T and P
// One workgroup of four waves per (chunk slot, head).  K K^T and Q K^T on the
// matrix cores (bf16: exact products, fp32 sums; fp32: fp32 instructions); the unit
// triangular inverse by substitution in 16 x 16 blocks, joined to 32 and 64 by
// fp32 products.  Alone a workgroup takes about 8 us, a chain of loads, products,
// inverse and joins, so what counts is how many a CU has at once: K and Q come in
// stages, and A and P, which waits in registers, take the same place in LDS (8224 of
// 128 columns, 268 MB of K and Q in, 256 MB of T and P out: three a CU 164 us, four,
// with A and P apart, 115, six 94, 5.6 TB/s; six with 88 bytes of spills 159).
constexpr int LS = PC + 4;                       // row stride of the fp32 matrices in LDS

template <int DK, typename AT>
__global__ void __launch_bounds__(256, sizeof(AT) == 4 ? 4 : 6) prompt_prep_kernel(PromptParams p) {
  constexpr bool F32 = sizeof(AT) == 4;
  // K and Q come in stages of 128 bytes of a row (8 pieces), two ahead in registers
  constexpr int PPR = 8, EPP = 16 / (int)sizeof(AT), STAGES = DK / (PPR * EPP), U = PC * PPR / 256;
  constexpr int KB = PC * PPR * 16;              // bytes of a stage of K or Q in LDS
  constexpr int MB = PC * LS * 4;                // bytes of A (T in its place), then P, over them
  __shared__ __align__(16) unsigned char s_big[2 * KB > MB ? 2 * KB : MB];
  __shared__ __align__(16) float s_al[PC], s_be[PC], s_pre[PC], s_suf[PC], s_blk[4], s_mid[16], s_din[PC * 17];
  __shared__ int s_lim;
  float* s_A = reinterpret_cast<float*>(s_big);

  // (the last chunks first: what the next launch begins with is then the most
  // recent in the memory-side cache)
  const int rslot = blockIdx.x / p.H, h = blockIdx.x - rslot * p.H, slot = p.nslots - 1 - rslot;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  // (a refused list may have no prompt that any other launch comes to: it is
  // reported here)
  if (rslot == 0) prompt_ok(p, 0, h, p.seqs ? p.seqs[0] : 0);
  int rank;
  const int i = slot_prompt(p, slot, 6, &rank);
  if (i < 0) return;
  const int s0 = p.start[i], s1 = p.start[i + 1];
  if (s0 < 0 || s1 < s0 || s1 > p.tokens) return;
  const int c0 = (slot - first_slot(s0, rank, 6)) * PC, len = s1 - s0;
  if (c0 >= len) return;
  const int nt = len - c0 < PC ? len - c0 : PC;
  const int64_t tok = (int64_t)s0 + c0;

  // pieces swizzled, zeros behind nt
  auto piece = [](int row, int pc) { return row * PPR + (pc ^ ((row >> 1) & (PPR - 1))); };
  u32x4* s_k = reinterpret_cast<u32x4*>(s_big);
  u32x4* s_q = reinterpret_cast<u32x4*>(s_big + KB);
  const AT* kp = reinterpret_cast<const AT*>(p.k) + tok * p.ks + (int64_t)h * DK;
  const AT* qp = reinterpret_cast<const AT*>(p.q) + tok * p.qs + (int64_t)h * DK;
  u32x4 rk[2][U], rq[2][U];
  auto fetch = [&](int st) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tid + 256 * u, row = c / PPR, col = (st * PPR + c % PPR) * EPP;
      rk[st & 1][u] = rq[st & 1][u] = u32x4{0, 0, 0, 0};
      if (row < nt) {
        rk[st & 1][u] = *reinterpret_cast<const u32x4*>(kp + row * p.ks + col);
        rq[st & 1][u] = *reinterpret_cast<const u32x4*>(qp + row * p.qs + col);
      }
    }
  };
  auto stage = [&](int st) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = tid + 256 * u;
      s_k[piece(c / PPR, c % PPR)] = rk[st & 1][u];
      s_q[piece(c / PPR, c % PPR)] = rq[st & 1][u];
    }
  };
  fetch(0);
  if (STAGES > 1) fetch(1);
  // s_lim: the first token with an infinity or a NaN in its key or factors (PC:
  // none).  From it on T and the keys' factors are those of no tokens, and g is
  // NaN, which takes the next launch's outputs from there on, and the state, with
  // it; tokens before see nothing of it.
  if (wv == 0) {
    const float al = tid < nt ? p.gate[(tok + tid) * p.gs + h] : 1.f, be = tid < nt ? p.beta[(tok + tid) * p.bs + h] : 0.f;
    s_al[tid] = al;
    s_be[tid] = be;
    const unsigned long long m = __ballot(!finite(al) || !finite(be));
    if (tid == 0) s_lim = m ? __builtin_ctzll(m) : PC;
  }
  stage(0);
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
    wave_lds_sync();
    if (lane < 16) {                                    // over the blocks between two
      float mid = 1.f;
#pragma unroll
      for (int t = 1; t < 3; ++t)
        if (t > (lane & 3) && t < (lane >> 2)) mid *= s_blk[t];
      s_mid[lane] = mid;
    }
  }
  __syncthreads();

  // tiles (ti, tj), tj <= ti, of K K^T and Q K^T: the t-th, t = wave + 4 n (the
  // last ones repeat tile 9 and are dropped: no branch between the products)
  f32x4s ak[3], aq[3];
  const int cg = lane & 15, g = lane >> 4;
  auto tile_of = [](int t, int* ti, int* tj) {
    *ti = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    *tj = t - *ti * (*ti + 1) / 2;
  };
  int ti[3], tj[3];
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    tile_of(wv + 4 * n < 10 ? wv + 4 * n : 9, &ti[n], &tj[n]);
    ak[n] = aq[n] = f32x4s{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int st = 0; st < STAGES; ++st) {
    if (st > 0) {
      __syncthreads();
      stage(st);
      __syncthreads();
    }
    if (st + 2 < STAGES) fetch(st + 2);
#pragma unroll
    for (int s = 0; s < PPR / 4; ++s) {
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        const u32x4 fk = s_k[piece(16 * ti[n] + cg, 4 * s + g)], fq = s_q[piece(16 * ti[n] + cg, 4 * s + g)];
        const u32x4 fb = s_k[piece(16 * tj[n] + cg, 4 * s + g)];
        if constexpr (F32) {                            // K-step e: columns 16 s + 4 k + e
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float b = __uint_as_float(fb[e]);
            ak[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fk[e]), b, ak[n], 0, 0, 0);
            aq[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fq[e]), b, aq[n], 0, 0, 0);
          }
        } else {
          ak[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(fk), as_frag(fb), ak[n], 0, 0, 0);
          aq[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_frag(fq), as_frag(fb), aq[n], 0, 0, 0);
        }
      }
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  // (a key with one has no finite product with itself; one whose square
  // overflows counts as such)
#pragma unroll
  for (int n = 0; n < 3; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (ti[n] == tj[n] && 4 * g + r == cg && !finite(ak[n][r])) atomicMin(&s_lim, 16 * ti[n] + cg);
  float D[3][4], be[3][4];                              // D_ij and beta_i of the lane's results
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    const float across = s_mid[4 * ti[n] + tj[n]] * s_suf[16 * tj[n] + cg];
    float pre[4];
    ld4(s_pre + 16 * ti[n] + 4 * g, pre);
    ld4(s_be + 16 * ti[n] + 4 * g, be[n]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float in = s_din[(16 * ti[n] + 4 * g + r) * 17 + cg];
      D[n][r] = ti[n] == tj[n] ? in : pre[r] * across;
    }
  }
  __syncthreads();                                      // K and Q are read: A over them
  const int lim = s_lim;
  if (tid >= lim && tid < PC) s_be[tid] = 0.f;
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    if (wv + 4 * n < 10) {                              // uniform over the wave
      const int j = 16 * tj[n] + cg;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int ii = 16 * ti[n] + 4 * g + r;
        // (selected, not multiplied by a zero: nothing above the diagonal may
        // reach the sums)
        s_A[ii * LS + j] = j < ii && ii < lim ? be[n][r] * D[n][r] * ak[n][r] : 0.f;
        aq[n][r] = j <= ii ? D[n][r] * aq[n][r] : 0.f;
      }
    }
  }
  // the 16 x 16 blocks above the diagonal that fragments cover: (0, 1), (2, 3)
  for (int c = tid; c < 2 * 256; c += 256) {
    const int b = c >> 8, r = (c >> 4) & 15, cc = c & 15;
    s_A[(32 * b + r) * LS + 32 * b + 16 + cc] = 0.f;
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
  constexpr int WORK = F32 ? CHUNK_WORK_F32 : CHUNK_WORK_BYTES;
  unsigned char* W = reinterpret_cast<unsigned char*>(p.work) + ((size_t)slot * p.H + h) * WORK;
  auto tiles = [&](unsigned char* to, bool beta) {      // fp32: four columns a lane
    for (int c = tid; c < F32_TILES * 64; c += 256) {
      const int ln = c & 63;
      int rb, kb;
      tile_of(c >> 6, &rb, &kb);
      const int row = 16 * rb + (ln & 15), k = 16 * kb + 4 * (ln >> 4);
      float t[4];
      ld4(s_A + row * LS + k, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] *= beta ? s_be[k + e] : 1.f;
      stn<4>(reinterpret_cast<float*>(to + c * 16), t);
    }
  };
  auto frags = [&](unsigned char* to, bool is_t) {      // bf16: eight columns a lane, of T split
    for (int c = tid; c < FRAGS * 64; c += 256) {
      const int f = c >> 6, ln = c & 63, pair = f >> 1;
      const int rb = pair > 0, kb = pair == 2;
      const int row = 32 * rb + block_row(ln & 15, f & 1), k = 32 * kb + 8 * (ln >> 4);
      float t[8];
      ldn<8>(s_A + row * LS + k, t);
      if (is_t) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= s_be[k + e];
        bf16x8 v[3];
        split8<true>(t, v);
#pragma unroll
        for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8*>(to + (f * 3 + n) * FRAG_BYTES + ln * 16) = v[n];
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
          *reinterpret_cast<f32x4s*>(to + (f * 2 + n) * FRAG_BYTES + ln * 16) =
              f32x4s{t[4 * n], t[4 * n + 1], t[4 * n + 2], t[4 * n + 3]};
      }
    }
  };
  if constexpr (F32) tiles(W, true);
  else frags(W, true);
  __syncthreads();                                      // T is read: P over it (what is above stays 0)
#pragma unroll
  for (int n = 0; n < 3; ++n)
    if (wv + 4 * n < 10) {
#pragma unroll
      for (int r = 0; r < 4; ++r) s_A[(16 * ti[n] + 4 * g + r) * LS + 16 * tj[n] + cg] = aq[n][r];
    }
  __syncthreads();
  if constexpr (F32) tiles(W + F32_TILES * FRAG_BYTES, false);
  else frags(W + T_BYTES, false);
  if (tid < PC) {
    const int b = tid >> 4;
    float pre = s_pre[tid], suf = s_suf[tid];
    for (int n = 0; n < b; ++n) pre *= s_blk[n];
    for (int n = b + 1; n < 4; ++n) suf *= s_blk[n];
    float* G = reinterpret_cast<float*>(W + WORK - 2 * PC * 4);
    G[tid] = tid < lim ? pre : __builtin_nanf("");
    G[PC + tid] = suf;
  }
}

// ------------------------------------------------------ chunk after chunk
// One workgroup of NW waves per (prompt, head, 16 NW columns); a wave holds 16
// columns of the state, all rows, in registers.  K, Q, V, T and P are in LDS
// twice: the next chunk's copy, straight from memory, is in flight over the
// present chunk.  K^T and V's columns come by transposing LDS reads.
//
// What bounds it is the chain from chunk to chunk (128 x 128: 3.7 us a chunk with
// one wave a SIMD, of which its matrix instructions are 1.8, and 7.8 with two), so
// a chunk's instructions are laid out by hand in regions: in each, the matrix instructions of one
// step, the LDS reads of the next step's fragments, and the vector work (three
// value splits above all) that a later step needs; the vector work runs in the
// shadow of the matrix instructions only where it stands between them.
template <int DK, int NW>
struct ChunkLds {
  static constexpr int K = 0;
  static constexpr int Q = K + PC * DK * 2;
  static constexpr int V = Q + PC * DK * 2;      // wave after wave: [64][16], then the outputs [16][64]
  static constexpr int W = V + PC * NW * 32;     // a chunk's workspace as it is
  static constexpr int BUF = W + CHUNK_WORK_BYTES + PROMPT_WORK_OVER;
  static constexpr int BYTES = 2 * BUF;
  static_assert(BYTES <= 160 * 1024, "LDS of a CU");
};

// Four runs of 1 KiB, one behind the other in memory and in LDS (the
// instruction's offset counts for both addresses).
__device__ __forceinline__ void copy16x4(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %2\n\ts_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %1\n\t"
      "global_load_lds_dwordx4 %0, %1 offset:0x400\n\t"
      "global_load_lds_dwordx4 %0, %1 offset:0x800\n\t"
      "global_load_lds_dwordx4 %0, %1 offset:0xc00" ::"v"(offset),
      "s"(reinterpret_cast<uint64_t>(base)), "s"(lds)
      : "memory", "m0");
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

// Where few tiles have many tokens (p.seg_shift != 0), prompts are cut into
// segments of 2^seg_shift tokens, and three launches take the place of one:
//   1. STATE: the segments but the last, at once, without outputs: each from a
//      zero state (the first from the prompt's), which gives B, and, as further
//      columns, from the identity with no values, which gives the segment's
//      transition M: the state behind a segment is M S + B;
//   2. prompt_join_kernel: the states between the segments, in order;
//   3. the segments at once, each from the state before it, with outputs.
template <int DK, int DV, int NW, bool OUT>
__global__ void __launch_bounds__(64 * NW, 2) prompt_chunk_kernel(PromptParams p) {
  using L = ChunkLds<DK, NW>;
  constexpr int PPR = DK / 8, DB = DK / 32;      // 16-byte pieces of a row, blocks of 32 rows
  // (dynamic: a workgroup of four waves, alone on its CU by its LDS, would
  // otherwise be given more than 256 registers a lane, half of them accumulation
  // registers that vector instructions reach by moves only)
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, hi = lane >> 4;
  // The parts of a tile are eight workgroups apart: on one XCD at one time, so
  // that its cache serves the K, Q, T and P that they share.
  constexpr int VPARTS = DV / (16 * NW), PARTS = VPARTS + (OUT ? 0 : DK / (16 * NW));
  const int tiles = (p.seg_shift ? p.nsegs : p.nchunked) * p.H;
  const int part = blockIdx.x / 8 % PARTS, tile = blockIdx.x / (8 * PARTS) * 8 + blockIdx.x % 8;
  if (tile >= tiles) return;
  const int h = tile % p.H;
  int rank = 0, seg = 0;
  const int i = p.seg_shift ? slot_prompt(p, tile / p.H, p.seg_shift, &rank) : chunked_prompt(p, tile / p.H, &rank);
  if (i < 0) return;
  int s0 = p.start[i], len = p.start[i + 1] - s0;
  const int b = p.seqs ? p.seqs[i] : i;
  bool last = true;                              // the prompt's last segment
  static_assert(DV <= DK, "a state fits the place of a transition");
  const bool unit = !OUT && part >= VPARTS;      // columns of the identity
  const int slot0 = first_slot(s0, rank, 6);
  float* own = nullptr;                          // this segment's B (then the state behind it) and M
  constexpr int SEG_FLOATS = DK * (DV + DK);
  if (p.seg_shift) {
    seg = tile / p.H - first_slot(s0, rank, p.seg_shift);
    const int64_t from = (int64_t)seg << p.seg_shift;
    if (from >= len && seg > 0) return;
    last = len - from <= (1 << p.seg_shift);
    if (!OUT && (last || (unit && seg == 0))) return;
    own = p.seg + ((size_t)(tile / p.H) * p.H + h) * SEG_FLOATS;
    s0 += (int)from;
    len = last ? len - (int)from : 1 << p.seg_shift;
  }
  if (!prompt_ok(p, i, h, b)) return;

  const int c0 = (unit ? part - VPARTS : part) * NW * 16 + wv * 16;       // the wave's first column
  float* Sg = p.S + ((size_t)b * p.H + h) * DK * DV + c0 + n;
  const bf16* kp = reinterpret_cast<const bf16*>(p.k) + s0 * p.ks + (int64_t)h * DK;      // (all uniform)
  const bf16* qp = reinterpret_cast<const bf16*>(p.q) + s0 * p.qs + (int64_t)h * DK;
  const bf16* vp = reinterpret_cast<const bf16*>(p.v) + s0 * p.vs + (int64_t)h * DV + (unit ? 0 : c0);
  const unsigned char* wp = reinterpret_cast<const unsigned char*>(p.work) +
                            ((size_t)(slot0 + (seg << (p.seg_shift ? p.seg_shift - 6 : 0))) * p.H + h) * CHUNK_WORK_BYTES;

  // ------------------------------------------------------------- copies
  // Rows of K and Q have their 16-byte pieces swizzled so that the rows of a
  // fragment spread over the banks.
  auto swz = [](int row) {
    const int s = (row & 3) | ((row >> 1) & 12);
    return (PPR == 16 ? s : s >> 1) & (PPR - 1);
  };
  auto piece = [&](int row, int pc) { return row * PPR + (pc ^ swz(row)); };
  const uint32_t lds0 = lds_address(smem);
  constexpr int KU = PPR / NW, KROWS = 64 * NW / PPR;      // a wave's units of 64 pieces of K, rows from one to the next
  // The workspace in runs of 1 KiB, RUNS to a wave; the last reaches into what
  // lies behind it, and the last wave begins one run early (there is one less
  // than the waves take).
  constexpr int WRUNS = (CHUNK_WORK_BYTES + PROMPT_WORK_OVER) / 1024, RUNS = (WRUNS + 1) / NW;
  static_assert((CHUNK_WORK_BYTES + PROMPT_WORK_OVER) % 1024 == 0 && (WRUNS + 1) % NW == 0 && RUNS % 4 == 0, "runs");
  constexpr int WU = RUNS / 4, UNITS = 2 * KU + WU + 2;
  // (without outputs P is not needed: of eight waves two have nothing but P and
  // take the last's runs once more)
  const bool tail = wv == NW - 1 || (!OUT && wv * RUNS * 1024 >= T_BYTES);
  const int run0 = (tail ? WRUNS - RUNS : wv * RUNS) * 1024;
  const int krow = (wv * 64 + lane) / PPR, kpc = lane % PPR, vrow = lane >> 1;
  // Byte offset of a lane's piece from a chunk's first row (unsigned 32 bits: 63
  // rows of at most 2^25 elements fit).  Rows behind the prompt's end repeat its
  // last one (`last` is its number in the chunk): their beta in T is 0, their
  // columns of P meet only zeros, and their outputs are not stored.
  auto koff = [&](int v, int64_t st, int last) {
    const int row = krow + KROWS * v;
    return (uint32_t)((row < last ? row : last) * st * 2) + (uint32_t)(kpc ^ swz(row)) * 16;
  };
  auto voff = [&](int v, int last) {
    const int row = vrow + 32 * v;
    return (uint32_t)((row < last ? row : last) * p.vs * 2) + (uint32_t)(lane & 1) * 16;
  };
  // In a whole chunk, the offsets of a wave's first unit from its own first row
  // (of K and Q also with the swizzle of its odd units: it has a period of 32
  // rows); the units' rows are added to the uniform base.
  const uint32_t krow2 = (uint32_t)(krow * p.ks * 2), qrow2 = (uint32_t)(krow * p.qs * 2);
  const uint32_t sw[2] = {(uint32_t)(kpc ^ swz(krow)) * 16, (uint32_t)(kpc ^ swz(krow + KROWS)) * 16};
  const uint32_t vo = voff(0, PC), wo = lane * 16;
  // unit u of a whole chunk into a buffer: K, Q, then the workspace, V last.
  // The uniform addresses go from chunk to chunk.
  const bf16 *kc = kp, *qc = qp, *vc = vp;
  const unsigned char* wc = wp + run0;
  auto copy_unit = [&](int u, uint32_t l0) {
    if (u < KU) {
      copy16(kc + u * KROWS * p.ks, krow2 + sw[u & 1], l0 + L::K + (NW * u + wv) * 1024);
    } else if (u < 2 * KU) {
      const int v = u - KU;
      if (OUT) copy16(qc + v * KROWS * p.qs, qrow2 + sw[v & 1], l0 + L::Q + (NW * v + wv) * 1024);
    } else if (u < 2 * KU + WU) {
      const int v = u - 2 * KU;
      copy16x4(wc + v * 4096, wo, l0 + L::W + run0 + v * 4096);
    } else {
      const int v = u - 2 * KU - WU;
      copy16(vc + 32 * v * p.vs, vo, l0 + L::V + wv * 2048 + v * 1024);
    }
  };
  auto next_chunk = [&]() {
    kc += PC * p.ks;
    qc += PC * p.qs;
    vc += PC * p.vs;
    wc += (size_t)p.H * CHUNK_WORK_BYTES;
  };
  // the whole of a chunk that may be a prompt's last
  auto copy_last = [&](int nt, uint32_t l0) {
#pragma unroll 1
    for (int v = 0; v < KU; ++v) {
      copy16(kc, koff(v, p.ks, nt - 1), l0 + L::K + (NW * v + wv) * 1024);
      if (OUT) copy16(qc, koff(v, p.qs, nt - 1), l0 + L::Q + (NW * v + wv) * 1024);
    }
#pragma unroll 1
    for (int v = 0; v < 2; ++v) copy16(vc, voff(v, nt - 1), l0 + L::V + wv * 2048 + v * 1024);
#pragma unroll
    for (int u = 2 * KU; u < 2 * KU + WU; ++u) copy_unit(u, l0);
  };
  if (len > 0) copy_last(len < PC ? len : PC, lds0);

  // --------------------------------------------------------- fragments
  const unsigned char* sb = smem;                // the present chunk's buffer
  const int ti = n >> 2, tc = 4 * (n & 3);
  auto frag_kq = [&](int at, int rb, int t, int kb) {      // tile t of block (rb, kb) of K or Q
    return as_frag(reinterpret_cast<const u32x4*>(sb + at)[piece(32 * rb + block_row(n, t), 4 * kb + hi)]);
  };
  auto frag_kt = [&](int db, int t, int kb) {              // of K^T: tokens 32 kb + 8 hi ..
    const int d = 32 * db + block_row(tc, t), tok = 32 * kb + 8 * hi + ti;
    const unsigned char* s = sb + L::K + (d & 7) * 2;
    return join(read_tr(s + piece(tok, d >> 3) * 16), read_tr(s + piece(tok + 4, d >> 3) * 16));
  };
  auto frag_t = [&](int f, int v) { return as_frag(reinterpret_cast<const u32x4*>(sb + L::W)[(f * 3 + v) * 64 + lane]); };
  auto frag_p = [&](int f, int v) {              // columns 4 v .. of the lane's eight
    return reinterpret_cast<const f32x4s*>(sb + L::W + T_BYTES)[(f * 2 + v) * 64 + lane];
  };
  typedef f32x4s Block[2];                       // 32 rows x 16 columns
  auto rows8 = [](const f32x4s (&a)[2], float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = a[e >> 2][e & 3];
  };

  Block S[DB];
  {
    // the prompt's state or zero; behind the first segment the state before it,
    // or, where that is not known yet, zero or the identity
    // (the first segment has no use for M: its place keeps the state that the
    // prompt starts from, which the last segment of the third launch overwrites
    // while the first may not have read it yet)
    const float* from = Sg;
    bool read = seg == 0 ? !p.has_state || p.has_state[i] != 0 : OUT;
    if (seg > 0) from = own - (size_t)p.H * SEG_FLOATS + c0 + n;
    if (OUT && seg == 0 && !last) {
      from = own + DK * DV + c0 + n;
      read = true;
    }
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 32 * db + 8 * hi + e;
        S[db][e >> 2][e & 3] = read ? from[(size_t)row * DV] : unit && row == c0 + n ? 1.f : 0.f;
      }
    if (!OUT && seg == 0) {
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          own[DK * DV + (size_t)(32 * db + 8 * hi + e) * DV + c0 + n] = S[db][e >> 2][e & 3];
    }
  }

  // The wave's outputs of a chunk leave in the next chunk's time: from LDS,
  // columns of 64 tokens in eight swizzled pieces, as rows of eight columns.
  bf16* op = reinterpret_cast<bf16*>(p.o) + s0 * p.os + (int64_t)h * DV + c0;
  u32x4 out[2];
  const int og = hi & 1, ot = 16 * (hi >> 1);
  const uint32_t oo = (uint32_t)((ot + n) * p.os * 2) + og * 16;
  auto read_out = [&](const unsigned char* s) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {                // lane i of a group: column 8 og + i / 4 (and + 4), tokens 4 (i % 4) ..
      const int t = ot + 32 * u + tc, c = 8 * og + ti;
      auto at = [&](int cc) { return s + cc * 128 + ((t >> 3) ^ (cc & 7)) * 16 + (t & 7) * 2; };
      out[u] = __builtin_bit_cast(u32x4, join(read_tr(at(c)), read_tr(at(c + 4))));
    }
  };
  auto store_out = [&](int t0, int cnt) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (ot + n + 32 * u < cnt)
        *reinterpret_cast<u32x4*>(reinterpret_cast<unsigned char*>(op + (t0 + 32 * u) * p.os) + oo) = out[u];
  };

  bf16x8 ss[DB][3];                              // the state's split blocks
  {
    float x[8];
    rows8(S[0], x);
    split8(x, ss[0]);
  }
  // Where R is no finite number it is left out, so that it reaches no earlier
  // token, and the state's column becomes NaN; `since`: the first token at which
  // that came to the lane's rows of its column, whose outputs from the column's
  // first on are put right at the end.
  int since = NEVER;
  int t0 = 0, buf = 0;
  // one chunk; `more`: a whole one follows (no branch may then stand between
  // two regions, or work for the second is not done in the first)
  auto chunk = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;
    // this wave's copies for the chunk have landed, then everybody's; and
    // everybody has read the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    sb = smem + buf * L::BUF;
    const float* s_g = reinterpret_cast<const float*>(sb + L::W + T_BYTES + P_BYTES);
    const unsigned char* s_v = sb + L::V + wv * 2048;
    const int left = len - t0 - PC;
    const uint32_t lnext = lds0 + (buf ^ 1) * L::BUF;
    auto copies = [&](int from, int to) {
      if constexpr (MORE) {
#pragma unroll
        for (int u = from; u < to; ++u)
          if (u < UNITS) copy_unit(u, lnext);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    bf16x8 fa[2][2][2], ft[2][2][2][3], fs[2][DB][2], vv[2];
    f32x4s fp[2][2][2][2];
    float gm[2][8], dm[2][8];
    auto load_kq = [&](int at, int j) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int t = 0; t < 2; ++t) fa[j & 1][rb][t] = frag_kq(at, rb, t, j % DB);
    };
    load_kq(L::K, 0);
    __builtin_amdgcn_sched_barrier(0);
    if (OUT && t0 > 0) read_out(smem + (buf ^ 1) * L::BUF + L::V + wv * 2048);
    const float gC = s_g[PC - 1];
    next_chunk();
    if (!MORE && left > 0) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the outputs are read where V will land
      copy_last(left, lnext);
    }
    __builtin_amdgcn_sched_barrier(0);

    Block R[2], O[2], U[2];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int t = 0; t < 2; ++t) R[rb][t] = O[rb][t] = U[rb][t] = f32x4s{0.f, 0.f, 0.f, 0.f};
    // R = K S (three values of S)
#pragma unroll
    for (int j = 0; j < DB; ++j) {
      if (j + 1 < DB) {
        load_kq(L::K, j + 1);
        float x[8];
        rows8(S[j + 1], x);
        split8(x, ss[j + 1]);
      } else if (OUT) {
        load_kq(L::Q, DB);                       // (block 0 of Q, into the buffer that follows)
      }
#pragma unroll
      for (int v = 0; v < 3; ++v)
#pragma unroll
        for (int rb = 0; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < 2; ++t) R[rb][t] = mm32(fa[j & 1][rb][t], ss[j][v], R[rb][t]);
      if (j < 2) {                               // what R and U need besides
        const int rb = j;
        ldn<8>(s_g + 32 * rb + 8 * hi, gm[rb]);
        ldn<8>(s_g + PC + 32 * rb + 8 * hi, dm[rb]);
        const unsigned char* sv = s_v + (32 * rb + 8 * hi + ti) * 32 + tc * 2;
        vv[rb] = join(read_tr(sv), read_tr(sv + 4 * 32));
      }
      region<12, 1, 4>();
      copies(2 * j, 2 * j + 2);
    }
    if (OUT && t0 > 0) store_out(t0 - PC, PC);
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 br[2][3];
    int low = 16;                                // the first of the lane's values of R that is none (8 rb + e)
    auto load_t = [&](int kb) {
#pragma unroll
      for (int rb = kb; rb < 2; ++rb)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int v = 0; v < 3; ++v) ft[kb][rb][t][v] = frag_t((rb + kb) * 2 + t, v);
    };
    auto split_r = [&](int rb) {
      float x[8];
      int l = 16;
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        const float v = !OUT && unit ? 0.f : (float)vv[rb][e];
        x[e] = v - gm[rb][e] * R[rb][e >> 2][e & 3];
        const bool ok = finite(x[e]);
        l = ok ? l : 8 * rb + e;
        x[e] = ok ? x[e] : 0.f;
      }
      low = min(low, l);
      split8<true>(x, br[rb]);
    };
    // O = Q S (three values);  R = V - g (K S) and its split meanwhile
#pragma unroll
    for (int j = 0; j < DB; ++j) {
      if constexpr (OUT) {
        if (j + 1 < DB) load_kq(L::Q, DB + j + 1);
        else load_t(0);
#pragma unroll
        for (int v = 2; v >= 0; --v)
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
#pragma unroll
            for (int t = 0; t < 2; ++t) O[rb][t] = mm32(fa[(DB + j) & 1][rb][t], ss[j][v], O[rb][t]);
      } else if (j == 0) {
        load_t(0);
      }
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
        if (j == (rb + 1) * DB / 4) split_r(rb);
      if constexpr (OUT) region<12, 2, 5>();
      copies(2 * DB + j, 2 * DB + j + 1);
    }
    bf16x8 bu[2][3];
    auto split_u = [&](int kb) {
      float x[8];
      rows8(U[kb], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= dm[kb][e];
      split8(x, bu[kb]);
    };
    auto load_ps = [&](int kb) {
#pragma unroll
      for (int rb = kb; rb < 2; ++rb)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (OUT) fp[kb][rb][t][v] = frag_p((rb + kb) * 2 + t, v);
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int t = 0; t < 2; ++t) fs[kb][db][t] = frag_kt(db, t, kb);
    };
    // U = T R, the smaller products first; O = g O and S = g_C S meanwhile
    constexpr int TA[6] = {0, 2, 1, 0, 1, 0}, TB[6] = {2, 0, 1, 1, 0, 0};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (kb == 0) load_t(1);
      else load_ps(0);
#pragma unroll
      for (int v = 0; v < 6; ++v)
#pragma unroll
        for (int rb = kb; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < 2; ++t) U[rb][t] = mm32(ft[kb][rb][t][TA[v]], br[kb][TB[v]], U[rb][t]);
      if (kb == 0) {
        const float gS = column_poison(low < 16, gC);
        if (OUT) since = low < 16 && since == NEVER ? t0 + 32 * (low >> 3) + 8 * hi + (low & 7) : since;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
          for (int rb = 0; rb < 2; ++rb)
            if (OUT) O[rb][e >> 2][e & 3] *= gm[rb][e];
#pragma unroll
          for (int db = 0; db < DB; ++db) S[db][e >> 2][e & 3] *= gS;
        }
        region<24, 1, 2>();
        copies(3 * DB, 3 * DB + 2);
      } else {
        split_u(0);                              // (U's first block has no second step)
        region<12, 2, 7>();
        copies(3 * DB + 2, 3 * DB + 3);
      }
    }
    // S += K^T (D_C U);  O += P U (fp32 instructions)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      if (kb == 0) {
        load_ps(1);
        split_u(1);
      }
#pragma unroll
      for (int d0 = 0; d0 < DB; d0 += 2)         // (two blocks at a time: the first are done early)
#pragma unroll
        for (int v = 2; v >= 0; --v)
#pragma unroll
          for (int db = d0; db < d0 + 2; ++db)
#pragma unroll
            for (int t = 0; t < 2; ++t) S[db][t] = mm32(fs[kb][db][t], bu[kb][v], S[db][t]);
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int rb = kb; rb < 2; ++rb)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (OUT) O[rb][t] = mm4(fp[kb][rb][t][e >> 2][e & 3], U[kb][e >> 2][e & 3], O[rb][t]);
      if (kb == 0) {
        region<(OUT ? 32 : 0) + 6 * DB, 1, 3>();
        copies(3 * DB + 3, UNITS);
      }
    }
    unsigned char* so = smem + buf * L::BUF + L::V + wv * 2048;
#pragma unroll
    for (int rb = 0; rb < (OUT ? 2 : 0); ++rb) {
      bf16x8 w;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = (__bf16)O[rb][e >> 2][e & 3];
      *reinterpret_cast<bf16x8*>(so + n * 128 + ((4 * rb + hi) ^ (n & 7)) * 16) = w;
    }
    float x[8];
    rows8(S[0], x);
    split8(x, ss[0]);
    region<(OUT ? 16 : 0) + 6 * DB, 0, 3>();
    t0 += PC;
    buf ^= 1;
  };
  while (len - t0 >= 2 * PC) chunk(std::true_type{});
  while (t0 < len) chunk(std::false_type{});
  if (OUT && len > 0) {
    wave_lds_sync();
    read_out(sb + L::V + wv * 2048);
    store_out(t0 - PC, len - (t0 - PC));
  }

  if (OUT && __any(since != NEVER)) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int first = column_first(since);
    for (int64_t t = (int64_t)first + hi; t < len; t += 4) op[t * p.os + n] = 0x7fc0;
  }
  if (OUT && !last) return;                      // (the state behind a segment is known already)
  float* to = OUT ? Sg : own + (unit ? DK * DV : 0) + c0 + n;
  const int ld = unit ? DK : DV;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int e = 0; e < 8; ++e) to[(size_t)(32 * db + 8 * hi + e) * ld] = S[db][e >> 2][e & 3];
  if (!OUT || !p.prime) return;
  const int off = p.sk.off[h], r = p.sk.off[h + 1] - off;
  if (r == 0) {                                  // a dense-fallback head: the state copy
    int slot = 0;
    while (slot + 1 < p.sk.ndense && p.sk.dense_list[slot] != h) ++slot;
    bf16* C = reinterpret_cast<bf16*>(p.sk.Sc) + ((size_t)b * p.sk.ndense + slot) * DK * DV + c0 + n;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int e = 0; e < 8; ++e) C[(size_t)(32 * db + 8 * hi + e) * DV] = f32_to_bf16(S[db][e >> 2][e & 3]);
    return;
  }
  bf16* Ug = reinterpret_cast<bf16*>(p.sk.U) + ((size_t)b * p.sk.R + off) * DV + c0 + n;
  for (int j = 0; j < r; ++j) {                  // u_j = S^T p_j
    const float* P = p.sk.Pt + (size_t)(off + j) * DK + 8 * hi;
    float a = 0.f;
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      float x[8], w[8];
      rows8(S[db], x);
      ldn<8>(P + 32 * db, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) a += x[e] * w[e];
    }
    a = xsum<4, 2>(a);                           // over the four row groups
    if (hi == 0) Ug[(size_t)j * DV] = f32_to_bf16(a);
  }
}

// The states between a prompt's segments: S behind segment g is M_g S + B_g,
// written over B_g.  One workgroup of four waves per (prompt, head, 32 columns), a
// wave per 16 columns and half of the rows (the fp32 products bound a step: 64 x 128
// x 16 of them a wave 1.9 us; all rows in a wave and 64 columns a workgroup took 6.4 us
// a step), in fp32 throughout: a tile of S (rows 4 hi + r of column n) is the B
// operand of v_mfma_f32_16x16x4_f32 with K-step r over rows {4 k + r}, so M is read as
// runs of four columns (from LDS, one segment ahead, its pieces swizzled by row),
// the state stays in registers, and the halves are exchanged as they are.
template <int DK, int DV>
__global__ void __launch_bounds__(256) prompt_join_kernel(PromptParams p) {
  constexpr int TB = DK / 16, HB = TB / 2, SEG_FLOATS = DK * (DV + DK), PPR = DK / 4, NW = 4, RUNS = DK * DK * 4 / 1024 / NW;
  extern __shared__ __align__(1024) unsigned char smem[];      // M twice, then the halves of S
  const int tile = blockIdx.x % (p.nchunked * p.H), x = tile / p.H, h = tile - x * p.H;
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, hi = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), cw = wv & 1, half = (wv >> 1) * HB;
  const int c0 = blockIdx.x / (p.nchunked * p.H) * 32 + cw * 16;
  int rank = 0;
  const int i = chunked_prompt(p, x, &rank);
  if (i < 0) return;
  const int s0 = p.start[i], len = p.start[i + 1] - s0;
  const int segs = (int)(((int64_t)len + (1 << p.seg_shift) - 1) >> p.seg_shift);
  if (!prompt_ok(p, i, h, p.seqs ? p.seqs[i] : i) || segs < 3) return;
  float* seg = p.seg + ((size_t)first_slot(s0, rank, p.seg_shift) * p.H + h) * SEG_FLOATS;
  const size_t step = (size_t)p.H * SEG_FLOATS;
  const uint32_t lds0 = lds_address(smem);
  f32x4s* s_x = reinterpret_cast<f32x4s*>(smem + 2 * DK * DK * 4) + cw * TB * 64 + lane;
  auto copy = [&](int g) {                       // M_g into its buffer
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      const int c = 64 * (u * NW + wv) + lane, row = c / PPR, pc = c % PPR;
      copy16(seg + g * step + DK * DV, (row * PPR + (pc ^ (row & 15))) * 16,
             lds0 + (g & 1) * DK * DK * 4 + (u * NW + wv) * 1024);
    }
  };
  f32x4s S[TB], N[HB];
  auto tile_at = [&](const float* B, int tb) {
    f32x4s v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = B[(size_t)(16 * tb + 4 * hi + r) * DV + c0 + n];
    return v;
  };
  copy(1);
#pragma unroll
  for (int tb = 0; tb < TB; ++tb) S[tb] = tile_at(seg, tb);
#pragma unroll
  for (int tb = 0; tb < HB; ++tb) N[tb] = tile_at(seg + step, half + tb);
  for (int g = 1; g + 1 < segs; ++g) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int tb = 0; tb < HB; ++tb) asm volatile("" : "+v"(N[tb]));      // (or its wait would be for the copies too)
    __syncthreads();
    if (g + 2 < segs) copy(g + 1);
    const float* Mg = reinterpret_cast<const float*>(smem + (g & 1) * DK * DK * 4) + half * 16 * DK;
#pragma unroll
    for (int kb = 0; kb < TB; ++kb)
#pragma unroll
      for (int tb = 0; tb < HB; ++tb) {
        float a[4];
        ld4(Mg + ((16 * tb + n) * PPR + ((4 * kb + hi) ^ n)) * 4, a);
#pragma unroll
        for (int r = 0; r < 4; ++r) N[tb] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], S[kb][r], N[tb], 0, 0, 0);
      }
    float* B = seg + g * step;
#pragma unroll
    for (int tb = 0; tb < HB; ++tb) {
      s_x[(half + tb) * 64] = N[tb];
#pragma unroll
      for (int r = 0; r < 4; ++r) B[(size_t)(16 * (half + tb) + 4 * hi + r) * DV + c0 + n] = N[tb][r];
    }
    if (g + 2 < segs) {
#pragma unroll
      for (int tb = 0; tb < HB; ++tb) N[tb] = tile_at(B + step, half + tb);
      __syncthreads();
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) S[tb] = s_x[tb * 64];
    }
  }
}

template <int DK, int DV, int NW, bool OUT>
void launch_chunks(const PromptParams& p, hipStream_t st) {
  const unsigned tiles = (unsigned)(p.seg_shift ? p.nsegs : p.nchunked) * p.H;
  constexpr unsigned PARTS = OUT ? DV / (16 * NW) : (DV + DK) / (16 * NW);
  hipLaunchKernelGGL((prompt_chunk_kernel<DK, DV, NW, OUT>), dim3((tiles + 7) / 8 * 8 * PARTS), dim3(64 * NW), (ChunkLds<DK, NW>::BYTES),
                     st, p);
}

template <int DK, int DV>
int launch(int act, const PromptParams& p, hipStream_t st) {
  constexpr int NW = DV / 16;                    // a workgroup has all columns of a tile
  const dim3 prep((unsigned)p.nslots * p.H);
  if (act == DT_F32) {
    hipLaunchKernelGGL((prompt_prep_kernel<DK, float>), prep, dim3(256), 0, st, p);
    return launch_prompt_chunks_f32(DK, DV, p, st);
  }
  hipLaunchKernelGGL((prompt_prep_kernel<DK, bf16>), prep, dim3(256), 0, st, p);
  if (p.seg_shift) {
    launch_chunks<DK, DV, NW, false>(p, st);
    hipLaunchKernelGGL((prompt_join_kernel<DK, DV>), dim3((unsigned)p.nchunked * p.H * (DV / 32)), dim3(256),
                       2 * DK * DK * 4 + 2 * DK * 64, st, p);
    launch_chunks<DK, DV, NW, true>(p, st);
  } else if (p.nchunked * p.H <= 128) {
    // .. unless that leaves CUs idle (128 x 128, 2048 tokens each, with four and
    // eight waves: 64 tiles 152 and 217 us, 128 205 and 258, 160 321 and 277,
    // 256 387 and 360)
    launch_chunks<DK, DV, 4, true>(p, st);
  } else {
    launch_chunks<DK, DV, NW, true>(p, st);
  }
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_prompt_chunks(int dk, int dv, int act, const PromptParams& p, hipStream_t st) {
  if (dk == 64 && dv == 64) return launch<64, 64>(act, p, st);
  if (dk == 128 && dv == 64) return launch<128, 64>(act, p, st);
  if (dk == 128 && dv == 128) return launch<128, 128>(act, p, st);
  return -2;
}

}  // namespace sk
