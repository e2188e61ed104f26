// Prompts through the gated delta rule in chunks of 64 tokens.  With alpha_i,
// beta_i of a chunk's tokens, g_i the product of the decays up to token i, D_ij the
// product of those after j up to i (so that no quotient of decays occurs), and S_0
// the state before the chunk:
//   A_ij = beta_i D_ij (k_i . k_j)  for j < i,       T = (I + A)^-1 diag(beta)
//   P_ij = D_ij (q_i . k_j)         for j <= i
//   R = V - diag(g) K S_0,   U = T R
//   O = diag(g) Q S_0 + P U,   S <- g_C S_0 + K^T diag(D_C) U
// T and P do not depend on the state: one launch forms them for every chunk of
// every prompt and head at once; a second goes through each prompt's chunks in
// order.
//
// Precision.  The state is fp32, and so is every product.  They run on the bf16
// matrix cores with each fp32 operand as an exact sum of three bf16 values: a
// product with bf16 data (K, Q, K^T) takes three instructions, one of two fp32
// operands (T R) the six whose terms reach 2^-24 of it.  P U, which only the outputs wait for, takes the fp32
// instructions, a sixteenth of the bf16 ones' rate: P in three values beside T's
// would be too much for LDS twice, and splitting it in registers for six
// instructions takes as long (24 prompts, 16062 tokens, 32 heads of 128 x 128: 371
// and 373 us).  fp32 activations use them throughout, since K and Q would have
// to be split too.
#pragma once

#include "sk_serve_device.hpp"

namespace sk {

constexpr int PC = PROMPT_CHUNK;                 // tokens of a chunk
constexpr int FRAGS = 6;                         // fragments of a lower-triangular 64 x 64 operand
constexpr int FRAG_BYTES = 1024;                 // 64 lanes x 8 bf16
constexpr int T_BYTES = FRAGS * 3 * FRAG_BYTES, P_BYTES = FRAGS * 2 * FRAG_BYTES;
// workspace of a chunk and head: the fragments of T (three values each), then
// of P (in fp32, the lower four columns of a lane's eight, then the upper), then
// g [64] and D_C [64]
constexpr int CHUNK_WORK_BYTES = T_BYTES + P_BYTES + 2 * PC * 4;
// in fp32: the 16 x 16 tiles of T on and below the diagonal, then of P, as A
// operands of the fp32 instruction (four columns a lane), then the same factors
constexpr int F32_TILES = 10;
constexpr int CHUNK_WORK_F32 = 2 * F32_TILES * FRAG_BYTES + 2 * PC * 4;
static_assert(PC == 64 && CHUNK_WORK_BYTES == PROMPT_CHUNK_WORK && CHUNK_WORK_F32 == PROMPT_CHUNK_WORK_F32,
              "workspace of a chunk");

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8 as_frag(const u32x4& x) { return __builtin_bit_cast(bf16x8, x); }

// The slot of a prompt's first chunk (shift 6) or segment of 2^shift tokens, for
// the r-th of the prompts that are taken in chunks: those of prompts that are
// behind one another are apart, and there are at most tokens / 2^shift + their
// number.
__device__ __forceinline__ int first_slot(int start, int r, int shift) { return (start >> shift) + r; }

// Operands of v_mfma_f32_16x16x32_bf16 (hi = lane / 16, n = lane % 16).  A
// block of 32 rows x 16 columns is two result tiles of four registers; MFMA
// row m of tile t is row ((m & 12) << 1) | (t << 2) | (m & 3) of the block, so
// that a lane's eight registers are rows 8 hi .. 8 hi + 7 of column n: the B
// operand of the next product as they stand, and runs of eight tokens.
__device__ __forceinline__ int block_row(int m, int t) { return ((m & 12) << 1) | (t << 2) | (m & 3); }
__device__ __forceinline__ f32x4s mm32(bf16x8 a, bf16x8 b, f32x4s c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4s mm4(float a, float b, f32x4s c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// Eight fp32 values as three bf16 fragments whose exact sum they are.  Cut, a value
// leaves up to 2^-7 of itself to the second and 2^-15 to the third; to nearest
// (values under 2^128 (1 - 2^-9)), 2^-8 and 2^-17, so that a product of two values
// to nearest without its three smallest terms is off by at most 2^-24 (cut: 2^-21,
// always towards zero).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
template <bool NEAREST = false>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&out)[3]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = r[2 * e], hi = r[2 * e + 1];
      if (NEAREST) {
        const bf16x2 v = {(__bf16)lo, (__bf16)hi};
        w[e] = __builtin_bit_cast(uint32_t, v);
      } else {
        w[e] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
      }
      if (t < 2) {
        r[2 * e] = lo - __uint_as_float(NEAREST ? w[e] << 16 : __float_as_uint(lo) & 0xffff0000u);
        r[2 * e + 1] = hi - __uint_as_float((NEAREST ? w[e] : __float_as_uint(hi)) & 0xffff0000u);
      }
    }
    out[t] = as_frag(w);
  }
}

// The prompt that has a slot (of 2^shift tokens: chunks, or segments of a
// prompt), and its rank among those taken in chunks: the last whose first slot
// is not behind this one (-1: none; its own end is for the caller to check).
__device__ __forceinline__ int slot_prompt(const PromptParams& p, int slot, int shift, int* rank) {
  const int lane = threadIdx.x & 63;
  int i = -1, ranks = 0;
  for (int j0 = 0; j0 < p.nseq; j0 += 64) {
    const int j = j0 + lane < p.nseq ? j0 + lane : p.nseq - 1;
    const int a = p.start[j];
    const bool mine = j0 + lane < p.nseq && (int64_t)p.start[j + 1] - a > p.len_lo;
    const unsigned long long all = __ballot(mine);
    const int r = ranks + __popcll(all & ((1ull << lane) - 1));
    const unsigned long long m = __ballot(mine && first_slot(a, r, shift) <= slot);
    if (m) {
      const int l = 63 - __clzll(m);
      i = j0 + l;
      *rank = ranks + __popcll(all & ((1ull << l) - 1));
    }
    ranks += __popcll(all);
  }
  return i;
}

// The x-th of the prompts taken in chunks (-1: there are not so many), and its
// rank among them as listed.  Up to 64 prompts are taken longest first (a lane
// each), so that the last workgroups to start are the shortest; more are taken
// as listed.
__device__ __forceinline__ int chunked_prompt(const PromptParams& p, int x, int* rank) {
  const int lane = threadIdx.x & 63;
  if (p.nseq <= 64) {
    const int j = lane < p.nseq ? lane : 0;
    const int len = p.start[j + 1] - p.start[j];
    const bool mine = lane < p.nseq && len > p.len_lo;
    const unsigned long long all = __ballot(mine);
    if (x >= __popcll(all)) return -1;
    int before = 0;
    for (int k = 0; k < p.nseq; ++k) {
      const int other = __builtin_amdgcn_readlane(len, k);
      before += (all >> k & 1) && (other > len || (other == len && k < lane));
    }
    const unsigned long long m = __ballot(mine && before == x);
    if (!m) return -1;
    const int i = __builtin_ctzll(m);
    *rank = __popcll(all & ((1ull << i) - 1));
    return i;
  }
  int ranks = 0;
  for (int j0 = 0; j0 < p.nseq; j0 += 64) {
    const int j = j0 + lane < p.nseq ? j0 + lane : p.nseq - 1;
    const bool mine = j0 + lane < p.nseq && (int64_t)p.start[j + 1] - p.start[j] > p.len_lo;
    const unsigned long long all = __ballot(mine);
    const unsigned long long m = __ballot(mine && ranks + __popcll(all & ((1ull << lane) - 1)) == x);
    if (m) {
      *rank = x;
      return j0 + __builtin_ctzll(m);
    }
    ranks += __popcll(all);
  }
  return -1;
}

// (The compiler warns that it would not save m0, a reserved register, around the
// statement; it has nothing there to save.)
#pragma clang diagnostic ignored "-Winline-asm"

// x, or NaN in the columns (n = lane % 16) of which one of the four lanes has `bad`.
__device__ __forceinline__ float column_poison(bool bad, float x) {
  const unsigned long long all = __ballot(bad);
  uint32_t m = (uint32_t)(all | all >> 32);
  m |= m >> 16;
  return m >> (threadIdx.x & 15) & 1 ? __builtin_nanf("") : x;
}
// The first of the four lanes' tokens.
constexpr int NEVER = INT32_MAX;
__device__ __forceinline__ int column_first(int t) {
  t = min(t, __shfl_xor(t, 16));
  return min(t, __shfl_xor(t, 32));
}

// 16 bytes of each lane, from base + its offset in memory to lds + 16 * lane
// in LDS (base and lds are uniform), in flight until the wave's next wait for
// its memory counter.  (The compiler would have every LDS read wait for a copy
// that it knows of, also where the two are in different buffers.)
__device__ __forceinline__ void copy16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset),
               "s"(reinterpret_cast<uint64_t>(base)), "s"(lds)
               : "memory", "m0");
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

// The end of a region: its instructions in the order of N times a matrix
// instruction, READS LDS reads and VALU vector instructions (as far as there
// are any), and nothing moved across.
template <int N, int READS, int VALU>
__device__ __forceinline__ void interleave() {
  if constexpr (N > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    if constexpr (VALU > 0) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    interleave<N - 1, READS, VALU>();
  }
}
template <int N, int READS, int VALU>
__device__ __forceinline__ void region() {
  interleave<N, READS, VALU>();
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace sk
