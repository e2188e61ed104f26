// Prompts through the gated delta rule in chunks of 64 tokens (bf16
// activations).  With alpha_i, beta_i of a chunk's tokens, g_i the product of
// the decays up to token i, D_ij the product of those after j up to i (so that
// no quotient of decays occurs), and S_0 the state before the chunk:
//   A_ij = beta_i D_ij (k_i . k_j)  for j < i,       T = (I + A)^-1 diag(beta)
//   P_ij = D_ij (q_i . k_j)         for j <= i
//   R = V - diag(g) K S_0,   U = T R
//   O = diag(g) Q S_0 + P U,   S <- g_C S_0 + K^T diag(D_C) U
// T and P do not depend on the state: one launch forms them for every chunk of
// every prompt and head at once; a second goes through each prompt's chunks in
// order.
//
// Precision.  The state is fp32, and so must be what is added to it.  Products
// run on the bf16 matrix cores with each fp32 operand as an exact sum of three
// bf16 values (its top 8 bits, the next 8, the last 8): a product with bf16
// data (K, K^T) takes three instructions, one of two fp32 operands (T R) the
// six whose terms reach 2^-24 of it.  What only reaches the output, which is
// rounded to bf16 at 2^-9, takes the first two values (2^-16).  The fp32 matrix
// instructions have a sixteenth of the bf16 ones' rate.
#pragma once

#include "sk_serve_device.hpp"

namespace sk {

constexpr int PC = PROMPT_CHUNK;                 // tokens of a chunk
constexpr int FRAGS = 6;                         // fragments of a lower-triangular 64 x 64 operand
constexpr int FRAG_BYTES = 1024;                 // 64 lanes x 8 bf16
constexpr int T_BYTES = FRAGS * 3 * FRAG_BYTES, P_BYTES = FRAGS * 2 * FRAG_BYTES;
// workspace of a chunk and head: the fragments of T (three values each), then
// of P (two), then g [64] and D_C [64] in fp32
constexpr int CHUNK_WORK_BYTES = T_BYTES + P_BYTES + 2 * PC * 4;
static_assert(PC == 64 && CHUNK_WORK_BYTES == PROMPT_CHUNK_WORK, "workspace of a chunk");

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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

// Eight fp32 values as bf16 fragments whose sum they are (three: exactly; the
// first two leave at most 2^-16 of a value).
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}
__device__ __forceinline__ float below(float x) {    // x less its top 8 bits
  return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
template <int TERMS>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&out)[TERMS]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = high_halves(r[2 * e], r[2 * e + 1]);
      if (t + 1 < TERMS) {
        r[2 * e] = below(r[2 * e]);
        r[2 * e + 1] = below(r[2 * e + 1]);
      }
    }
    out[t] = as_frag(w);
  }
}

}  // namespace sk
