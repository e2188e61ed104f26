// Device code shared by the prompt and state-cache kernels: which prompt a
// workgroup may take, and the sketch of a tile held in registers.
#pragma once

#include "sk_device.hpp"
#include "sk_serve.hpp"

namespace sk {

typedef float f32x4s __attribute__((ext_vector_type(4)));

// Whether an entry before position i of a device list names the same index
// (every thread of the workgroup takes part; uniform result).
__device__ __forceinline__ bool listed_before(const int32_t* list, int i, int idx) {
  int dup = 0;
  for (int j = threadIdx.x; j < i; j += blockDim.x) dup |= list[j] == idx;
  return __syncthreads_or(dup) != 0;
}

// Prompt i and its sequence, checked.  A list of first tokens that falls
// anywhere, or leaves [0, tokens], reports ERRBIT_SEQ and is refused whole (so
// that no two prompts share tokens, and at most tokens / n prompts have n
// tokens); an index outside the batch, or a sequence that an earlier prompt
// has (which keeps it), refuses this prompt; a tile whose ring still holds
// entries reports ERRBIT_COUNT.  Uniform over the workgroup, whose threads
// all take part.
__device__ __forceinline__ bool prompt_ok(const PromptParams& p, int i, int h, int b) {
  int wrong = 0;
  for (int j = threadIdx.x; j < p.nseq; j += blockDim.x) {
    const int s0 = p.start[j], s1 = p.start[j + 1];
    wrong |= s0 < 0 || s1 < s0 || s1 > p.tokens;
    if (p.seqs && j < i) wrong |= p.seqs[j] == b;
  }
  wrong |= b < 0 || b >= p.B;
  int bad = __syncthreads_or(wrong) ? ERRBIT_SEQ : 0;
  if (!bad && p.count[(size_t)b * p.H + h] != 0) bad = ERRBIT_COUNT;
  if (bad && threadIdx.x == 0) atomicOr(p.err, bad);
  return bad == 0;
}

// Sum over the four rows of 16 lanes; every lane receives it.  (Lane swaps are
// vector instructions: no LDS permute in the chain from token to token.)
__device__ __forceinline__ float row_groups_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Registers of a wave's 16 NCC columns of a tile (NCC = 2: as the flush holds
// them): with cg = lane % 16 and rg = lane / 16,
//   s[mb][c][v] = S[16 mb + 4 rg + v][col0 + NCC cg + c].
// The layout is the A operand of v_mfma_f32_16x16x4_f32 for S^T (K-step
// (mb, v) covers rows 16 mb + 4 k + v), so the sketch needs no data movement:
// lane holds u_j, j = cg, at columns col0 + NCC (4 rg + vv) + c.
template <int DK, int DV, typename UT, int NCC>
__device__ __forceinline__ void sketch_tile(const SketchOut& sk, const float (&s)[DK / 16][NCC][4], int b, int h,
                                            int col0, int lane) {
  constexpr int MB = DK / 16;
  const int cg = lane & 15, rg = lane >> 4;
  const int off = sk.off[h], r = sk.off[h + 1] - off;
  if (r == 0) {                       // a dense-fallback head: the state copy
    int slot = 0;
    while (slot + 1 < sk.ndense && sk.dense_list[slot] != h) ++slot;
    UT* C = reinterpret_cast<UT*>(sk.Sc) + ((size_t)b * sk.ndense + slot) * DK * DV + col0 + NCC * cg;
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float x[NCC];
#pragma unroll
        for (int c = 0; c < NCC; ++c) x[c] = s[mb][c][v];
        stn<NCC>(C + (size_t)(16 * mb + 4 * rg + v) * DV, x);
      }
    return;
  }
  f32x4s u[NCC];
#pragma unroll
  for (int c = 0; c < NCC; ++c) u[c] = f32x4s{0.f, 0.f, 0.f, 0.f};
  const float* pr = sk.Pt + (size_t)(off + (cg < r ? cg : 0)) * DK + 4 * rg;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    float x[4];
    ld4(pr + 16 * mb, x);
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int c = 0; c < NCC; ++c) u[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(s[mb][c][v], x[v], u[c], 0, 0, 0);
  }
  if (cg < r) {                       // (columns j >= r repeat row 0 and are dropped)
    UT* U = reinterpret_cast<UT*>(sk.U) + ((size_t)b * sk.R + off + cg) * DV + col0 + 4 * NCC * rg;
    float x[4 * NCC];
#pragma unroll
    for (int vv = 0; vv < 4; ++vv)
#pragma unroll
      for (int c = 0; c < NCC; ++c) x[NCC * vv + c] = u[c][vv];
    stn<4 * NCC>(U, x);
  }
}

}  // namespace sk
