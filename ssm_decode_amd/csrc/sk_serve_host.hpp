// Host-side checks shared by the calls around the decode steps.
#pragma once

#include <stdint.h>

#include "sketchssm.h"
#include "sk_serve.hpp"

namespace sk {
namespace host {

// (tiles of a launch: its threads, 256 or 512 to a tile, are counted in 32 bits)
constexpr int64_t kMaxTiles = (1 << 22) - 1;

inline bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A row stride whose rows stay 16-byte aligned and do not overlap (the kernels'
// offsets within a group of rows are 32 bits).
constexpr int64_t kMaxStride = 1 << 25;
inline bool row_stride(int64_t stride, int64_t row, int esize) {
  return stride >= row && stride <= kMaxStride && (stride * esize) % 16 == 0;
}

inline int check_layer(const sketchssm_layer* L) {
  const int64_t w = sketchssm_workspace_bytes(L);
  return w < 0 ? (int)w : SKSSM_OK;
}

// The sketch of the written tiles (prime): the fixed map only, since a
// state-dependent map is formed by the flush.
inline int check_sketch(const sketchssm_layer* L, const sketchssm_buffers* B, int32_t prime) {
  if (prime != 0 && prime != 1) return SKSSM_EFLAG;
  if (!prime) return SKSSM_OK;
  if (L->coef_map != SKSSM_COEF_FIXED) return SKSSM_EFLAG;
  bool dense = false;
  for (int h = 0; h < L->heads; ++h) dense |= L->rank_offsets_host[h + 1] == L->rank_offsets_host[h];
  if (L->rank_offsets_host[L->heads] > 0 && (!aligned(B->U, 16) || !aligned(B->Pt, 16))) return SKSSM_EINVAL;
  if (dense && !aligned(B->Scopy, 16)) return SKSSM_EINVAL;
  return aligned(B->rank_offsets, 16) ? SKSSM_OK : SKSSM_EINVAL;
}

inline void fill_sketch(sk::SketchOut* s, const sketchssm_layer* L, const sketchssm_buffers* B) {
  s->U = B->U;
  s->Pt = B->Pt;
  s->off = B->rank_offsets;
  s->Sc = B->Scopy;
  s->R = L->rank_offsets_host[L->heads];
  int nd = 0;                                    // (at most DENSE_LIST_MAX: check_layer)
  for (int h = 0; h < L->heads; ++h)
    if (L->rank_offsets_host[h + 1] == L->rank_offsets_host[h]) s->dense_list[nd++] = (int16_t)h;
  s->ndense = nd;
}

}  // namespace host
}  // namespace sk
