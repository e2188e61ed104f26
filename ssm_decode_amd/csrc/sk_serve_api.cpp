// C ABI of the calls around the decode steps: prompts, the state cache and
// the output norm.  Every check runs before any HIP call, so an invalid call
// launches nothing and writes nothing.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "sketchssm.h"
#include "sk_serve_host.hpp"

using namespace sk::host;

namespace {

constexpr int kMaxWidth = 8192;

// Prompts of up to this many tokens go token by token where the launch has
// both kinds.  A chunk's two launches take about as long for 4 tokens as for 64,
// the other form's time grows by the token; measured, token by token and in
// chunks (us): bf16 128 x 128, 1024 tiles of 24 tokens 75 and 109, of 32 89 and 110,
// 64 tiles of 16 21 and 25, of 24 28 and 24; fp32 128 x 128, 1024 tiles of 32 133
// and 155, 64 tiles of 32 30 and 27; 64 x 64, 1024 tiles of 64 tokens 57 and 73
// (fp32 64 and 80), 128 tiles of fp32 of 32 17 and 21, of 64 28 and 22.
int short_prompt(const sketchssm_layer* L) { return L->dk == 64 ? 48 : L->act_dtype == SKSSM_F32 ? 32 : 24; }
// Prompts in segments: up to kSplitTiles (prompt, head) tiles, at least kMinSegs
// segments of 2^kMinSegShift tokens or more to a prompt on average, at most
// kMaxSegs (the states between them are joined in order, 4 us each) and kSegTiles
// of all tiles (the CUs).  Measured on 128 x 128 tiles, whole and in segments (us): 8
// tiles of 2048 tokens 126 and 109, of 4096 238 and 127, of 12000 654 and 211; 32 of
// 2048 137 and 124, of 16384 1011 and 600; 4 of 32768 1724 and 289; what stays whole:
// 8 of 1600 in three 102 and 103; 48 of 4096 275 and 282; 64 of 16384 1126 and 1156.
// The smaller shapes, whose transitions cost less, gain within these limits (32 tiles
// of 2048 tokens: 128 x 64 142 and 96, 64 x 64 109 and 73; of 16384, 1053 and 513, 844
// and 345) and would beyond (64 of 16384: 1154 and 808, 925 and 642).  fp32 has no
// launch without outputs and goes whole.  The rule knows totals alone: one prompt of
// 16384 tokens of 32 heads goes whole, in 1020 us in place of 600, with any other
// prompt beside it.
constexpr int kSplitTiles = 32, kSegTiles = 256, kMinSegShift = 9, kMinSegs = 4, kMaxSegs = 48;

// How prompts of these sizes are taken: `chunked` prompts at most in chunks (0:
// none), all of them or those of more than short_prompt tokens; in segments of
// 2^seg_shift tokens (0: whole), with the bytes of their states at seg_at.
struct Plan {
  int64_t chunked, slots, nsegs, seg_at, bytes;
  bool all;
  int seg_shift;
};
Plan plan(const sketchssm_layer* L, int64_t tokens, int64_t nseq) {
  Plan p{};
  const int shrt = short_prompt(L);
  if (!sk::prompt_chunked(L->dk) || nseq == 0) return p;
  // No prompt is longer unless others are empty (a decode batch through this
  // call): one launch for all, which takes a long prompt too (32 heads of 128 x
  // 128, with the chunks' launches and without: 256 sequences, a token each, 217 and
  // 212 us; 48 50 and 42; 1024 819 and 787; all others empty, a prompt of 100 tokens
  // in the middle of 256 223 and 214, of 200 241 and 295, of 1018 in 1024 910 and 1338).
  if (tokens - nseq < shrt) return p;
  // mostly long prompts: the chunked form takes the short ones too, and one
  // launch is saved
  p.all = tokens > sk::PROMPT_CHUNK * nseq;
  const int64_t most = tokens / (shrt + 1);
  p.chunked = p.all || nseq < most ? nseq : most;
  p.slots = sk::prompt_slots(tokens, p.chunked, 6);
  p.bytes = p.slots * L->heads * sk::prompt_chunk_work(L->act_dtype) + sk::PROMPT_WORK_OVER;
  // Few tiles with many tokens: segments, as long as one of each tile fills the
  // CUs about once
  if (L->act_dtype == SKSSM_BF16 && p.chunked * L->heads <= kSplitTiles) {
    int shift = kMinSegShift;
    while ((tokens >> shift) * L->heads > kSegTiles || (tokens >> shift) > kMaxSegs * p.chunked) ++shift;
    if ((tokens >> shift) >= kMinSegs * p.chunked) {
      p.seg_shift = shift;
      p.nsegs = sk::prompt_slots(tokens, p.chunked, shift);
      p.seg_at = (p.bytes + 255) / 256 * 256;
      p.bytes = p.seg_at + p.nsegs * L->heads * (int64_t)L->dk * (L->dk + L->dv) * 4;
    }
  }
  return p;
}

int check_cache(const sketchssm_layer* L, const sketchssm_buffers* B, const sketchssm_state_cache* C,
                const int32_t* seqs, const int32_t* slots, int32_t n) {
  if (int rc = check_layer(L)) return rc;
  if (!B || !C) return SKSSM_EINVAL;
  if (C->bits != 8 && C->bits != 4) return SKSSM_EDTYPE;
  if (C->slots < 0 || n < 0) return SKSSM_EDIM;
  if ((int64_t)n * L->heads > kMaxTiles) return SKSSM_EDIM;
  if (n == 0) return SKSSM_OK;
  if (!aligned(seqs, 4) || !aligned(slots, 4)) return SKSSM_EINVAL;
  if (!aligned(B->S, 16) || !aligned(B->count, 16) || !aligned(B->err, 16)) return SKSSM_EINVAL;
  if (!aligned(C->codes, 16) || !aligned(C->scale, 16)) return SKSSM_EINVAL;
  return SKSSM_OK;
}

sk::CacheParams cache_params(const sketchssm_layer* L, const sketchssm_buffers* B, const sketchssm_state_cache* C,
                             const int32_t* seqs, const int32_t* slots, int32_t n) {
  sk::CacheParams p{};
  p.B = L->batch;
  p.H = L->heads;
  p.slots = C->slots;
  p.n = n;
  p.bits = C->bits;
  p.seqs = seqs;
  p.slot = slots;
  p.S = B->S;
  p.count = B->count;
  p.err = B->err;
  p.codes = C->codes;
  p.scale = C->scale;
  return p;
}

}  // namespace

extern "C" {

int64_t sketchssm_prefill_workspace_bytes(const sketchssm_layer* layer, int32_t tokens, int32_t nseq) {
  try {
    if (int rc = check_layer(layer)) return rc;
    if (layer->family != SKSSM_GDN || tokens < 0 || nseq < 0 || nseq > layer->batch) return SKSSM_EDIM;
    if ((int64_t)nseq * layer->heads > kMaxTiles) return SKSSM_EDIM;
    const Plan pl = plan(layer, tokens, nseq);
    return pl.slots * layer->heads > kMaxTiles ? SKSSM_EDIM : pl.bytes;
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_prefill(const sketchssm_layer* layer, const sketchssm_buffers* bufs, const sketchssm_prompts* pr,
                      void* hip_stream) {
  try {
    int rc = check_layer(layer);
    if (rc) return rc;
    if (!bufs || !pr) return SKSSM_EINVAL;
    const int64_t need = sketchssm_prefill_workspace_bytes(layer, pr->tokens, pr->nseq);
    if (need < 0) return (int)need;
    if ((rc = check_sketch(layer, bufs, pr->prime))) return rc;
    if (pr->nseq == 0) return SKSSM_OK;
    const int H = layer->heads, dk = layer->dk, dv = layer->dv;
    const int es = layer->act_dtype == SKSSM_F32 ? 4 : 2;
    if (!aligned(bufs->S, 16) || !aligned(bufs->count, 16) || !aligned(bufs->err, 16)) return SKSSM_EINVAL;
    if (!aligned(pr->seq_start, 4)) return SKSSM_EINVAL;
    if ((pr->seqs && !aligned(pr->seqs, 4)) || (pr->has_state && !aligned(pr->has_state, 4))) return SKSSM_EINVAL;
    if (pr->tokens > 0) {
      if (!aligned(pr->q, 16) || !aligned(pr->k, 16) || !aligned(pr->v, 16) || !aligned(pr->o, 16))
        return SKSSM_EINVAL;
      if (!aligned(pr->gate, 4) || !aligned(pr->beta, 4)) return SKSSM_EINVAL;
      if (!row_stride(pr->q_stride, (int64_t)H * dk, es) || !row_stride(pr->k_stride, (int64_t)H * dk, es) ||
          !row_stride(pr->v_stride, (int64_t)H * dv, es) || !row_stride(pr->o_stride, (int64_t)H * dv, es))
        return SKSSM_EDIM;
      if (pr->gate_stride < H || pr->beta_stride < H || pr->gate_stride > kMaxStride || pr->beta_stride > kMaxStride)
        return SKSSM_EDIM;
    }
    if (need > 0 && (!aligned(pr->work, 16) || pr->work_bytes < need)) return SKSSM_EINVAL;
    sk::PromptParams p{};
    p.B = layer->batch;
    p.H = H;
    p.tokens = pr->tokens;
    p.nseq = pr->nseq;
    p.q = pr->q;
    p.k = pr->k;
    p.v = pr->v;
    p.gate = pr->gate;
    p.beta = pr->beta;
    p.o = pr->o;
    p.qs = pr->q_stride;
    p.ks = pr->k_stride;
    p.vs = pr->v_stride;
    p.gs = pr->gate_stride;
    p.bs = pr->beta_stride;
    p.os = pr->o_stride;
    p.start = pr->seq_start;
    p.seqs = pr->seqs;
    p.has_state = pr->has_state;
    p.S = bufs->S;
    p.count = bufs->count;
    p.err = bufs->err;
    p.prime = pr->prime;
    if (pr->prime) fill_sketch(&p.sk, layer, bufs);
    p.work = pr->work;
    hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
    p.len_hi = INT32_MAX;
    const Plan pl = plan(layer, pr->tokens, pr->nseq);
    if (pl.chunked > 0) {
      p.nchunked = (int)pl.chunked;
      p.nslots = (int)pl.slots;
      p.seg_shift = pl.seg_shift;
      p.nsegs = (int)pl.nsegs;
      p.seg = reinterpret_cast<float*>(static_cast<char*>(pr->work) + pl.seg_at);
      p.len_lo = pl.all ? -1 : short_prompt(layer);
      if ((rc = sk::launch_prompt_chunks(dk, dv, layer->act_dtype, p, st)) || pl.all) return rc;
      p.len_hi = short_prompt(layer);
    }
    return sk::launch_prompt_step(dk, dv, layer->act_dtype, p, st);
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_state_save(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                         const sketchssm_state_cache* cache, const int32_t* seqs, const int32_t* slots, int32_t n,
                         void* hip_stream) {
  try {
    if (int rc = check_cache(layer, bufs, cache, seqs, slots, n)) return rc;
    if (n == 0) return SKSSM_OK;
    return sk::launch_state_save(layer->dk, layer->dv, cache_params(layer, bufs, cache, seqs, slots, n),
                                 reinterpret_cast<hipStream_t>(hip_stream));
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_state_load(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                         const sketchssm_state_cache* cache, const int32_t* seqs, const int32_t* slots, int32_t n,
                         int32_t prime, void* hip_stream) {
  try {
    if (int rc = check_cache(layer, bufs, cache, seqs, slots, n)) return rc;
    if (int rc = check_sketch(layer, bufs, prime)) return rc;
    if (n == 0) return SKSSM_OK;
    sk::CacheParams p = cache_params(layer, bufs, cache, seqs, slots, n);
    p.prime = prime;
    if (prime) fill_sketch(&p.sk, layer, bufs);
    return sk::launch_state_load(layer->dk, layer->dv, layer->sketch_dtype, p,
                                 reinterpret_cast<hipStream_t>(hip_stream));
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_group_norm(const sketchssm_norm* nm, void* hip_stream) {
  try {
    if (!nm) return SKSSM_EINVAL;
    if (nm->dtype != SKSSM_F32 && nm->dtype != SKSSM_BF16) return SKSSM_EDTYPE;
    const int es = nm->dtype == SKSSM_F32 ? 4 : 2;
    if (nm->rows < 0 || nm->groups < 1 || nm->groups > 65535 || nm->width < 8 || nm->width > kMaxWidth ||
        nm->width % 8 != 0)
      return SKSSM_EDIM;
    if (nm->activation < SKSSM_ACT_NONE || nm->activation > SKSSM_ACT_SIGMOID) return SKSSM_EFLAG;
    if ((nm->centred != 0 && nm->centred != 1) || (nm->gate_first != 0 && nm->gate_first != 1)) return SKSSM_EFLAG;
    if (!(isfinite(nm->eps) && nm->eps >= 0.f)) return SKSSM_EINVAL;
    if (nm->rows == 0) return SKSSM_OK;
    if ((nm->first && !aligned(nm->first, 4)) || (nm->end && !aligned(nm->end, 4))) return SKSSM_EINVAL;
    const int64_t row = (int64_t)nm->groups * nm->width;
    if (!aligned(nm->x, 16) || !aligned(nm->y, 16) || (nm->gate && !aligned(nm->gate, 16))) return SKSSM_EINVAL;
    if ((nm->weight && !aligned(nm->weight, 16)) || (nm->bias && !aligned(nm->bias, 16))) return SKSSM_EINVAL;
    if (nm->group_weights != 0 && nm->group_weights != 1) return SKSSM_EFLAG;
    if (!row_stride(nm->x_stride, row, es) || !row_stride(nm->y_stride, row, es) ||
        (nm->gate && !row_stride(nm->gate_stride, row, es)))
      return SKSSM_EDIM;
    sk::NormParams p{};
    p.x = nm->x;
    p.gate = nm->gate;
    p.y = nm->y;
    p.weight = nm->weight;
    p.bias = nm->bias;
    p.xs = nm->x_stride;
    p.zs = nm->gate_stride;
    p.ys = nm->y_stride;
    p.rows = nm->rows;
    p.first = nm->first;
    p.end = nm->end;
    p.groups = nm->groups;
    p.width = nm->width;
    p.wgs = nm->group_weights ? nm->width : 0;
    p.centred = nm->centred;
    p.act = nm->activation;
    p.gate_first = nm->gate_first;
    p.eps = nm->eps;
    return sk::launch_group_norm(nm->dtype, p, reinterpret_cast<hipStream_t>(hip_stream));
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

}  // extern "C"
