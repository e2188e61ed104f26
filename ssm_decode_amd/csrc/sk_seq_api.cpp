// C ABI of the scan over prompts, the short convolution, the selection of beams
// and the sequences' reordering.  Every check runs before any HIP call, so an
// invalid call launches nothing and writes nothing.
#include <math.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

#include "sketchssm.h"
#include "sk_beam.hpp"
#include "sk_conv.hpp"
#include "sk_scan.hpp"
#include "sk_serve_host.hpp"

using namespace sk::host;

namespace {

int es_of(int32_t dtype) { return dtype == SKSSM_F32 ? 4 : 2; }

// Prompts of up to this many tokens go token by token where the launch has both
// kinds.  Token by token and in chunks, in us at 8, 24 and 48 tokens each: one prompt of
// 64 heads of 128 x 64 11 and 21, 21 and 22, 35 and 22; 64 prompts 66 and 114, 96 and
// 115, 148 and 117; 64 of heads of 64 x 64 38 and 79, 58 and 80, 87 and 83; of heads of
// 128 x 128 119 and 223, 175 and 231, 264 and 238.
constexpr int kShort = 24;

// Workgroups of a convolution's launch along the tokens: its threads are 32 bits.
constexpr int64_t kMaxConvSlots = (1 << 24) - 1;

// How prompts of these sizes are taken: `chunked` prompts at most in chunks (0:
// none), all of them or those of more than kShort tokens; in segments of
// 2^seg_shift tokens (0: whole), with the bytes of their states and decays.
struct Plan {
  int64_t chunked, nsegs, decay_at, bytes;
  bool all, in_chunks;         // (in_chunks false: token by token, all in segments)
  int seg_shift, waves, parts;
};
constexpr int kMinSegShift = 7, kCus = 256;

// Up to so many segments in chunks are joined by those that start from them, each for
// itself, and by a launch of their own where there are more.  128 heads of 128 x 64 in 8
// groups, us with a launch and without: a prompt of 300 tokens (3 segments) 46 and 38, 517
// (5) 51 and 43, 900 (8) 57 and 50, 16384 (8) 449 and 449.
constexpr int kFewSegs = 8;

Plan plan(const sketchssm_layer* L, int64_t tokens, int64_t nseq) {
  Plan p{};
  if (nseq == 0) return p;
  auto segments = [&](int shift) {
    p.seg_shift = shift;
    p.nsegs = sk::prompt_slots(tokens, p.chunked, shift);
    p.decay_at = p.nsegs * L->heads * (int64_t)L->dk * L->dv * 4;
    p.bytes = p.decay_at + (p.nsegs * L->heads * 4 + 15) / 16 * 16;
  };
  if (L->dk < 64 || L->act_dtype != SKSSM_BF16) {
    // Token by token: in segments where tiles are few and prompts long on average,
    // as short as leaves the segments' states within 16 MB.  Prompts of 512 tokens in
    // fp32, whole and in segments: 8 with 16 heads of 64 x 64 122 us and 64 (of 64 tokens;
    // 73 of 32, 81 of 128), 32 of them 141 and 182; 2 with 64 heads of 128 x 64 183 and 107
    // (of 128), 4 of them 183 and 185.  8 of 256 tokens with 16 heads of 64 x 64 65 and 46
    // (of 32), 8 of 128 tokens 34 and 35.
    const int64_t state = (int64_t)L->heads * L->dk * L->dv;
    if (nseq * state <= 1 << 20 && tokens >= 160 * nseq) {
      int shift = 5;
      while ((tokens >> shift) * state > 1 << 22) ++shift;
      if (tokens >> shift >= 2 * nseq) {
        p.chunked = nseq;
        segments(shift);
      }
    }
    return p;
  }
  p.in_chunks = true;
  if (tokens - nseq < kShort) return p;            // (no prompt is longer unless others are empty)
  // Of a mean length above 40, all in chunks.  64 heads of 128 x 64 in 4 groups, us of both
  // launches and of one: 8 prompts of 300 tokens and 64 of 2 (mean 35) 117 and 149; 48 of 48
  // 92 and 88; 4 of 1000 and 60 of 1 (63) 200 and 152; 8 of 600 and 32 of 5 (124) 139 and
  // 111; 16 of 300 and 16 of 5 (153) 101 and 105.
  p.all = tokens > 40 * nseq;
  const int64_t most = tokens / (kShort + 1);
  p.chunked = p.all || nseq < most ? nseq : most;
  const int units = L->heads / L->qk_groups * (L->dv / sk::SCAN_COLS);
  p.parts = (units + sk::SCAN_WAVES - 1) / sk::SCAN_WAVES;
  p.waves = (units / 2 + p.parts - 1) / p.parts * 2;      // (two waves share their values' rows)
  const int64_t row = L->qk_groups * p.parts;    // workgroups of a segment
  // Few workgroups with many tokens: segments, as long as one of each fills the CUs
  // about once (what the prompts' last ones have more than that is short on average);
  // 128 tokens only where even those fit.  Heads of 128 x 64 in 8 groups of 16, us of one
  // prompt in segments of 128, 256 and 512 tokens, and whole: of 517 tokens 48, 63, 98 and
  // 83; of 1100 84, 69, 106 and 154; of 2100 127, 100, 113 and 270.  16384 tokens in
  // segments of 512, 1024, 2048, 4096 and whole: 528, 473, 449, 749 and 2041.  24 prompts
  // of 15715 tokens together in segments of 1024, 2048, 4096 and whole: 493, 527, 406 and
  // 344.
  auto most_segs = [&](int s) {
    return p.chunked == 1 ? (tokens + ((int64_t)1 << s) - 1) >> s : (tokens >> s) + p.chunked;
  };
  int shift = kMinSegShift;
  if (most_segs(shift) * row > kCus) ++shift;
  while ((tokens >> shift) * row > kCus) ++shift;
  if (tokens >> shift >= 2 * p.chunked && p.chunked * row * 2 <= kCus) segments(shift);
  return p;
}

}  // namespace

extern "C" {

int64_t sketchssm_scan_workspace_bytes(const sketchssm_layer* layer, int32_t tokens, int32_t nseq) {
  try {
    if (int rc = check_layer(layer)) return rc;
    if (layer->family != SKSSM_MAMBA2 || tokens < 0 || nseq < 0 || nseq > layer->batch) return SKSSM_EDIM;
    if ((int64_t)nseq * layer->heads > kMaxTiles) return SKSSM_EDIM;
    const Plan pl = plan(layer, tokens, nseq);
    return pl.nsegs * layer->heads > kMaxTiles ? SKSSM_EDIM : pl.bytes;
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_scan(const sketchssm_layer* layer, const sketchssm_buffers* bufs, const sketchssm_scan_prompts* pr,
                   void* hip_stream) {
  try {
    int rc = check_layer(layer);
    if (rc) return rc;
    if (!bufs || !pr) return SKSSM_EINVAL;
    const int64_t need = sketchssm_scan_workspace_bytes(layer, pr->tokens, pr->nseq);
    if (need < 0) return (int)need;
    if ((rc = check_sketch(layer, bufs, pr->prime))) return rc;
    if (pr->nseq == 0) return SKSSM_OK;
    const int H = layer->heads, G = layer->qk_groups, dk = layer->dk, dv = layer->dv;
    const int es = es_of(layer->act_dtype);
    if (!aligned(bufs->S, 16) || !aligned(bufs->count, 16) || !aligned(bufs->err, 16) || !aligned(bufs->A, 16))
      return SKSSM_EINVAL;
    if (!aligned(pr->seq_start, 4)) return SKSSM_EINVAL;
    if ((pr->seqs && !aligned(pr->seqs, 4)) || (pr->has_state && !aligned(pr->has_state, 4))) return SKSSM_EINVAL;
    if (pr->tokens > 0) {
      if (!aligned(pr->q, 16) || !aligned(pr->k, 16) || !aligned(pr->v, 16) || !aligned(pr->o, 16) ||
          !aligned(pr->dt, es))
        return SKSSM_EINVAL;
      if (!row_stride(pr->q_stride, (int64_t)G * dk, es) || !row_stride(pr->k_stride, (int64_t)G * dk, es) ||
          !row_stride(pr->v_stride, (int64_t)H * dv, es) || !row_stride(pr->o_stride, (int64_t)H * dv, es) ||
          pr->dt_stride < H || pr->dt_stride > kMaxStride)
        return SKSSM_EDIM;
    }
    if (need > 0 && (!aligned(pr->work, 16) || pr->work_bytes < need)) return SKSSM_EINVAL;
    sk::ScanParams p{};
    p.B = layer->batch;
    p.H = H;
    p.G = G;
    p.A = bufs->A;
    p.tokens = pr->tokens;
    p.nseq = pr->nseq;
    p.q = pr->q;
    p.k = pr->k;
    p.v = pr->v;
    p.gate = static_cast<const float*>(pr->dt);
    p.o = pr->o;
    p.qs = pr->q_stride;
    p.ks = pr->k_stride;
    p.vs = pr->v_stride;
    p.gs = pr->dt_stride;
    p.os = pr->o_stride;
    p.start = pr->seq_start;
    p.seqs = pr->seqs;
    p.has_state = pr->has_state;
    p.S = bufs->S;
    p.count = bufs->count;
    p.err = bufs->err;
    p.prime = pr->prime;
    if (pr->prime) fill_sketch(&p.sk, layer, bufs);
    hipStream_t st = reinterpret_cast<hipStream_t>(hip_stream);
    p.len_hi = INT32_MAX;
    const Plan pl = plan(layer, pr->tokens, pr->nseq);
    if (pl.chunked > 0) {
      p.nchunked = (int)pl.chunked;
      p.seg_shift = pl.seg_shift;
      p.nsegs = (int)pl.nsegs;
      p.seg = static_cast<float*>(pr->work);
      p.seg_decay = reinterpret_cast<float*>(static_cast<char*>(pr->work) + pl.decay_at);
      p.waves = pl.waves;
      p.parts = pl.parts;
      p.joined = pl.nsegs > kFewSegs;
      p.len_lo = pl.all || !pl.in_chunks ? -1 : kShort;
      if (pl.in_chunks) {
        if ((rc = sk::launch_scan_chunks(dk, dv, p, st)) || pl.all) return rc;
        p.len_hi = kShort;
        p.nchunked = 0;
      }
    }
    return sk::launch_scan_step(dk, dv, layer->act_dtype, p, st);
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_conv(const sketchssm_convolution* cv, void* hip_stream) {
  try {
    if (!cv) return SKSSM_EINVAL;
    if (cv->dtype != SKSSM_F32 && cv->dtype != SKSSM_BF16) return SKSSM_EDTYPE;
    const int es = es_of(cv->dtype);
    if (cv->activation < SKSSM_ACT_NONE || cv->activation > SKSSM_ACT_SIGMOID) return SKSSM_EFLAG;
    if (cv->taps < 2 || cv->taps > sk::CONV_MAX_TAPS) return SKSSM_EDIM;
    if (!(isfinite(cv->eps) && cv->eps >= 0.f)) return SKSSM_EINVAL;
    if (cv->batch < 0 || cv->tokens < 0 || cv->nseq < 0 || cv->nseq > cv->batch || cv->nseq > kMaxTiles) return SKSSM_EDIM;
    if (!cv->seq_start && cv->tokens != cv->nseq) return SKSSM_EDIM;
    sk::ConvParams p{};
    int64_t channels = 0;
    for (int i = 0; i < sk::CONV_PIECES; ++i) {
      const sketchssm_conv_piece& q = cv->piece[i];
      if (q.channels < 0 || q.channels % 8 != 0) return SKSSM_EDIM;
      if (q.unit != 0 && q.unit != 16 && q.unit != 64 && q.unit != 128) return SKSSM_EDIM;
      if (q.unit != 0 && q.channels % q.unit != 0) return SKSSM_EDIM;
      p.piece[i].y = q.y;
      p.piece[i].ys = q.y_stride;
      p.piece[i].first = (int)channels;
      p.piece[i].size = q.channels;
      p.piece[i].unit = q.unit;
      channels += q.channels;
    }
    if (channels > kMaxStride) return SKSSM_EDIM;
    if (cv->nseq == 0 || channels == 0) return SKSSM_OK;
    if (!aligned(cv->weight, 16) || (cv->bias && !aligned(cv->bias, 16)) || !aligned(cv->state, 16) ||
        !aligned(cv->err, 4))
      return SKSSM_EINVAL;
    if ((cv->seq_start && !aligned(cv->seq_start, 4)) || (cv->seqs && !aligned(cv->seqs, 4)) ||
        (cv->has_state && !aligned(cv->has_state, 4)))
      return SKSSM_EINVAL;
    if (cv->tokens > 0) {
      if (!aligned(cv->x, 16)) return SKSSM_EINVAL;
      if (!row_stride(cv->x_stride, channels, es)) return SKSSM_EDIM;
      for (int i = 0; i < sk::CONV_PIECES; ++i) {
        if (p.piece[i].size == 0) continue;
        if (!aligned(p.piece[i].y, 16)) return SKSSM_EINVAL;
        if (!row_stride(p.piece[i].ys, p.piece[i].size, es)) return SKSSM_EDIM;
      }
    }
    p.x = cv->x;
    p.xs = cv->x_stride;
    p.weight = cv->weight;
    p.bias = cv->bias;
    p.state = cv->state;
    p.B = cv->batch;
    p.channels = (int)channels;
    p.act = cv->activation;
    p.tokens = cv->tokens;
    p.nseq = cv->nseq;
    p.start = cv->seq_start;
    p.seqs = cv->seqs;
    p.has_state = cv->has_state;
    p.err = cv->err;
    p.eps = cv->eps;
    // Blocks of 32 tokens, shorter where that leaves CUs idle (each takes taps - 1
    // more rows).  12288 channels in bf16, in blocks of 8, 16 and 32 tokens: one prompt
    // of 517 12.3, 14.0 and 22.3 us, of 2048 29, 26 and 31, of 4096 50, 47 and 43.
    p.shift = 5;
    const int64_t parts = (channels * es / 1024 + 6) / 4;
    while (p.shift > 3 && ((cv->tokens >> p.shift) + cv->nseq) * parts < 800) --p.shift;
    while (((int64_t)cv->tokens >> p.shift) + cv->nseq > kMaxConvSlots) ++p.shift;
    return sk::launch_conv(cv->dtype, cv->taps, p, reinterpret_cast<hipStream_t>(hip_stream));
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int64_t sketchssm_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t vocab, int32_t dtype) {
  if (dtype != SKSSM_F32 && dtype != SKSSM_BF16) return SKSSM_EDTYPE;
  if (groups < 0 || beams < 1 || beams > sk::BEAM_MAX || vocab < 1 || vocab > 1 << 24) return SKSSM_EDIM;
  const int64_t parts = (int64_t)groups * beams * sk::beam_parts(vocab, es_of(dtype));
  return parts > kMaxTiles ? SKSSM_EDIM : parts * (int64_t)sizeof(sk::BeamPart);
}

int sketchssm_beam_select(const sketchssm_beams* bm, void* hip_stream) {
  try {
    if (!bm) return SKSSM_EINVAL;
    const int64_t need = sketchssm_beam_workspace_bytes(bm->groups, bm->beams, bm->vocab, bm->dtype);
    if (need < 0) return (int)need;
    if (bm->end_token < -1 || bm->end_token >= bm->vocab) return SKSSM_EDIM;
    if (bm->stride < bm->vocab || bm->stride > INT32_MAX) return SKSSM_EDIM;
    if (bm->groups == 0) return SKSSM_OK;
    if (!aligned(bm->logits, es_of(bm->dtype)) || !aligned(bm->scores, 4) || (bm->ended && !aligned(bm->ended, 4)) ||
        !aligned(bm->new_scores, 4) || !aligned(bm->new_ended, 4) || !aligned(bm->parents, 4) ||
        !aligned(bm->tokens, 4) || !aligned(bm->err, 4))
      return SKSSM_EINVAL;
    if (!aligned(bm->work, 16) || bm->work_bytes < need) return SKSSM_EINVAL;
    sk::BeamParams p{};
    p.logits = bm->logits;
    p.stride = bm->stride;
    p.scores = bm->scores;
    p.ended = bm->ended;
    p.new_scores = bm->new_scores;
    p.new_ended = bm->new_ended;
    p.parents = bm->parents;
    p.tokens = bm->tokens;
    p.err = bm->err;
    p.groups = bm->groups;
    p.beams = bm->beams;
    p.vocab = bm->vocab;
    p.end_token = bm->end_token;
    p.parts = sk::beam_parts(bm->vocab, es_of(bm->dtype));
    p.part = static_cast<sk::BeamPart*>(bm->work);
    return sk::launch_beam_select(bm->dtype, p, reinterpret_cast<hipStream_t>(hip_stream));
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

int sketchssm_reorder(const sketchssm_layer* layer, const sketchssm_buffers* bufs, const sketchssm_rows* extra,
                      int32_t nextra, const int32_t* parents, int32_t beams, void* hip_stream) {
  try {
    if (int rc = check_layer(layer)) return rc;
    if (!bufs || (nextra > 0 && !extra)) return SKSSM_EINVAL;
    if (beams < 1 || beams > sk::BEAM_MAX || layer->batch % beams != 0 || nextra < 0 || nextra > 4) return SKSSM_EDIM;
    if (!aligned(parents, 4) || !aligned(bufs->err, 16)) return SKSSM_EINVAL;
    const int64_t B = layer->batch, H = layer->heads, G = layer->qk_groups, dk = layer->dk, dv = layer->dv;
    const int64_t W = layer->window, R = layer->rank_offsets_host[layer->heads], es = es_of(layer->act_dtype);
    const bool m2 = layer->family == SKSSM_MAMBA2;
    int64_t dense = 0;
    for (int h = 0; h < H; ++h) dense += layer->rank_offsets_host[h + 1] == layer->rank_offsets_host[h];
    sk::ReorderParams p{};
    int64_t blocks = 0;
    bool ok = true;
    auto add = [&](void* data, int64_t bytes) {
      if (bytes == 0) return;
      ok = ok && aligned(data, 16);
      auto& r = p.rows[p.nrows++];
      r.data = static_cast<char*>(data);
      r.bytes = bytes;
      r.unit = bytes % 16 == 0 ? 16 : bytes % 4 == 0 ? 4 : 2;
      blocks += bytes / r.unit / 256 + 1;
    };
    add(bufs->S, H * dk * dv * 4);
    add(bufs->U, R * dv * es);
    if (layer->coef_map == SKSSM_COEF_STATE) add(bufs->Cstate, R * dk * es);
    add(bufs->Scopy, dense * dk * dv * es);
    add(bufs->ring_k, G * W * dk * es);
    add(bufs->ring_v, H * W * dv * es);
    add(bufs->ring_gate, layer->family == SKSSM_KDA ? H * W * dk * 4 : H * W * (m2 ? es : 4));
    if (!m2) add(bufs->ring_beta, H * W * 4);
    if (!m2 && layer->pullback == SKSSM_PULLBACK_PROJ) add(bufs->ring_pc, H * W * 64);
    add(bufs->count, H * 4);
    const int own = p.nrows;
    for (int i = 0; i < nextra; ++i) {
      if (extra[i].row_bytes < 0 || extra[i].row_bytes % 16 != 0 || extra[i].row_bytes > kMaxTiles * 4096) return SKSSM_EDIM;
      add(extra[i].data, extra[i].row_bytes);
    }
    if (!ok) return SKSSM_EINVAL;
    if (blocks * (B / beams) > kMaxTiles) return SKSSM_EDIM;
    // (rows listed twice would be moved twice, at once)
    for (int i = own; i < p.nrows; ++i)
      for (int j = 0; j < i; ++j) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(p.rows[i].data), y = reinterpret_cast<uintptr_t>(p.rows[j].data);
        if (x < y + B * p.rows[j].bytes && y < x + B * p.rows[i].bytes) return SKSSM_EINVAL;
      }
    p.groups = (int)(B / beams);
    p.beams = beams;
    p.parents = parents;
    p.err = bufs->err;
    if (p.groups == 0) return SKSSM_OK;
    return sk::launch_reorder(p, reinterpret_cast<hipStream_t>(hip_stream));
  } catch (...) {
    return SKSSM_ELAUNCH;
  }
}

}  // extern "C"
