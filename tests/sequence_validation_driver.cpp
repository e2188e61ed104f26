// Host-only driver of the validation of the scan, convolution, beam and reorder
// calls, built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_sequence_sanitizers.py.  The kernel launchers are stubs: those of the
// scan and the convolution walk random lists of prompts through the slots and bytes
// that the plan gives them, and no invalid call may reach a launch.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "sketchssm.h"
#include "../ssm_decode_amd/csrc/sk_beam.hpp"
#include "../ssm_decode_amd/csrc/sk_conv.hpp"
#include "../ssm_decode_amd/csrc/sk_scan.hpp"

static int g_launches = 0, g_fail = 0, g_segmented = 0, g_step_segments = 0, g_both = 0, g_moved = 0;
static int64_t g_need = 0;
#define EXPECT(cond)                                                         \
  do {                                                                       \
    if (!(cond)) {                                                           \
      fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);      \
      ++g_fail;                                                              \
    }                                                                        \
  } while (0)

static std::mt19937 g_rng(11);
static int draw(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g_rng); }

static std::vector<int> random_list(int rep, int nseq, int tokens, int len_lo) {
  std::vector<int> start(nseq + 1);
  for (int& s : start) s = rep == 0 ? 0 : draw(0, tokens);
  if (rep == 0 || rep > 2) start[nseq] = tokens;
  std::sort(start.begin(), start.end());
  if (rep == 1)                                  // as many of the shortest as there may be
    for (int i = 0; i <= nseq; ++i) {
      const int64_t at = (int64_t)i * (len_lo + 1);
      start[i] = (int)(at < tokens ? at : tokens);
    }
  return start;
}

// The slots that the kernels give to a list's prompts, as the device code
// counts them, stay apart and within `slots`.
static void walk(const std::vector<int>& start, int64_t len_lo, int shift, int64_t slots, int64_t most) {
  int64_t rank = 0, next = 0;
  for (size_t i = 0; i + 1 < start.size(); ++i) {
    const int64_t len = start[i + 1] - start[i];
    if (len <= len_lo) continue;
    const int64_t first = ((int64_t)start[i] >> shift) + rank;
    EXPECT(first >= next);
    next = first + (len + ((int64_t)1 << shift) - 1) / ((int64_t)1 << shift);
    EXPECT(next <= slots);
    ++rank;
  }
  EXPECT(rank <= most);
}

static void scan_slots(int dk, int dv, const sk::ScanParams& p) {
  for (int rep = 0; rep < 6; ++rep) {
    const std::vector<int> start = random_list(rep, p.nseq, p.tokens, p.len_lo);
    int64_t chunked = 0;
    for (int i = 0; i < p.nseq; ++i) chunked += start[i + 1] - start[i] > p.len_lo;
    EXPECT(chunked <= p.nchunked);
    if (p.seg_shift) walk(start, p.len_lo, p.seg_shift, p.nsegs, p.nchunked);
  }
  if (!p.seg_shift) return;
  // the states, and the decays behind them
  const int64_t states = (int64_t)p.nsegs * p.H * dk * dv * 4;
  const int64_t at = reinterpret_cast<char*>(p.seg_decay) - reinterpret_cast<char*>(p.seg);
  EXPECT(at % 16 == 0 && at >= states && at + (int64_t)p.nsegs * p.H * 4 <= g_need);
  EXPECT(p.seg_shift >= 5 && p.seg_shift < 31);
  EXPECT(p.len_lo == -1 || dk >= 64);
  // the join's threads, 32 bits of them
  EXPECT((int64_t)p.nchunked * p.H * ((dk * dv / 4 + 255) / 256) * 256 <= UINT32_MAX);
}

namespace sk {
int launch_m2(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int launch_gdn(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int launch_kda(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int noalloc_scratch(void** out) { *out = nullptr; return 0; }

static int g_chunk_len_lo;
int launch_scan_chunks(int dk, int dv, const ScanParams& p, hipStream_t) {
  ++g_launches;
  scan_slots(dk, dv, p);
  g_segmented += p.seg_shift != 0;
  const int units = p.H / p.G * (dv / SCAN_COLS);
  EXPECT(dk >= 64 && p.waves >= 2 && p.waves <= SCAN_WAVES && p.waves % 2 == 0 && p.parts >= 1);
  EXPECT(p.waves * p.parts >= units && p.waves * (p.parts - 1) < units);
  EXPECT(((int64_t)(p.seg_shift ? p.nsegs : p.nchunked) * p.G + 7) * p.parts * 64 * p.waves <= UINT32_MAX);
  g_chunk_len_lo = p.len_lo;
  return 0;
}
int launch_scan_step(int dk, int dv, int act, const ScanParams& p, hipStream_t) {
  ++g_launches;
  if (p.nchunked > 0) {                          // all prompts, in segments
    EXPECT(p.seg_shift && p.len_lo == -1 && p.len_hi == INT32_MAX);
    scan_slots(dk, dv, p);
    EXPECT((int64_t)p.nsegs * p.H * 512 <= UINT32_MAX);
    ++g_step_segments;
  } else if (g_chunk_len_lo != INT_MIN) {        // what the chunked form left, and no more
    EXPECT(p.len_hi == g_chunk_len_lo);
    ++g_both;
  } else {
    EXPECT(p.len_hi == INT32_MAX || p.tokens - p.nseq < 64);
  }
  EXPECT((int64_t)p.nseq * p.H * 512 <= UINT32_MAX);
  (void)act;
  return 0;
}
int launch_conv(int dtype, int taps, const ConvParams& p, hipStream_t) {
  ++g_launches;
  const int vec = dtype == SKSSM_F32 ? 4 : 8;
  int64_t channels = 0, waves = 0;
  for (const auto& q : p.piece) {
    EXPECT(q.first == channels);
    channels += q.size;
    waves += ((int64_t)q.size + 64 * vec - 1) / (64 * vec);
  }
  EXPECT(channels == p.channels && waves > 0 && (waves + 3) / 4 <= 65535 && taps >= 2 && taps <= CONV_MAX_TAPS);
  if (p.start) {
    const int64_t slots = ((int64_t)p.tokens >> p.shift) + p.nseq;
    EXPECT(p.shift >= 3 && p.shift < 31 && slots * 256 <= UINT32_MAX);
    for (int rep = 0; rep < 6 && p.nseq <= 1000; ++rep) walk(random_list(rep, p.nseq, p.tokens, 0), -1, p.shift, slots, p.nseq);
  } else {
    EXPECT(p.tokens == p.nseq);
  }
  return 0;
}
int launch_beam_select(int dtype, const BeamParams& p, hipStream_t) {
  ++g_launches;
  const int64_t rows = (int64_t)p.groups * p.beams, es = dtype == SKSSM_F32 ? 4 : 2;
  EXPECT((int64_t)p.parts * BEAM_PART >= p.vocab + 16 / es - 1);      // at any alignment
  EXPECT(rows * p.parts * 256 <= UINT32_MAX && rows * p.parts * (int64_t)sizeof(BeamPart) <= g_need);
  EXPECT((int64_t)p.beams * p.vocab <= INT32_MAX);
  return 0;
}
int launch_reorder(const ReorderParams& p, hipStream_t) {
  ++g_launches;
  int64_t blocks = 0;
  EXPECT(p.nrows >= 1 && p.nrows <= MOVE_MAX && p.groups >= 1);
  for (int r = 0; r < p.nrows; ++r) {
    const auto& q = p.rows[r];
    EXPECT(q.bytes > 0 && q.bytes % q.unit == 0 && reinterpret_cast<uintptr_t>(q.data) % 16 == 0);
    blocks += (q.bytes / q.unit + 255) / 256;
  }
  EXPECT(blocks * p.groups * 256 <= UINT32_MAX);
  g_moved = p.nrows;
  return 0;
}
}  // namespace sk

static void* const FAKE = reinterpret_cast<void*>(0x10000);

static sketchssm_buffers bufs() {
  sketchssm_buffers b;
  memset(&b, 0, sizeof b);
  b.S = static_cast<float*>(FAKE);
  b.U = b.Scopy = b.ring_k = b.ring_v = b.ring_gate = FAKE;
  b.Pt = b.A = static_cast<const float*>(FAKE);
  b.ring_beta = static_cast<float*>(FAKE);
  b.ring_pc = static_cast<decltype(b.ring_pc)>(FAKE);
  b.rank_offsets = static_cast<const int32_t*>(FAKE);
  b.count = static_cast<int32_t*>(FAKE);
  b.err = static_cast<int32_t*>(FAKE);
  return b;
}

int main() {
  std::vector<int32_t> off;
  auto layer = [&](int family, int batch, int heads, int groups, int dk, int dv, int dt) {
    off.assign(heads + 1, 0);
    for (int h = 0; h < heads; ++h) off[h + 1] = off[h] + (h == 0 && heads > 1 ? 0 : 4);
    sketchssm_layer L;
    memset(&L, 0, sizeof L);
    L.family = family;
    L.batch = batch;
    L.heads = heads;
    L.qk_groups = groups;
    L.dk = dk;
    L.dv = dv;
    L.window = 8;
    L.act_dtype = L.sketch_dtype = dt;
    L.rank_offsets_host = off.data();
    return L;
  };
  const int shapes[4][2] = {{16, 32}, {64, 64}, {128, 64}, {128, 128}};
  const sketchssm_buffers B = bufs();
  const int32_t* ix = static_cast<const int32_t*>(FAKE);

  // the scan: lengths from nothing to the most, the plan walked by the stubs
  for (int rep = 0; rep < 3000; ++rep) {
    const int* sh = shapes[draw(0, 3)];
    const int groups = draw(1, 8), heads = groups * draw(1, 16), dt = draw(0, 1) ? SKSSM_F32 : SKSSM_BF16;
    const int nseq = draw(0, 4) ? draw(0, 6) : draw(0, 300);
    const int tokens = draw(0, 1) ? draw(0, 400) : draw(0, 1 << draw(1, 22));
    const sketchssm_layer L = layer(SKSSM_MAMBA2, nseq + draw(1, 3), heads, groups, sh[0], sh[1], dt);
    const int64_t need = sketchssm_scan_workspace_bytes(&L, tokens, nseq);
    if (need < 0) {
      EXPECT(need == SKSSM_EDIM);
      continue;
    }
    sketchssm_scan_prompts p;
    memset(&p, 0, sizeof p);
    p.q = p.k = p.v = p.dt = p.o = p.work = FAKE;
    p.q_stride = p.k_stride = groups * sh[0];
    p.v_stride = p.o_stride = heads * sh[1];
    p.dt_stride = heads;
    p.tokens = tokens;
    p.nseq = nseq;
    p.seq_start = ix;
    p.prime = draw(0, 1);
    p.work_bytes = g_need = need;
    sk::g_chunk_len_lo = INT_MIN;
    const int before = g_launches;
    EXPECT(sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_OK);
    EXPECT((g_launches > before) == (nseq > 0));
    const int now = g_launches;
    if (need > 0) {
      p.work_bytes = need - 1;
      EXPECT(sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_EINVAL);
      p.work_bytes = need;
    }
    if (nseq > 0) {
      p.prime = 2;
      EXPECT(sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_EFLAG);
      p.prime = 0;
      p.seq_start = nullptr;
      EXPECT(sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_EINVAL);
      if (tokens > 0) {
        p.seq_start = ix;
        p.dt_stride = INT64_MAX;
        EXPECT(sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_EDIM);
        p.dt_stride = heads;
        p.o_stride = INT64_MIN;
        EXPECT(sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_EDIM);
      }
    }
    EXPECT(g_launches == now);
  }
  EXPECT(g_segmented > 20 && g_step_segments > 20 && g_both > 20);
  {
    const sketchssm_layer L = layer(SKSSM_MAMBA2, INT_MAX, 64, 1, 128, 128, SKSSM_BF16);
    EXPECT(sketchssm_scan_workspace_bytes(&L, INT_MAX, INT_MAX) < 0);
    EXPECT(sketchssm_scan_workspace_bytes(&L, -1, 1) < 0);
    EXPECT(sketchssm_scan_workspace_bytes(&L, 1, -1) < 0);
    EXPECT(sketchssm_scan_workspace_bytes(nullptr, 1, 1) < 0);
    const sketchssm_layer D = layer(SKSSM_GDN, 4, 8, 8, 128, 128, SKSSM_BF16);
    EXPECT(sketchssm_scan_workspace_bytes(&D, 1, 1) < 0);
  }

  // the convolution
  for (int rep = 0; rep < 2000; ++rep) {
    sketchssm_convolution c;
    memset(&c, 0, sizeof c);
    c.dtype = draw(0, 1) ? SKSSM_F32 : SKSSM_BF16;
    int64_t channels = 0;
    for (auto& q : c.piece) {
      const int units[4] = {0, 16, 64, 128};
      q.unit = units[draw(0, 3)];
      q.channels = draw(0, 40) * (q.unit ? q.unit : 8);
      q.y = FAKE;
      q.y_stride = q.channels + 8;
      channels += q.channels;
    }
    c.x = c.state = FAKE;
    c.x_stride = channels;
    c.weight = static_cast<const float*>(FAKE);
    c.err = static_cast<int32_t*>(FAKE);
    c.taps = draw(2, 8);
    c.activation = draw(SKSSM_ACT_NONE, SKSSM_ACT_SIGMOID);
    c.nseq = draw(0, 3) ? draw(0, 20) : draw(0, 5000);
    c.batch = c.nseq + draw(0, 3);
    const bool step = draw(0, 1);
    c.seq_start = step ? nullptr : ix;
    c.tokens = step ? c.nseq : draw(0, 1 << draw(1, 30));
    int now = g_launches;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_OK);
    EXPECT(g_launches == now + (c.nseq > 0 && channels > 0));
    now = g_launches;
    const sketchssm_convolution good = c;
    if (c.nseq == 0 || channels == 0) continue;
    c.seq_start = nullptr;
    c.tokens = c.nseq + 1;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EDIM);
    c = good;
    c.piece[1].channels = INT_MAX;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EDIM);
    c.piece[0].channels = c.piece[1].channels = c.piece[2].channels = INT_MAX / 128 * 128;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EDIM);
    c = good;
    c.taps = draw(0, 1) ? 1 : 9;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EDIM);
    c = good;
    c.eps = NAN;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EINVAL);
    c = good;
    c.nseq = c.batch + 1;
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EDIM);
    c = good;
    c.state = reinterpret_cast<void*>(0x10008);
    EXPECT(sketchssm_conv(&c, nullptr) == SKSSM_EINVAL);
    EXPECT(g_launches == now);
  }
  EXPECT(sketchssm_conv(nullptr, nullptr) == SKSSM_EINVAL);

  // the selection of beams
  for (int rep = 0; rep < 2000; ++rep) {
    sketchssm_beams b;
    memset(&b, 0, sizeof b);
    b.groups = draw(0, 1) ? draw(0, 80) : draw(0, INT_MAX);
    b.beams = draw(1, 16);
    b.vocab = draw(1, 1 << draw(0, 24));
    b.dtype = draw(0, 1) ? SKSSM_F32 : SKSSM_BF16;
    b.end_token = draw(-1, b.vocab - 1);
    b.stride = b.vocab + (int64_t)draw(0, 9);
    b.logits = b.work = FAKE;
    b.scores = static_cast<const float*>(FAKE);
    b.new_scores = static_cast<float*>(FAKE);
    b.new_ended = b.parents = b.tokens = b.err = static_cast<int32_t*>(FAKE);
    const int64_t need = sketchssm_beam_workspace_bytes(b.groups, b.beams, b.vocab, b.dtype);
    int now = g_launches;
    b.work_bytes = g_need = need;
    if (need < 0) {
      EXPECT(need == SKSSM_EDIM && sketchssm_beam_select(&b, nullptr) == SKSSM_EDIM && g_launches == now);
      continue;
    }
    EXPECT(sketchssm_beam_select(&b, nullptr) == SKSSM_OK);
    EXPECT(g_launches == now + (b.groups > 0));
    now = g_launches;
    b.end_token = b.vocab;
    EXPECT(sketchssm_beam_select(&b, nullptr) == SKSSM_EDIM);
    b.end_token = -1;
    b.stride = (int64_t)INT_MAX + 1;
    EXPECT(sketchssm_beam_select(&b, nullptr) == SKSSM_EDIM);
    b.stride = b.vocab;
    b.work_bytes = need - 1;
    if (b.groups > 0) EXPECT(sketchssm_beam_select(&b, nullptr) == SKSSM_EINVAL);
    EXPECT(g_launches == now);
  }
  EXPECT(sketchssm_beam_workspace_bytes(-1, 1, 1, SKSSM_F32) < 0);
  EXPECT(sketchssm_beam_workspace_bytes(1, 17, 1, SKSSM_F32) < 0);
  EXPECT(sketchssm_beam_workspace_bytes(1, 1, (1 << 24) + 1, SKSSM_F32) < 0);

  // the reordering
  for (int rep = 0; rep < 500; ++rep) {
    const int* sh = shapes[draw(0, 3)];
    const int beams = draw(1, 16), family = draw(0, 1) ? SKSSM_MAMBA2 : SKSSM_GDN, heads = draw(1, 9);
    const sketchssm_layer L = layer(family, beams * draw(1, 20), heads, family == SKSSM_MAMBA2 ? 1 : heads, sh[0], sh[1],
                                    draw(0, 1) ? SKSSM_F32 : SKSSM_BF16);
    sketchssm_rows x[4];
    for (int i = 0; i < 4; ++i) x[i] = {reinterpret_cast<void*>((uintptr_t)(i + 1) << 40), 16 * (int64_t)draw(0, 5000)};
    int now = g_launches;
    EXPECT(sketchssm_reorder(&L, &B, x, 4, ix, beams, nullptr) == SKSSM_OK);
    EXPECT(sketchssm_reorder(&L, &B, nullptr, 0, ix, beams, nullptr) == SKSSM_OK);
    EXPECT(g_launches == now + 2 && g_moved >= 5);
    now = g_launches;
    EXPECT(sketchssm_reorder(&L, &B, x, 5, ix, beams, nullptr) == SKSSM_EDIM);
    EXPECT(sketchssm_reorder(&L, &B, x, -1, ix, beams, nullptr) == SKSSM_EDIM);
    EXPECT(sketchssm_reorder(&L, &B, nullptr, 1, ix, beams, nullptr) == SKSSM_EINVAL);
    EXPECT(sketchssm_reorder(&L, &B, x, 1, nullptr, beams, nullptr) == SKSSM_EINVAL);
    EXPECT(sketchssm_reorder(&L, &B, x, 1, ix, 17, nullptr) == SKSSM_EDIM);
    x[2] = x[3];
    x[2].row_bytes += 16;
    EXPECT(x[3].row_bytes == 0 || sketchssm_reorder(&L, &B, x, 4, ix, beams, nullptr) == SKSSM_EINVAL);
    x[0].row_bytes = INT64_MAX / 16 * 16;
    EXPECT(sketchssm_reorder(&L, &B, x, 1, ix, beams, nullptr) == SKSSM_EDIM);
    x[1].row_bytes = x[2].row_bytes = x[3].row_bytes = x[0].row_bytes;
    EXPECT(sketchssm_reorder(&L, &B, x, 4, ix, beams, nullptr) == SKSSM_EDIM);
    const sketchssm_layer M = layer(SKSSM_MAMBA2, INT_MAX, 1, 1, 16, 32, SKSSM_F32);
    EXPECT(sketchssm_reorder(&M, &B, x, 4, ix, 1, nullptr) == SKSSM_EDIM);
    x[0].row_bytes = 24;
    EXPECT(sketchssm_reorder(&L, &B, x, 1, ix, beams, nullptr) == SKSSM_EDIM);
    EXPECT(g_launches == now);
  }

  if (g_fail) return 1;
  printf("all checks passed\n");
  return 0;
}
