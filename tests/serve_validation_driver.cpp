// Host-only driver of the validation of the prompt, state-cache and norm
// calls, built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_serving_sanitizers.py.  The kernel launchers are stubs: the
// prompt one walks random lists of prompts through the slots and bytes that
// the plan gives them, and no invalid call may reach a launch.
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <vector>

#include "sketchssm.h"
#include "../ssm_decode_amd/csrc/sk_serve.hpp"

static int g_launches = 0, g_fail = 0, g_segmented = 0;
#define EXPECT(cond)                                                         \
  do {                                                                       \
    if (!(cond)) {                                                           \
      fprintf(stderr, "FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);      \
      ++g_fail;                                                              \
    }                                                                        \
  } while (0)

static std::mt19937 g_rng(7);
static int draw(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g_rng); }

// The slots that the kernels give to a list's prompts, as the device code
// counts them, stay apart and within `slots`.
static void walk(const std::vector<int>& start, int64_t len_lo, int shift, int64_t slots, int64_t most) {
  int64_t rank = 0, next = 0;
  for (size_t i = 0; i + 1 < start.size(); ++i) {
    const int64_t len = start[i + 1] - start[i];
    if (len <= len_lo) continue;
    const int64_t first = ((int64_t)start[i] >> shift) + rank;
    EXPECT(first >= next);
    next = first + (len + (1 << shift) - 1) / (1 << shift);
    EXPECT(next <= slots);
    ++rank;
  }
  EXPECT(rank <= most);
}

namespace sk {
int launch_m2(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int launch_gdn(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int launch_kda(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int noalloc_scratch(void** out) { *out = nullptr; return 0; }

int launch_prompt_chunks(int dk, int dv, int, const PromptParams& p, hipStream_t) {
  ++g_launches;
  for (int rep = 0; rep < 6; ++rep) {
    std::vector<int> start(p.nseq + 1);
    for (int& s : start) s = rep == 0 ? 0 : draw(0, p.tokens);
    if (rep == 0 || rep > 2) start[p.nseq] = p.tokens;
    std::sort(start.begin(), start.end());
    if (rep == 1)                                // as many of the shortest as there may be
      for (int i = 0; i <= p.nseq; ++i) start[i] = (int)((int64_t)i * (p.len_lo + 1) < p.tokens ? i * (p.len_lo + 1) : p.tokens);
    walk(start, p.len_lo, 6, p.nslots, p.nchunked);
    if (p.seg_shift) walk(start, p.len_lo, p.seg_shift, p.nsegs, p.nchunked);
  }
  if (p.seg_shift) {
    ++g_segmented;
    const int64_t at = reinterpret_cast<char*>(p.seg) - static_cast<char*>(p.work);
    EXPECT(at % 16 == 0 && at >= (int64_t)p.nslots * p.H * PROMPT_CHUNK_WORK + PROMPT_WORK_OVER);
    EXPECT(p.seg_shift >= 6 && p.seg_shift < 31);
  }
  // the threads of the launches, 32 bits of them
  EXPECT((int64_t)p.nslots * p.H * 256 <= UINT32_MAX && (int64_t)p.nchunked * p.H * 512 <= UINT32_MAX);
  (void)dk;
  (void)dv;
  return 0;
}
int launch_prompt_step(int, int, int, const PromptParams& p, hipStream_t) {
  ++g_launches;
  EXPECT((int64_t)p.nseq * p.H * 512 <= UINT32_MAX);
  return 0;
}
int launch_state_save(int, int, const CacheParams& p, hipStream_t) {
  ++g_launches;
  EXPECT((int64_t)p.n * p.H * 256 <= UINT32_MAX);
  return 0;
}
int launch_state_load(int, int, int, const CacheParams& p, hipStream_t) {
  ++g_launches;
  EXPECT((int64_t)p.n * p.H * 256 <= UINT32_MAX);
  EXPECT(!p.prime || p.sk.ndense == 1);
  return 0;
}
int launch_group_norm(int, const NormParams& p, hipStream_t) {
  ++g_launches;
  EXPECT(p.rows > 0 && p.width <= 8192 && p.groups <= 65535);
  return 0;
}
}  // namespace sk

static void* const FAKE = reinterpret_cast<void*>(0x10000);

static sketchssm_buffers bufs() {
  sketchssm_buffers b;
  memset(&b, 0, sizeof b);
  b.S = static_cast<float*>(FAKE);
  b.U = b.Scopy = FAKE;
  b.Pt = static_cast<const float*>(FAKE);
  b.rank_offsets = static_cast<const int32_t*>(FAKE);
  b.count = static_cast<int32_t*>(FAKE);
  b.err = static_cast<int32_t*>(FAKE);
  return b;
}

int main() {
  std::vector<int32_t> off;
  auto layer = [&](int batch, int heads, int dk, int dv, int dt) {
    off.assign(heads + 1, 0);
    for (int h = 0; h < heads; ++h) off[h + 1] = off[h] + (h == 0 && heads > 1 ? 0 : 4);
    sketchssm_layer L;
    memset(&L, 0, sizeof L);
    L.family = SKSSM_GDN;
    L.batch = batch;
    L.heads = heads;
    L.qk_groups = heads;
    L.dk = dk;
    L.dv = dv;
    L.window = 8;
    L.act_dtype = L.sketch_dtype = dt;
    L.rank_offsets_host = off.data();
    return L;
  };
  const int shapes[4][2] = {{16, 32}, {64, 64}, {128, 64}, {128, 128}};
  const sketchssm_buffers B = bufs();

  // prompts: lengths from nothing to the most, the plan walked by the stub
  for (int rep = 0; rep < 3000; ++rep) {
    const int* sh = shapes[draw(0, 3)];
    const int heads = draw(0, 3) ? draw(1, 8) : draw(9, 64), dt = draw(0, 1) ? SKSSM_F32 : SKSSM_BF16;
    const int nseq = draw(0, 4) ? draw(0, 6) : draw(0, 300);
    const int tokens = draw(0, 1) ? draw(0, 400) : draw(0, 1 << draw(1, 22));
    const sketchssm_layer L = layer(nseq + draw(1, 3), heads, sh[0], sh[1], dt);
    const int64_t need = sketchssm_prefill_workspace_bytes(&L, tokens, nseq);
    if (need < 0) {
      EXPECT(need == SKSSM_EDIM);
      continue;
    }
    sketchssm_prompts p;
    memset(&p, 0, sizeof p);
    p.q = p.k = p.v = p.o = p.work = FAKE;
    p.gate = p.beta = static_cast<const float*>(FAKE);
    p.q_stride = p.k_stride = heads * sh[0];
    p.v_stride = p.o_stride = heads * sh[1];
    p.gate_stride = p.beta_stride = heads;
    p.tokens = tokens;
    p.nseq = nseq;
    p.seq_start = static_cast<const int32_t*>(FAKE);
    p.prime = draw(0, 1);
    p.work_bytes = need;
    const int before = g_launches;
    EXPECT(sketchssm_prefill(&L, &B, &p, nullptr) == SKSSM_OK);
    EXPECT((g_launches > before) == (nseq > 0));
    const int now = g_launches;
    if (need > 0) {
      p.work_bytes = need - 1;
      EXPECT(sketchssm_prefill(&L, &B, &p, nullptr) == (nseq > 0 ? SKSSM_EINVAL : SKSSM_OK));
      p.work_bytes = need;
    }
    if (nseq > 0) {
      p.prime = 2;
      EXPECT(sketchssm_prefill(&L, &B, &p, nullptr) == SKSSM_EFLAG);
      p.prime = 0;
      p.seq_start = nullptr;
      EXPECT(sketchssm_prefill(&L, &B, &p, nullptr) == SKSSM_EINVAL);
      if (tokens > 0) {
        p.seq_start = static_cast<const int32_t*>(FAKE);
        p.o_stride = INT64_MAX;
        EXPECT(sketchssm_prefill(&L, &B, &p, nullptr) == SKSSM_EDIM);
        p.o_stride = INT64_MIN;
        EXPECT(sketchssm_prefill(&L, &B, &p, nullptr) == SKSSM_EDIM);
      }
    }
    EXPECT(g_launches == now);
  }
  EXPECT(g_segmented > 20);
  {
    const sketchssm_layer L = layer(INT_MAX, 64, 128, 128, SKSSM_BF16);
    EXPECT(sketchssm_prefill_workspace_bytes(&L, INT_MAX, INT_MAX) < 0);
    EXPECT(sketchssm_prefill_workspace_bytes(&L, -1, 1) < 0);
    EXPECT(sketchssm_prefill_workspace_bytes(&L, 1, -1) < 0);
    EXPECT(sketchssm_prefill_workspace_bytes(nullptr, 1, 1) < 0);
  }

  // the state cache
  for (int rep = 0; rep < 300; ++rep) {
    const int* sh = shapes[draw(0, 3)];
    const sketchssm_layer L = layer(8, draw(2, 9), sh[0], sh[1], draw(0, 1) ? SKSSM_F32 : SKSSM_BF16);
    sketchssm_state_cache C = {FAKE, static_cast<float*>(FAKE), draw(0, 5), draw(0, 1) ? 8 : 4};
    const int32_t* ix = static_cast<const int32_t*>(FAKE);
    const int now = g_launches;
    EXPECT(sketchssm_state_save(&L, &B, &C, ix, ix, 3, nullptr) == SKSSM_OK);
    EXPECT(sketchssm_state_load(&L, &B, &C, ix, ix, 3, 1, nullptr) == SKSSM_OK);
    EXPECT(g_launches == now + 2);
    EXPECT(sketchssm_state_load(&L, &B, &C, ix, ix, 0, 1, nullptr) == SKSSM_OK);
    EXPECT(sketchssm_state_load(&L, &B, &C, ix, ix, INT_MAX, 1, nullptr) == SKSSM_EDIM);
    EXPECT(sketchssm_state_save(&L, &B, &C, ix, ix, -1, nullptr) == SKSSM_EDIM);
    EXPECT(sketchssm_state_save(&L, &B, nullptr, ix, ix, 1, nullptr) == SKSSM_EINVAL);
    EXPECT(sketchssm_state_save(&L, &B, &C, nullptr, ix, 1, nullptr) == SKSSM_EINVAL);
    C.bits = 16;
    EXPECT(sketchssm_state_save(&L, &B, &C, ix, ix, 1, nullptr) == SKSSM_EDTYPE);
    EXPECT(g_launches == now + 2);
  }

  // the norm
  sketchssm_norm n;
  memset(&n, 0, sizeof n);
  n.x = n.y = FAKE;
  n.x_stride = n.y_stride = (int64_t)65535 * 8;
  n.rows = INT64_MAX;
  n.groups = 65535;
  n.width = 8;
  n.dtype = SKSSM_BF16;
  int now = g_launches;
  EXPECT(sketchssm_group_norm(&n, nullptr) == SKSSM_OK);
  EXPECT(g_launches == now + 1);
  n.eps = -1.f;
  EXPECT(sketchssm_group_norm(&n, nullptr) == SKSSM_EINVAL);
  n.eps = INFINITY;
  EXPECT(sketchssm_group_norm(&n, nullptr) == SKSSM_EINVAL);
  n.eps = 0.f;
  n.first = reinterpret_cast<const int32_t*>(0x10002);
  EXPECT(sketchssm_group_norm(&n, nullptr) == SKSSM_EINVAL);
  n.first = nullptr;
  n.groups = INT_MAX;
  EXPECT(sketchssm_group_norm(&n, nullptr) == SKSSM_EDIM);
  EXPECT(sketchssm_group_norm(nullptr, nullptr) == SKSSM_EINVAL);
  EXPECT(g_launches == now + 1);

  if (g_fail) return 1;
  printf("all checks passed\n");
  return 0;
}
