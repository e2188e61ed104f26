// Host-only driver of the scan's dispatch, built and read by tests/test_scan_dispatch.py:
// the launchers are stubs that print what they are given.
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "sketchssm.h"
#include "../ssm_decode_amd/csrc/sk_beam.hpp"
#include "../ssm_decode_amd/csrc/sk_conv.hpp"
#include "../ssm_decode_amd/csrc/sk_scan.hpp"

namespace sk {
int launch_m2(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int launch_gdn(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int launch_kda(int, int, int, int, int, int, const Params&, hipStream_t) { return 0; }
int noalloc_scratch(void** out) { *out = nullptr; return 0; }
int launch_conv(int, int, const ConvParams&, hipStream_t) { return 0; }
int launch_beam_select(int, const BeamParams&, hipStream_t) { return 0; }
int launch_reorder(const ReorderParams&, hipStream_t) { return 0; }

int launch_scan_chunks(int, int, const ScanParams& p, hipStream_t) {
  printf("chunks %d %d", p.len_lo, p.seg_shift ? 1 << p.seg_shift : 0);
  printf(p.seg_shift ? p.joined ? " launch\n" : " each\n" : "\n");
  return 0;
}
int launch_scan_step(int, int, int, const ScanParams& p, hipStream_t) {
  const bool cut = p.nchunked > 0 && p.seg_shift;
  if (p.len_hi == INT_MAX) printf("step all");
  else printf("step %d", p.len_hi);
  printf(" %d%s\n", cut ? 1 << p.seg_shift : 0, cut ? " launch" : "");
  return 0;
}
}  // namespace sk

// arguments: heads groups dk dv fp32 tokens prompts
int main(int argc, char** argv) {
  if (argc != 8) return 2;
  int a[7];
  for (int i = 0; i < 7; ++i) a[i] = atoi(argv[i + 1]);
  void* const fake = reinterpret_cast<void*>(0x10000);
  std::vector<int32_t> off(a[0] + 1);
  for (int h = 0; h < a[0]; ++h) off[h + 1] = off[h] + 2;
  sketchssm_layer L;
  memset(&L, 0, sizeof L);
  L.family = SKSSM_MAMBA2;
  L.batch = a[6];
  L.heads = a[0];
  L.qk_groups = a[1];
  L.dk = a[2];
  L.dv = a[3];
  L.window = 4;
  L.act_dtype = L.sketch_dtype = a[4] ? SKSSM_F32 : SKSSM_BF16;
  L.rank_offsets_host = off.data();
  sketchssm_buffers B;
  memset(&B, 0, sizeof B);
  B.S = static_cast<float*>(fake);
  B.U = fake;
  B.Pt = B.A = static_cast<const float*>(fake);
  B.rank_offsets = static_cast<const int32_t*>(fake);
  B.count = B.err = static_cast<int32_t*>(fake);
  sketchssm_scan_prompts p;
  memset(&p, 0, sizeof p);
  p.q = p.k = p.v = p.dt = p.o = p.work = fake;
  p.q_stride = p.k_stride = a[1] * a[2];
  p.v_stride = p.o_stride = a[0] * a[3];
  p.dt_stride = a[0];
  p.tokens = a[5];
  p.nseq = a[6];
  p.seq_start = static_cast<const int32_t*>(fake);
  p.work_bytes = INT64_MAX;
  return sketchssm_scan(&L, &B, &p, nullptr) == SKSSM_OK ? 0 : 1;
}
