// Argument block and launchers of the selective state space scan over prompts
// (sketchssm_scan).
#pragma once

#include "sk_serve.hpp"

namespace sk {

// (q and k hold G groups' rows, gate holds dt in the activation dtype; beta is unused;
// seg: [nsegs][H] states behind the segments, dk x dv)
struct ScanParams : PromptParams {
  int G;
  int waves, parts;         // chunked form: waves of a workgroup, workgroups of a group's heads
  bool joined;              // .. the segments' states by a launch of their own
  const float* A;           // [H]
  float* seg_decay;         // [nsegs][H] products of the segments' decays
};

// Chunked form: a wave has 32 columns of a head's state, a workgroup up to eight
// waves with the keys and queries of one group.
constexpr int SCAN_COLS = 32, SCAN_WAVES = 8;

int launch_scan_join(int dk, int dv, const ScanParams& p, hipStream_t st);
int launch_scan_step(int dk, int dv, int act, const ScanParams& p, hipStream_t st);
int launch_scan_chunks(int dk, int dv, const ScanParams& p, hipStream_t st);

}  // namespace sk
