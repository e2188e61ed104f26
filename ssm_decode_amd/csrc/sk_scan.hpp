// Argument block and launchers of the selective state space scan over prompts
// (sketchssm_scan).
#pragma once

#include "sk_serve.hpp"

namespace sk {

// (q and k hold G groups' rows, gate holds dt in the activation dtype; beta is unused)
struct ScanParams : PromptParams {
  int G;
  int waves, parts;         // chunked form: waves of a workgroup, workgroups of a group's heads
  const float* A;           // [H]
};

// Chunked form: tokens of a chunk, and the bytes of a segment's workspace (a
// head's state and its decay).
constexpr int SCAN_CHUNK = 64;
inline int64_t scan_seg_floats(int dk, int dv) { return (int64_t)dk * dv; }

int launch_scan_step(int dk, int dv, int act, const ScanParams& p, hipStream_t st);
int launch_scan_chunks(int dk, int dv, const ScanParams& p, hipStream_t st);

}  // namespace sk
