// Argument blocks and launchers of the beam selection (sketchssm_beam_select) and
// of the sequences' reordering (sketchssm_reorder).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sk_params.hpp"

namespace sk {

constexpr int BEAM_MAX = 16;             // beams of a group
constexpr int BEAM_THREADS = 256, BEAM_VALUES = 32;      // .. and a lane's values of a part
enum BeamErrBit { ERRBIT_LOGIT = 16 };

// A workgroup's part of a row: its values' maximum and the sum of their
// exponentials over it (wave by wave), and its best values with their indices.
struct BeamPart {
  float top[4], sum[4];
  float value[BEAM_MAX];
  int32_t index[BEAM_MAX];
};

struct BeamParams {
  const void* logits;       // [groups * beams][vocab]
  int64_t stride;
  const float* scores;      // [groups * beams]
  const int32_t* ended;     // [groups * beams] or null
  float* new_scores;
  int32_t* new_ended;
  int32_t* parents;
  int32_t* tokens;
  int32_t* err;
  int groups, beams, vocab, end_token;
  int parts;                // workgroups of a row
  BeamPart* part;           // [groups * beams][parts]
};

// Elements of a workgroup's part of a row.  (Half as many: 320 rows of 128000 in bf16 37 us,
// not 31; 256 in fp32 83, not 49; twice as many: 35 in bf16.)
constexpr int BEAM_PART = BEAM_THREADS * BEAM_VALUES;
// (a vector's elements less one more than the row has: where the row ends just at a
// part's end the last part is empty, which adds nothing)
inline int beam_parts(int vocab, int esize) {
  return (int)(((int64_t)vocab + 16 / esize - 1 + BEAM_PART - 1) / BEAM_PART);
}

int launch_beam_select(int dtype, const BeamParams& p, hipStream_t st);

constexpr int MOVE_MAX = 16;             // buffers of a reordering
struct ReorderParams {
  struct Rows {
    char* data;             // [B] rows
    int64_t bytes;          // of a row
    int unit;               // bytes of a lane's piece: 16, 4 or 2
    int first;              // the launch's first block of a row
  } rows[MOVE_MAX];
  int nrows, blocks;        // buffers, blocks of a group
  int groups, beams;
  const int32_t* parents;   // [groups * beams]
  int32_t* err;
};
int launch_reorder(const ReorderParams& p, hipStream_t st);

}  // namespace sk
