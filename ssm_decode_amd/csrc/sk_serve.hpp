// Argument blocks and launchers of the calls around the decode steps: prompts
// (sketchssm_prefill), the state cache (sketchssm_state_save / _load) and the
// output norm (sketchssm_group_norm).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sk_params.hpp"

namespace sk {

enum ServeErrBit { ERRBIT_SLOT = 8 };

// What a kernel that leaves a tile's state behind needs to leave its sketch
// too (fixed coefficient map): U = S^T P, or the state copy of a dense head.
struct SketchOut {
  void* U;
  const float* Pt;
  const int32_t* off;   // [H+1] device rank offsets
  void* Sc;
  int R, ndense;
  int16_t dense_list[DENSE_LIST_MAX];
};

struct PromptParams {
  int B, H;
  int tokens, nseq;
  int len_lo, len_hi;       // the launch takes prompts of more than len_lo and up to len_hi tokens
  int nchunked, nslots;     // chunked form: prompts it may have, chunk slots of the workspace
  int seg_shift, nsegs;     // prompts cut into segments of 2^seg_shift tokens (0: not), their slots
  float* seg;               // [nsegs][H] states behind the segments (dk x dv) and their transitions (dk x dk)
  const void* q;
  const void* k;
  const void* v;
  const float* gate;
  const float* beta;
  void* o;
  int64_t qs, ks, vs, gs, bs, os;   // elements from a token's row to the next
  const int32_t* start;     // [nseq+1]
  const int32_t* seqs;      // [nseq] or null (prompt i belongs to sequence i)
  const int32_t* has_state; // [nseq] or null (every prompt goes on from its state)
  float* S;
  const int32_t* count;
  int32_t* err;
  int prime;
  SketchOut sk;
  void* work;
};

struct CacheParams {
  int B, H, slots, n, bits;
  const int32_t* seqs;      // [n]
  const int32_t* slot;      // [n]
  float* S;
  int32_t* count;
  int32_t* err;
  void* codes;
  float* scale;
  int prime;
  SketchOut sk;
};

struct NormParams {
  const void* x;
  const void* gate;
  void* y;
  const float* weight;
  const float* bias;
  int64_t xs, zs, ys;       // elements from a row to the next
  int64_t rows;
  const int32_t* first;     // rows *first up to *end (null: 0, rows)
  const int32_t* end;
  int groups, width;
  int wgs;                  // elements from a group's weight to the next (0: shared)
  int centred, act, gate_first;
  float eps;
};

// Chunked form: tokens of a chunk, workspace of a chunk and head by activation
// type, and whether the shape has it.
constexpr int PROMPT_CHUNK = 64;
constexpr int PROMPT_CHUNK_WORK = 30 * 1024 + 512;
constexpr int PROMPT_WORK_OVER = 512;    // read, not used, behind the last one
constexpr int PROMPT_CHUNK_WORK_F32 = 20 * 1024 + 512;
inline bool prompt_chunked(int dk) { return dk >= 64; }
inline int prompt_chunk_work(int act) { return act == DT_F32 ? PROMPT_CHUNK_WORK_F32 : PROMPT_CHUNK_WORK; }
// Slots of 2^shift tokens that n prompts of together up to `tokens` tokens may take.
inline int64_t prompt_slots(int64_t tokens, int64_t n, int shift) { return (tokens >> shift) + n; }

int launch_prompt_chunks(int dk, int dv, int act, const PromptParams& p, hipStream_t st);
int launch_prompt_chunks_f32(int dk, int dv, const PromptParams& p, hipStream_t st);
int launch_prompt_step(int dk, int dv, int act, const PromptParams& p, hipStream_t st);
int launch_state_save(int dk, int dv, const CacheParams& p, hipStream_t st);
int launch_state_load(int dk, int dv, int sketch, const CacheParams& p, hipStream_t st);
int launch_group_norm(int dtype, const NormParams& p, hipStream_t st);

}  // namespace sk
