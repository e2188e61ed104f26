// Argument block and launcher of the short causal convolution (sketchssm_conv).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sk_params.hpp"

namespace sk {

constexpr int CONV_PIECES = 3, CONV_MAX_TAPS = 8;

struct ConvParams {
  const void* x;            // [tokens][channels]
  int64_t xs;               // elements from a token's row to the next
  const float* weight;      // [channels][taps]
  const float* bias;        // [channels] or null
  void* state;              // [B][taps - 1][channels]
  int B, channels, act, tokens, nseq;
  int shift;                // prompts are taken in blocks of 2^shift tokens
  const int32_t* start;     // [nseq + 1] or null: a token each
  const int32_t* seqs;      // [nseq] or null
  const int32_t* has_state; // [nseq] or null
  int32_t* err;
  struct Piece {
    void* y;                // [tokens][size] of the channels from `first` on
    int64_t ys;
    int first, size;
    int unit;               // width of the heads brought to unit length (0: none)
    int waves;              // waves that a row of the piece takes
  } piece[CONV_PIECES];
  float eps;
};

int launch_conv(int dtype, int taps, const ConvParams& p, hipStream_t st);

}  // namespace sk
