// Sequences in a new order behind a selection of beams: within each group of
// `beams` consecutive sequences, sequence b becomes a copy of sequence parents[b],
// in place, in every buffer that holds something of a sequence.
//
// Bound by memory: what moves is read once (a parent of several beams comes again
// from the caches) and written once; a beam that stays is not touched.  A lane holds
// the pieces of all beams of its group at one place of a row before it writes any of
// them, so no copy of the states is needed and no order among lanes matters.
#include "sk_beam.hpp"
#include "sk_device.hpp"

namespace sk {
namespace {

constexpr int MOVE_THREADS = 256;

template <typename P, int K>
__device__ __forceinline__ void move(char* data, int64_t bytes, int64_t at, int first, int beams, const int (&from)[K]) {
  if (at >= bytes) return;
  P x[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < beams && from[k] != k) x[k] = *reinterpret_cast<const P*>(data + (int64_t)(first + from[k]) * bytes + at);
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (k < beams && from[k] != k) *reinterpret_cast<P*>(data + (int64_t)(first + k) * bytes + at) = x[k];
}

// One workgroup per (block of a row, group).
template <int K>
__global__ void __launch_bounds__(MOVE_THREADS) reorder_kernel(ReorderParams p) {
  const int g = blockIdx.x / p.blocks, block = blockIdx.x - g * p.blocks, first = g * p.beams;
  int from[K];
  bool wrong = false;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    from[k] = k < p.beams ? p.parents[first + k] - first : k;
    wrong |= from[k] < 0 || from[k] >= (k < p.beams ? p.beams : K);
  }
  if (wrong) {
    if (threadIdx.x == 0 && block == 0) atomicOr(p.err, 4);
    return;
  }
  int r = 0;
  while (r + 1 < p.nrows && block >= p.rows[r + 1].first) ++r;
  const ReorderParams::Rows rows = p.rows[r];
  const int64_t at = ((int64_t)(block - rows.first) * MOVE_THREADS + threadIdx.x) * rows.unit;
  if (rows.unit == 16) move<uint4, K>(rows.data, rows.bytes, at, first, p.beams, from);
  else if (rows.unit == 4) move<uint32_t, K>(rows.data, rows.bytes, at, first, p.beams, from);
  else move<uint16_t, K>(rows.data, rows.bytes, at, first, p.beams, from);
}

}  // namespace

int launch_reorder(const ReorderParams& q, hipStream_t st) {
  ReorderParams p = q;
  int blocks = 0;
  for (int r = 0; r < p.nrows; ++r) {
    p.rows[r].first = blocks;
    blocks += (int)((p.rows[r].bytes / p.rows[r].unit + MOVE_THREADS - 1) / MOVE_THREADS);
  }
  p.blocks = blocks;
  const dim3 grid((unsigned)blocks * p.groups), block(MOVE_THREADS);
  if (p.beams <= 4) hipLaunchKernelGGL((reorder_kernel<4>), grid, block, 0, st, p);
  else if (p.beams <= 8) hipLaunchKernelGGL((reorder_kernel<8>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((reorder_kernel<16>), grid, block, 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sk
