// Sequences in a new order behind a selection of beams: within each group of
// `beams` consecutive sequences, sequence b becomes a copy of sequence parents[b],
// in place, in every buffer that holds something of a sequence.
//
// Bound by memory: what moves is read once (a parent of several beams comes again
// from the caches) and written once; a beam that stays is not touched.  A lane holds
// the pieces of all beams of its group at one place of a row before it writes any of
// them, so no copy of the states is needed and no order among lanes matters.  Loads and
// stores go past the caches: 320 sequences of 128 heads of 128 x 64 in groups of four, a
// random choice of parents, 1.99 GB in 336 us, 5.9 TB/s (through the caches, a beam at a
// time: 376).  Four beams of 32 heads of 128 x 128: 5.4 us.
#include "sk_beam.hpp"
#include "sk_device.hpp"

namespace sk {
namespace {

constexpr int MOVE_THREADS = 256;

// N pieces (a number known here: under a condition for each, the compiler keeps every
// combination in registers of its own).
template <typename P, int K, int N>
__device__ __forceinline__ void move_n(char* data, int64_t bytes, const int (&from)[K], const int (&to)[K]) {
  P x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = __builtin_nontemporal_load(reinterpret_cast<const P*>(data + from[k] * bytes));
#pragma unroll
  for (int k = 0; k < N; ++k) __builtin_nontemporal_store(x[k], reinterpret_cast<P*>(data + to[k] * bytes));
}
template <typename P, int K, int N = K>
__device__ __forceinline__ void move(char* data, int64_t bytes, int n, const int (&from)[K], const int (&to)[K]) {
  if constexpr (N > 0) {
    if (n == N) move_n<P, K, N>(data, bytes, from, to);
    else move<P, K, N - 1>(data, bytes, n, from, to);
  }
}

// One workgroup per (block of a row, group).  What a workgroup needs first, the
// parents and its buffer, is read at once: a request's states alone are a chain of
// reads, and no more.
template <int K>
__global__ void __launch_bounds__(MOVE_THREADS) reorder_kernel(ReorderParams p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int g = blockIdx.x / p.blocks, block = blockIdx.x - g * p.blocks, first = g * p.beams;
  int from[K];
#pragma unroll
  for (int k = 0; k < K; ++k) from[k] = uload(p.parents, first + (k < p.beams ? k : p.beams - 1)) - first;
  int r = -1;                                    // (compared with all at once: no chain of loads)
#pragma unroll
  for (int j = 0; j < MOVE_MAX; ++j) r += j < p.nrows && block >= p.rows[j].first;
  const ReorderParams::Rows rows = p.rows[r];
  // the beams that move, one behind the other
  int src[K], dst[K], n = 0;
  bool wrong = false;
#pragma unroll
  for (int k = 0; k < K; ++k) src[k] = dst[k] = 0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    wrong |= (uint32_t)from[k] >= (uint32_t)p.beams;
    const bool moves = k < p.beams && from[k] != k;
#pragma unroll
    for (int j = 0; j <= k; ++j) {
      const bool here = moves && j == n;
      src[j] = here ? from[k] : src[j];
      dst[j] = here ? k : dst[j];
    }
    n += moves;
  }
  if (wrong) {
    if (threadIdx.x == 0 && block == 0) atomicOr(p.err, 4);
    return;
  }
  const int64_t at = ((int64_t)(block - rows.first) * MOVE_THREADS + threadIdx.x) * rows.unit;
  if (at >= rows.bytes) return;
  char* data = rows.data + (int64_t)first * rows.bytes + at;
  if (rows.unit == 16) move<u32x4, K>(data, rows.bytes, n, src, dst);
  else if (rows.unit == 4) move<uint32_t, K>(data, rows.bytes, n, src, dst);
  else move<uint16_t, K>(data, rows.bytes, n, src, dst);
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
  if (p.beams <= 2) hipLaunchKernelGGL((reorder_kernel<2>), grid, block, 0, st, p);
  else if (p.beams <= 4) hipLaunchKernelGGL((reorder_kernel<4>), grid, block, 0, st, p);
  else if (p.beams <= 8) hipLaunchKernelGGL((reorder_kernel<8>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((reorder_kernel<16>), grid, block, 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sk
