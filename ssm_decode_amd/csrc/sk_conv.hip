// The short causal convolution in front of a layer, over prompts and over single
// tokens:
//   y_t = act(bias + sum_j w_j x_(t - taps + 1 + j)),  j = 0 .. taps - 1,
// channel by channel, where the inputs before a prompt's first are those that its
// sequence holds (zeros where it starts anew), and the last taps - 1 inputs are
// held for the next call.  Heads of queries and keys may be brought to unit
// length on the way, y / sqrt(sum of squares + eps), in 32 bits, rounded once.
//
// Bound by memory: a row in, a row out, and the held inputs once a call.  A lane has 16
// bytes of a row, its weights in registers, and goes from token to token with the last
// inputs in registers, the next two rows in flight (four or eight at once: 1 and 3% slower,
// their registers cost waves); a block of a prompt's tokens reads the taps - 1 rows before
// it again, from the caches.  A wave's channels are of one piece (queries, keys or
// values), so that a head is a whole group of lanes.  Outputs go past the caches: 15715
// tokens of 10240 channels in bf16 135 us, 4.7 TB/s (through them 145).  A decode step of 320
// such tokens 10.2 us, 5.2 TB/s.
#include "sk_act.hpp"
#include "sk_conv.hpp"

namespace sk {
namespace {

constexpr int CONV_THREADS = 256, CONV_WAVES = CONV_THREADS / 64;

// A wave's piece and the lane's first channel in it (false: the wave has none).
__device__ __forceinline__ bool conv_piece(const ConvParams& p, int unit, int n, ConvParams::Piece* pc, int* c) {
  for (int i = 0; i < CONV_PIECES; ++i) {
    if (unit < p.piece[i].waves) {
      *pc = p.piece[i];
      *c = (unit * 64 + (threadIdx.x & 63)) * n;
      return true;
    }
    unit -= p.piece[i].waves;
  }
  return false;
}

// Prompt i and its sequence, checked as prompt_ok does (no rings here): a list
// that falls or leaves [0, tokens] is refused whole, a sequence outside the batch
// or listed before refuses its prompt.
__device__ __forceinline__ bool conv_ok(const ConvParams& p, int i, int b) {
  int wrong = 0;
  for (int j = threadIdx.x; j < p.nseq; j += CONV_THREADS) {
    if (p.start) {
      const int s0 = p.start[j], s1 = p.start[j + 1];
      wrong |= s0 < 0 || s1 < s0 || s1 > p.tokens;
    }
    if (p.seqs && j < i) wrong |= p.seqs[j] == b;
  }
  wrong |= b < 0 || b >= p.B;
  const bool bad = __syncthreads_or(wrong) != 0;
  if (bad && threadIdx.x == 0) atomicOr(p.err, 4);
  return !bad;
}

// The prompt of a slot of 2^shift tokens (sk_prompt_chunk.hpp, first_slot): the
// last whose first slot is not behind it.
__device__ __forceinline__ int conv_prompt(const ConvParams& p, int slot) {
  const int lane = threadIdx.x & 63;
  int i = -1;
  for (int j0 = 0; j0 < p.nseq; j0 += 64) {
    const int j = j0 + lane < p.nseq ? j0 + lane : p.nseq - 1;
    const unsigned long long m = __ballot(j0 + lane < p.nseq && (p.start[j] >> p.shift) + j <= slot);
    if (!m) break;
    i = j0 + 63 - __clzll(m);
  }
  return i;
}

template <typename T, int TAPS>
struct Conv {
  static constexpr int N = Vec<T>::N, H = TAPS - 1;
  float w[TAPS][N], b[N];
  float hist[H][N];

  __device__ __forceinline__ void weights(const ConvParams& p, int c) {
    float all[N * TAPS];
    const float* at = p.weight + (int64_t)c * TAPS;
#pragma unroll
    for (int e = 0; e < N * TAPS; e += 4) {
      float x[4];
      ld4(at + e, x);
#pragma unroll
      for (int f = 0; f < 4; ++f) all[e + f] = x[f];
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
#pragma unroll
      for (int j = 0; j < TAPS; ++j) w[j][e] = all[e * TAPS + j];
#pragma unroll
    for (int e = 0; e < N; ++e) b[e] = 0.f;
    if (p.bias) ldn<N>(p.bias + c, b);
  }
  // The output of the token whose inputs are x; x becomes the newest held.
  __device__ __forceinline__ u32x4 token(const u32x4& raw, int act, int unit, float eps) {
    float x[N], y[N];
    unpack(raw, x);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      y[e] = b[e];
#pragma unroll
      for (int j = 0; j < H; ++j) y[e] = fmaf(w[j][e], hist[j][e], y[e]);
      y[e] = fmaf(w[H][e], x[e], y[e]);
#pragma unroll
      for (int j = 0; j + 1 < H; ++j) hist[j][e] = hist[j + 1][e];
      hist[H - 1][e] = x[e];
      y[e] = activation<T>(y[e], act);
    }
    if (unit) {                                  // (uniform over the wave; whole heads are in or out)
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) s = fmaf(y[e], y[e], s);
      const int lanes = unit / N;
      s = lanes == 2 ? group_sum<2>(s) : lanes == 4 ? group_sum<4>(s) : lanes == 8 ? group_sum<8>(s)
          : lanes == 16 ? group_sum<16>(s) : group_sum<32>(s);
      const float r = 1.f / sqrtf(s + eps);
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] *= r;
    }
    return pack(y);
  }
};

// What a prompt's sequence holds (zeros: it starts anew), 16 bytes a row.
template <typename T, int H>
__device__ __forceinline__ void held_rows(const ConvParams& p, int b, bool read, int c, u32x4 (&raw)[H]) {
  const T* at = reinterpret_cast<const T*>(p.state) + (int64_t)b * H * p.channels + c;
#pragma unroll
  for (int j = 0; j < H; ++j)
    raw[j] = read ? *reinterpret_cast<const u32x4*>(at + (int64_t)j * p.channels) : u32x4{0, 0, 0, 0};
}

// One workgroup per (slot of 2^shift tokens, four waves of channels).  The slot
// with a prompt's first tokens reads what the sequence holds and leaves its last
// inputs there (the same lanes, so that the one is read before the other is
// written); the others take the inputs before their first from x.
template <typename T, int TAPS>
__global__ void __launch_bounds__(CONV_THREADS) conv_prompt_kernel(ConvParams p) {
  using C = Conv<T, TAPS>;
  constexpr int N = C::N, H = C::H, U = 2;
  const int slot = blockIdx.x, i = conv_prompt(p, slot);
  // (a refused list may have no prompt that any slot comes to: it is reported here)
  if (slot == 0 && i != 0) conv_ok(p, 0, p.seqs ? p.seqs[0] : 0);
  if (i < 0) return;
  const int b = p.seqs ? p.seqs[i] : i;
  if (!conv_ok(p, i, b)) return;
  const int s0 = p.start[i], len = p.start[i + 1] - s0;
  const int64_t c0 = (int64_t)(slot - ((s0 >> p.shift) + i)) << p.shift;
  if (c0 >= len && c0 > 0) return;
  ConvParams::Piece pc;
  int cp;
  if (!conv_piece(p, blockIdx.y * CONV_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), N, &pc, &cp) || cp >= pc.size)
    return;
  const int c = pc.first + cp;
  const T* X = reinterpret_cast<const T*>(p.x) + (int64_t)s0 * p.xs + c;
  auto row = [&](int64_t t) { return *reinterpret_cast<const u32x4*>(X + t * p.xs); };
  u32x4 raw[H];
  if (c0 == 0) {
    held_rows<T, H>(p, b, !p.has_state || p.has_state[i] != 0, c, raw);
  } else {
#pragma unroll
    for (int j = 0; j < H; ++j) raw[j] = row(c0 - H + j);
  }
  C k;
  k.weights(p, c);
#pragma unroll
  for (int j = 0; j < H; ++j) unpack(raw[j], k.hist[j]);
  const int64_t end = c0 + (1 << p.shift) < len ? c0 + (1 << p.shift) : len;
  T* Y = reinterpret_cast<T*>(pc.y) + (int64_t)s0 * pc.ys + cp;
  u32x4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) x[u] = c0 + u < end ? row(c0 + u) : u32x4{0, 0, 0, 0};
  for (int64_t t = c0; t < end; t += U) {
    u32x4 now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) now[u] = x[u];
#pragma unroll
    for (int u = 0; u < U; ++u)                  // the next tokens, in flight over these
      if (t + U + u < end) x[u] = row(t + U + u);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + u < end)
        __builtin_nontemporal_store(k.token(now[u], p.act, pc.unit, p.eps), reinterpret_cast<u32x4*>(Y + (t + u) * pc.ys));
  }
  if (c0 == 0) {
    T* S = reinterpret_cast<T*>(p.state) + (int64_t)b * H * p.channels + c;
    u32x4 last[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
      last[j] = u32x4{0, 0, 0, 0};
      if (len - H + j >= 0) {
        last[j] = row(len - H + j);
      } else {                                   // row len + j of what was held
#pragma unroll
        for (int m = j; m < H; ++m)
          if (len + j == m) last[j] = raw[m];
      }
    }
#pragma unroll
    for (int j = 0; j < H; ++j) *reinterpret_cast<u32x4*>(S + (int64_t)j * p.channels) = last[j];
  }
}

// Single tokens: one workgroup per (ROWS tokens, four waves of channels).
template <typename T, int TAPS, int ROWS>
__global__ void __launch_bounds__(CONV_THREADS) conv_step_kernel(ConvParams p) {
  using C = Conv<T, TAPS>;
  constexpr int N = C::N, H = C::H;
  const int i0 = blockIdx.x * ROWS, rows = p.nseq - i0 < ROWS ? p.nseq - i0 : ROWS;
  bool ok[ROWS];
  int seq[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    seq[r] = r < rows ? (p.seqs ? p.seqs[i0 + r] : i0 + r) : 0;
    ok[r] = r < rows && (!p.seqs ? seq[r] < p.B : conv_ok(p, i0 + r, seq[r]));
  }
  ConvParams::Piece pc;
  int cp;
  if (!conv_piece(p, blockIdx.y * CONV_WAVES + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), N, &pc, &cp) || cp >= pc.size)
    return;
  const int c = pc.first + cp;
  u32x4 raw[ROWS][H], x[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (ok[r]) {
      held_rows<T, H>(p, seq[r], !p.has_state || p.has_state[i0 + r] != 0, c, raw[r]);
      x[r] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const T*>(p.x) + (int64_t)(i0 + r) * p.xs + c);
    }
  C k;
  k.weights(p, c);
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (ok[r]) {
#pragma unroll
      for (int j = 0; j < H; ++j) unpack(raw[r][j], k.hist[j]);
      *reinterpret_cast<u32x4*>(reinterpret_cast<T*>(pc.y) + (int64_t)(i0 + r) * pc.ys + cp) =
          k.token(x[r], p.act, pc.unit, p.eps);
      T* S = reinterpret_cast<T*>(p.state) + (int64_t)seq[r] * H * p.channels + c;
#pragma unroll
      for (int j = 0; j < H; ++j) *reinterpret_cast<u32x4*>(S + (int64_t)j * p.channels) = j + 1 < H ? raw[r][j + 1 < H ? j + 1 : j] : x[r];
    }
}

template <typename T, int TAPS>
int launch(ConvParams p, hipStream_t st) {
  int waves = 0;
  for (auto& q : p.piece) {
    q.waves = (q.size + 64 * Vec<T>::N - 1) / (64 * Vec<T>::N);
    waves += q.waves;
  }
  const unsigned parts = (unsigned)(waves + CONV_WAVES - 1) / CONV_WAVES;
  if (p.start) {
    const unsigned slots = (unsigned)((p.tokens >> p.shift) + p.nseq);
    hipLaunchKernelGGL((conv_prompt_kernel<T, TAPS>), dim3(slots, parts), dim3(CONV_THREADS), 0, st, p);
  } else {
    // Four tokens share the weights' loads; where the CUs have few workgroups each has its
    // own: us with one and four, 10240 channels in bf16, of 16 tokens 3.5 and 5.6, of 96
    // 5.6 and 6.5, of 128 7.1 and 6.8, of 320 13.6 and 10.2 (two 11.2, eight 11.1).
    if ((int64_t)p.nseq * parts <= 640) {
      hipLaunchKernelGGL((conv_step_kernel<T, TAPS, 1>), dim3(p.nseq, parts), dim3(CONV_THREADS), 0, st, p);
    } else {
      hipLaunchKernelGGL((conv_step_kernel<T, TAPS, 4>), dim3((unsigned)(p.nseq + 3) / 4, parts), dim3(CONV_THREADS), 0, st, p);
    }
  }
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <typename T>
int launch_type(int taps, const ConvParams& p, hipStream_t st) {
  switch (taps) {
    case 2: return launch<T, 2>(p, st);
    case 3: return launch<T, 3>(p, st);
    case 4: return launch<T, 4>(p, st);
    case 5: return launch<T, 5>(p, st);
    case 6: return launch<T, 6>(p, st);
    case 7: return launch<T, 7>(p, st);
    case 8: return launch<T, 8>(p, st);
    default: return -2;
  }
}

}  // namespace

int launch_conv(int dtype, int taps, const ConvParams& p, hipStream_t st) {
  return dtype == DT_F32 ? launch_type<float>(taps, p, st) : launch_type<bf16>(taps, p, st);
}

}  // namespace sk
