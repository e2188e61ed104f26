// Selection of beams: for each group of `beams` sequences, the best `beams` of
//   score_b + x_bj - log sum_j' exp(x_bj')
// over its beams b and the vocabulary j, in falling order, ties to the lowest
// b * vocab + j.  An ended beam has one candidate, its end token at its own score.
//
// Bound by memory: the logits, once.  One launch takes each row in parts, a part's
// values in registers: their maximum, the sum of their exponentials and the best of
// them, by value (a row's order is that of its values, so no rounding enters it);
// a second joins a group's parts in 64 bits and takes the best of its candidates.
// 320 rows of 128000 bf16 logits: 22 us (3.6 TB/s; half of it vector instructions, the
// exponentials and the search for the best) and 8 us, a chain of reads, of logarithms and of
// one maximum after the other.  Five rows of 50001 fp32 logits: 6 and 7 us.
#include <type_traits>

#include "sk_beam.hpp"
#include "sk_device.hpp"

namespace sk {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
template <typename T> using u32x4_at = std::conditional_t<sizeof(T) == 2, u32x4_at2, u32x4_at4>;

// A value and its index as one number that is larger for the better candidate:
// the value's order above, the lower index above the higher.  (+ 0.f: a negative
// zero is a zero.)
__device__ __forceinline__ uint64_t beam_key(float x, int index) {
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t order = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (uint64_t)order << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t order = (uint32_t)(k >> 32);
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint64_t wave_max(uint64_t k) {
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)k, s);
    k = o > k ? o : k;
  }
  return k;
}
// Largest of the wave's values (a NaN counts for nothing), in every lane.
__device__ __forceinline__ float wave_maxf(float x) {
  x = fmaxf(x, dpp_f<0xB1>(x, x));
  x = fmaxf(x, dpp_f<0x4E>(x, x));
  x = fmaxf(x, dpp_f<0x141>(x, x));
  x = fmaxf(x, dpp_f<0x140>(x, x));
  x = fmaxf(x, dpp_f<0x142, 0xA>(x, x));
  x = fmaxf(x, dpp_f<0x143, 0xC>(x, x));
  return lane_value(x, 63);
}

// The best of a wave's values: those of at least the bound that as many lanes reach
// as there are beams (so the best are among them) are listed, and a listed value's
// place is how many are better (found one by one: 61 us for the 320 rows, not 33).  Only
// where ties make the list too long are they found one by one.
constexpr int LIST = 64;

template <typename T>
__global__ void __launch_bounds__(BEAM_THREADS) beam_part_kernel(BeamParams p) {
  constexpr int N = 16 / (int)sizeof(T), E = BEAM_VALUES, V = E / N;      // values of a vector, of a lane; vectors
  __shared__ uint64_t s_list[4][LIST], s_key[4 * BEAM_MAX];
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  if (p.ended && p.ended[row] != 0) return;
  const T* X = reinterpret_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  // Rows of any length begin anywhere.  A value's lane goes by its index, not by its
  // address, so that equal rows have equal sums (or equal beams would be no ties): the
  // vectors are at the alignment of an element.
  const int first = part * BEAM_PART;
  float x[E];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int at = first + (v * BEAM_THREADS + tid) * N;
    if (at + N <= p.vocab) {
      const u32x4 w = *reinterpret_cast<const u32x4_at<T>*>(X + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          x[v * N + 2 * e] = __uint_as_float(w[e] << 16);
          x[v * N + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        } else {
          x[v * N + e] = __uint_as_float(w[e]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x[v * N + e] = at + e < p.vocab ? ld(X + at + e) : -__builtin_inff();
    }
  }
  constexpr float NONE = -__builtin_inff();
  float mine = NONE;
#pragma unroll
  for (int e = 0; e < E; ++e) mine = fmaxf(mine, x[e]);
  const float top = wave_maxf(mine);
  // Exponentials by the instruction, of differences to the maximum: off by 2^-24 of the
  // exponent's magnitude, and where that is large the term is small.  (A NaN, or an
  // infinity as the maximum, makes the sum a NaN; ruled out values add nothing.)
  float sum = 0.f;
  if (top != NONE) {
#pragma unroll
    for (int e = 0; e < E; ++e) sum += __builtin_amdgcn_exp2f((x[e] - top) * 1.44269504f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) sum += x[e] == NONE ? 0.f : x[e];      // (a NaN among ruled out values)
  }
  sum = wave_sum(sum);
  BeamPart* out = p.part + (int64_t)row * p.parts + part;
  if (lane == 0) {
    out->top[wv] = top;
    out->sum[wv] = sum;
  }
  auto index = [&](int e) { return first + ((e / N) * BEAM_THREADS + tid) * N + e % N; };
  if (lane < p.beams) s_key[wv * BEAM_MAX + lane] = 0;
  wave_lds_sync();
  // the bound: lanes' maxima in falling order until as many lanes as beams have one
  float bound = top, rest = mine;
  for (int n = 0;;) {
    const bool it = rest == bound && bound > NONE;
    n += __popcll(__ballot(it));
    if (n >= p.beams) break;
    rest = it ? NONE : rest;
    const float next = wave_maxf(rest);
    if (!(next > NONE)) {                        // (fewer lanes have any: all that they have)
      bound = bound > NONE ? -3.402823466e38f : NONE;
      break;
    }
    bound = next;
  }
  int listed = 0;
  const unsigned long long below = (1ull << lane) - 1;
  if (bound > NONE) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool it = x[e] >= bound;
      const unsigned long long m = __ballot(it);
      if (m) {
        const int at = listed + __popcll(m & below);
        if (it && at < LIST) s_list[wv][at] = beam_key(x[e], index(e));
        listed += __popcll(m);
      }
    }
  }
  wave_lds_sync();
  if (listed <= LIST) {
    const uint64_t k = lane < listed ? s_list[wv][lane] : 0;
    int place = 0;
    for (int j = 0; j < listed; j += 8)          // (eight reads at once: LIST is a multiple of it)
#pragma unroll
      for (int e = 0; e < 8; ++e) place += s_list[wv][j + e] > k && j + e < listed;
    if (lane < listed && place < p.beams) s_key[wv * BEAM_MAX + place] = k;
  } else {
    uint64_t last = ~0ull;
    for (int r = 0; r < p.beams; ++r) {          // the best of what is worse than the last
      uint64_t best = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint64_t k = x[e] > NONE ? beam_key(x[e], index(e)) : 0;
        best = k < last && k > best ? k : best;
      }
      last = wave_max(best);
      if (lane == 0) s_key[wv * BEAM_MAX + r] = last;
      if (last == 0) break;                      // (none is left)
    }
  }
  __syncthreads();
  if (wv == 0) {                                 // the best of the waves'
    const bool mine = lane % BEAM_MAX < p.beams;
    const uint64_t k = mine ? s_key[lane] : 0;
    int place = 0;
    for (int r = 0; r < p.beams; ++r)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint64_t o = s_key[w * BEAM_MAX + r];
        place += o > k || (o == k && w * BEAM_MAX + r < lane);
      }
    if (mine && place < p.beams) {
      out->value[place] = k ? key_value(k) : NONE;
      out->index[place] = key_index(k);
    }
  }
}

// The wave's largest value, in every lane.
__device__ __forceinline__ double wave_maxd(double x) {
  auto with = [](double v, auto ctrl, auto mask) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
    const uint32_t l = __builtin_amdgcn_update_dpp(lo, lo, decltype(ctrl)::value, decltype(mask)::value, 0xF, false);
    const uint32_t h = __builtin_amdgcn_update_dpp(hi, hi, decltype(ctrl)::value, decltype(mask)::value, 0xF, false);
    return fmax(v, __builtin_bit_cast(double, (uint64_t)h << 32 | l));
  };
  typedef std::integral_constant<int, 0xF> All;
  x = with(x, std::integral_constant<int, 0xB1>{}, All{});
  x = with(x, std::integral_constant<int, 0x4E>{}, All{});
  x = with(x, std::integral_constant<int, 0x141>{}, All{});
  x = with(x, std::integral_constant<int, 0x140>{}, All{});
  x = with(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
  x = with(x, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The wave's best of what its lanes offer, lane by lane, `take` of them at most, in
// falling order, ties to the lower place: got(n, score, at) for each, and next(&score,
// &at) in the lane whose offer it was.
constexpr double NO_SCORE = -__builtin_inf();
template <typename Got, typename Next>
__device__ __forceinline__ void wave_best(int take, double score, int at, Got got, Next next) {
  const int lane = threadIdx.x & 63;
  for (int n = 0; n < take; ++n) {
    const double top = wave_maxd(score);
    if (!(top > NO_SCORE)) return;
    unsigned long long m = __ballot(score == top);
    int who = __builtin_ctzll(m), best = __builtin_amdgcn_readlane(at, who);
    while (m &= m - 1) {                         // (a tie)
      const int other = __builtin_ctzll(m), a = __builtin_amdgcn_readlane(at, other);
      if (a < best) {
        best = a;
        who = other;
      }
    }
    if (lane == who) {
      got(n, top, best);
      next(&score, &at);
    }
  }
}

// One workgroup per group.  (Places b * vocab + j are below 16 * 2^24.)
// JOIN_CHAIN: up to as many beams the best are taken one by one, more from a list: 16
// groups over 128000 bf16 logits, both launches, 14 and 22 us with 4 beams, 29 and 33 with
// 8, 42 and 40 with 10, 86 and 79 with 16.
constexpr int JOIN_LIST = 256, JOIN_CHAIN = 8;
// HELD: a lane's candidates that are read at once with the rows' sums: k of each part
// of a row (an ended row's only one is its first; k: none).  (Those beyond are read again
// for each that is taken: with four 16 groups of 16 beams 229 us.)
template <int HELD>
__global__ void __launch_bounds__(BEAM_THREADS) beam_join_kernel(BeamParams p) {
  __shared__ double s_lse[BEAM_MAX], s_score[4 * BEAM_MAX], s_out[BEAM_MAX];
  __shared__ float s_in[BEAM_MAX];
  __shared__ int s_ended[BEAM_MAX], s_at[4 * BEAM_MAX], s_pick[BEAM_MAX];
  __shared__ double s_list[4][JOIN_LIST];
  __shared__ int s_place[4][JOIN_LIST];
  const int g = blockIdx.x, k = p.beams, tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  constexpr int FAR = INT32_MAX;
  const int per = p.parts * k, all = per * k;
  // (c < 2^20: the quotients' errors are less than the half)
  const float by_per = 1.f / per, by_k = 1.f / k;
  auto candidate = [&](int c, int* b, float* v, int* a) {
    *b = (int)((c + 0.5f) * by_per);
    const int j = c - *b * per, row = g * k + *b, x = (int)((j + 0.5f) * by_k);
    const bool ended = p.ended && p.ended[row] != 0;
    const BeamPart* part = p.part + (int64_t)row * p.parts + x;
    *v = part->value[j - x * k];
    *a = *b * p.vocab + part->index[j - x * k];
    if (ended) {
      *v = 0.f;
      *a = *b * p.vocab + (p.end_token > 0 ? p.end_token : 0);
      if (j > 0) *b = k;
    }
  };
  float hv[HELD];
  int hb[HELD], ha[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    hb[i] = k;
    ha[i] = FAR;
    const int c = tid + i * BEAM_THREADS;
    if (c < all) candidate(c, &hb[i], &hv[i], &ha[i]);
  }
  if (tid < 4 * BEAM_MAX) {
    s_score[tid] = NO_SCORE;
    s_at[tid] = FAR;
  }
  if (tid < BEAM_MAX) s_pick[tid] = FAR;
  // the rows' sums: a wave a row, or 16 lanes where there are more rows than waves
  auto row_sums = [&](auto lanes) {
    constexpr int LANES = decltype(lanes)::value;
    const int b = tid / LANES, first = tid % LANES;
    if (b >= k) return;                          // (whole groups of lanes)
    const int row = g * k + b;
    const float in = p.scores[row];
    const bool ended = p.ended && p.ended[row] != 0;
    const BeamPart* part = p.part + (int64_t)row * p.parts;
    const int n = ended ? 0 : 4 * p.parts;
    float top = -__builtin_inff();
#pragma unroll 4
    for (int j = first; j < n; j += LANES) top = fmaxf(top, part[j >> 2].top[j & 3]);
#pragma unroll
    for (int s = 1; s < LANES; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
    double sum = 0;
#pragma unroll 4
    for (int j = first; j < n; j += LANES) {
      const float t = part[j >> 2].top[j & 3], s = part[j >> 2].sum[j & 3];
      sum += s == 0.f ? 0. : exp((double)t - top) * s;
    }
#pragma unroll
    for (int s = 1; s < LANES; s *= 2) sum += __shfl_xor(sum, s);
    if (first == 0) {
      // a row without a finite sum, and a score that is none, take the beam out; all
      // ruled out is no error
      const bool wrong = !(fabs(sum) < __builtin_inf()) || in != in || in == __builtin_inff();
      if (wrong) atomicOr(p.err, ERRBIT_LOGIT);
      s_in[b] = wrong ? -__builtin_inff() : in;
      s_ended[b] = ended;
      s_lse[b] = (double)top + log(sum);
    }
  };
  if (k <= 4) row_sums(std::integral_constant<int, 64>{});
  else row_sums(std::integral_constant<int, 16>{});
  __syncthreads();
  // candidates, k of each part of a row
  auto rate = [&](int b, float v) -> double {
    const float in = s_in[b];
    if (s_ended[b]) return in;
    return in > -__builtin_inf() && v > -__builtin_inf() ? (double)in + ((double)v - s_lse[b]) : NO_SCORE;
  };
  double hs[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) hs[i] = hb[i] < k ? rate(hb[i], hv[i]) : NO_SCORE;
  // (where a row has more parts than lanes hold candidates of, the others are read again)
  auto further = [&](int c, int* a) -> double {
    int b;
    float v;
    candidate(c, &b, &v, a);
    return b < k ? rate(b, v) : NO_SCORE;
  };
  // A wave's best, as the parts': those of at least the bound that as many lanes reach as
  // there are beams are listed, and a listed one's place is how many are better.
  int listed = JOIN_LIST + 1;
  if (k > JOIN_CHAIN) {
    double mine = NO_SCORE;
  #pragma unroll
    for (int i = 0; i < HELD; ++i) mine = fmax(mine, hs[i]);
    for (int c = tid + HELD * BEAM_THREADS, a; c < all; c += BEAM_THREADS) mine = fmax(mine, further(c, &a));
    s_list[wv][lane] = mine;
    wave_lds_sync();
    int place = 0;
  #pragma unroll 16
    for (int j = 0; j < 64; ++j) {
      const double o = s_list[wv][j];
      place += o > mine || (o == mine && j < lane);
    }
    const double bound = s_list[wv][__builtin_ctzll(__ballot(place == k - 1))];
    wave_lds_sync();
    listed = 0;
    auto list = [&](double score, int a) {
      const bool it = score > NO_SCORE && score >= bound;
      const unsigned long long m = __ballot(it);
      const int to = listed + __popcll(m & ((1ull << lane) - 1));
      if (it && to < JOIN_LIST) {
        s_list[wv][to] = score;
        s_place[wv][to] = a;
      }
      listed += __popcll(m);
    };
  #pragma unroll
    for (int i = 0; i < HELD; ++i) list(hs[i], ha[i]);
    for (int c = tid + HELD * BEAM_THREADS; c - tid < all; c += BEAM_THREADS) {
      int a = FAR;
      const double score = c < all ? further(c, &a) : NO_SCORE;
      list(score, a);
    }
    wave_lds_sync();
  }
  if (listed <= JOIN_LIST) {
    for (int e = lane; e < listed; e += 64) {
      const double score = s_list[wv][e];
      const int a = s_place[wv][e];
      int better = 0;
      for (int j = 0; j < listed; j += 8)
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          const double o = s_list[wv][j + f];
          better += (o > score || (o == score && s_place[wv][j + f] < a)) && j + f < listed;
        }
      if (better < k) {
        s_score[wv * BEAM_MAX + better] = score;
        s_at[wv * BEAM_MAX + better] = a;
      }
    }
  } else {                                       // (one by one)
    auto offer = [&](double* score, int* at) {   // the lane's best behind the last that was taken
      const double last = *score;
      const int last_at = *at;
      double best = NO_SCORE;
      int best_at = FAR;
      auto consider = [&](double x, int a) {
        const bool behind = x < last || (x == last && a > last_at);
        if (behind && (x > best || (x == best && a < best_at))) {
          best = x;
          best_at = a;
        }
      };
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (hb[i] < k) consider(hs[i], ha[i]);
      for (int c = tid + HELD * BEAM_THREADS; c < all; c += BEAM_THREADS) {
        int a;
        const double x = further(c, &a);
        consider(x, a);
      }
      *score = best;
      *at = best_at;
    };
    double score = __builtin_inf();
    int at = -1;
    offer(&score, &at);
    wave_best(k, score, at,
              [&](int n, double x, int a) {
                s_score[wv * BEAM_MAX + n] = x;
                s_at[wv * BEAM_MAX + n] = a;
              },
              offer);
  }
  __syncthreads();
  if (wv > 0) return;
  if (k > JOIN_CHAIN) {                          // the best of the waves'
    const double score = s_score[lane];
    const int a = s_at[lane];
    int better = 0;
#pragma unroll 16
    for (int j = 0; j < 4 * BEAM_MAX; ++j) better += s_score[j] > score || (s_score[j] == score && s_at[j] < a);
    if (score > NO_SCORE && better < k) {
      s_out[better] = score;
      s_pick[better] = a;
    }
  } else {
    wave_best(k, s_score[lane], s_at[lane],
              [&](int n, double x, int a) {
                s_out[n] = x;
                s_pick[n] = a;
              },
              [](double* x, int*) { *x = NO_SCORE; });
  }
  wave_lds_sync();
  if (lane < k) {
    const int row = g * k + lane, pick = s_pick[lane];
    const bool none = pick == FAR;
    const int b = none ? lane : pick / p.vocab;
    const bool over = !none && s_ended[b];
    const int token = none ? -1 : over ? p.end_token : pick % p.vocab;
    p.parents[row] = g * k + b;
    p.tokens[row] = token;
    p.new_scores[row] = none ? -__builtin_inff() : (float)s_out[lane];
    p.new_ended[row] = over || (!none && token == p.end_token);
  }
}

}  // namespace

int launch_beam_select(int dtype, const BeamParams& p, hipStream_t st) {
  const dim3 grid((unsigned)p.parts * p.groups * p.beams), block(BEAM_THREADS);
  if (dtype == DT_F32) hipLaunchKernelGGL((beam_part_kernel<float>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((beam_part_kernel<bf16>), grid, block, 0, st, p);
  if (p.parts * p.beams * p.beams <= 4 * BEAM_THREADS)
    hipLaunchKernelGGL((beam_join_kernel<4>), dim3((unsigned)p.groups), block, 0, st, p);
  else
    hipLaunchKernelGGL((beam_join_kernel<16>), dim3((unsigned)p.groups), block, 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace sk
