// Prompts through the selective state space scan in chunks of 64 tokens.  With
// l_t = -dt_t exp(A_h), L_i the sum of a chunk's l up to token i, and S_0 the state
// before the chunk:
//   P_ij = exp(L_i - L_j) dt_j (q_i . k_j)   for j <= i, 0 above
//   O = diag(exp L) Q S_0 + P V
//   S = exp(L_C) S_0 + K^T diag(exp(L_C - L_j) dt_j) V
// The sums L run in 64 bits, so that a difference of two is that of the tokens
// between them, whatever came before; decays are exponentials of differences of the
// right sign, so no quotient overflows.
//
// Precision.  The state is fp32, and so is every product.  They run on the bf16 matrix
// cores with each fp32 operand (S_0, P, the weighted V) as an exact sum of three
// bf16 values, so a product with bf16 data (Q, V, K^T) takes three instructions.
//
// Layout.  A wave has 64 columns of one head's state, all rows, in registers, and a
// workgroup up to eight waves of one group, whose keys and queries it shares: K and Q
// are in LDS twice (the next chunk's copy, straight from memory, is in flight over
// the present one), the triangle of K Q^T is formed once a chunk by all waves, and V,
// which is a wave's own, comes through registers one chunk ahead.  All products are
// the transposed ones, so that a lane's results are runs of columns of one token.
#include <type_traits>

#include "sk_prompt_chunk.hpp"
#include "sk_scan.hpp"

namespace sk {
namespace {

constexpr int NCB = SCAN_COLS / 16;              // 16-column tiles of a wave
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <int DK, bool OUT>
struct ScanLds {
  static constexpr int K = 0;                    // [2][64][DK]
  static constexpr int Q = K + 2 * PC * DK * 2;
  static constexpr int QK = Q + (OUT ? 2 * PC * DK * 2 : 0);      // six fragments of K Q^T in fp32
  static constexpr int V = QK + (OUT ? FRAGS * 2 * FRAG_BYTES : 0);
  static constexpr int V_BYTES = PC * SCAN_COLS * 2, F_BYTES = 6 * PC * 4;
  static constexpr int bytes(int waves) { return V + waves * (V_BYTES + F_BYTES); }
};

// Sum of the lanes up to this one, in 64 bits.
__device__ __forceinline__ double wave_prefix(double x) {
  auto from = [](double v, auto ctrl, auto mask) {
    constexpr int C = decltype(ctrl)::value, M = decltype(mask)::value;
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, C, M, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), C, M, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  typedef std::integral_constant<int, 0xF> All;
  x += from(x, std::integral_constant<int, 0x111>{}, All{});      // row_shr:1, 2, 4, 8
  x += from(x, std::integral_constant<int, 0x112>{}, All{});
  x += from(x, std::integral_constant<int, 0x114>{}, All{});
  x += from(x, std::integral_constant<int, 0x118>{}, All{});
  x += from(x, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});      // row_bcast:15, 31
  x += from(x, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
  return x;
}
// Lane 63's value in every lane.
__device__ __forceinline__ double wave_last(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// 2^x in fp32 of an exponent in 64 bits: of what rounding it leaves, to first order.
__device__ __forceinline__ float exp2_of(double x) {
  const float f = (float)x, e = __builtin_amdgcn_exp2f(f);
  return fmaf(e, (float)(x - (double)f) * 0.693147182f, e);
}

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ const void* uniform(const void* x) {
  const uint64_t u = reinterpret_cast<uint64_t>(x);
  return reinterpret_cast<const void*>((uint64_t)uniform((uint32_t)(u >> 32)) << 32 | uniform((uint32_t)u));
}

// Fragment f of the triangle: rows (tokens i) 16 rb .., columns (tokens j) 32 kh ..
__device__ __forceinline__ constexpr int frag_rb(int f) { return f < 2 ? f : 2 + (f - 2) / 2; }
__device__ __forceinline__ constexpr int frag_kh(int f) { return f < 2 ? 0 : (f - 2) & 1; }
constexpr int frag_of(int rb, int kh) { return rb < 2 ? rb : 2 + 2 * (rb - 2) + kh; }

// One workgroup per (segment or prompt, group, part of its heads).  Where prompts are
// cut into segments of 2^seg_shift tokens, three launches take the place of one:
//   1. without outputs, the segments but the last, at once: each from a zero state
//      (the first from the prompt's) its state behind it, B, and the product g of
//      its decays: the state behind a segment is g S + B;
//   2. scan_join_kernel: the states between the segments, in order;
//   3. the segments at once, each from the state before it, with outputs.
// The first segment leaves the state that the prompt starts from in the last one's
// place, which has no use for it: the prompt's own place is written by the third
// launch's last segment, maybe before its first one reads.
template <int DK, int DV, bool OUT>
__global__ void __launch_bounds__(64 * SCAN_WAVES, 2) scan_chunk_kernel(ScanParams p) {
  using L = ScanLds<DK, OUT>;
  constexpr int PPR = DK / 8, DB = DK / 32, UPH = DV / SCAN_COLS, UNIT = DK * SCAN_COLS;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6), NW = p.waves;
  const int n = lane & 15, hi = lane >> 4;
  // (the parts of a group are eight workgroups apart: on one XCD at one time)
  const int part = blockIdx.x / 8 % p.parts, tile = blockIdx.x / (8 * p.parts) * 8 + blockIdx.x % 8;
  const int g = tile % p.G, slot = tile / p.G, E = p.H / p.G;
  if (slot >= (p.seg_shift ? p.nsegs : p.nchunked)) return;
  // (a refused list may have no prompt that any launch comes to: it is reported here)
  if (slot == 0 && prompt_wrong(p, 0, p.seqs ? p.seqs[0] : 0) && tid == 0) atomicOr(p.err, ERRBIT_SEQ);
  int rank = 0, seg = 0;
  const int i = p.seg_shift ? slot_prompt(p, slot, p.seg_shift, &rank) : chunked_prompt(p, slot, &rank);
  if (i < 0) return;
  int s0 = p.start[i], len = p.start[i + 1] - s0, slots = 1;
  const int b = p.seqs ? p.seqs[i] : i;
  if (p.seg_shift) {
    seg = slot - first_slot(s0, rank, p.seg_shift);
    const int64_t from = (int64_t)seg << p.seg_shift;
    if (from >= len && seg > 0) return;
    slots = (int)(((int64_t)len + (1 << p.seg_shift) - 1) >> p.seg_shift);
    s0 += (int)from;
    len = len - from <= (1 << p.seg_shift) ? len - (int)from : 1 << p.seg_shift;
  }
  const bool last = seg + 1 >= slots;
  if (!OUT && last) return;
  if (const int bad = prompt_wrong(p, i, b)) {
    if (tid == 0) atomicOr(p.err, bad);
    return;
  }
  const int u = part * NW + wv;                  // the wave's unit of the group: head and columns
  const int h = __builtin_amdgcn_readfirstlane(g * E + (u < E * UPH ? u / UPH : 0)), c0 = u % UPH * SCAN_COLS;
  bool active = u < E * UPH;
  if (active && p.count[(size_t)b * p.H + h] != 0) {
    if (lane == 0) atomicOr(p.err, (int)ERRBIT_COUNT);
    active = false;
  }

  // ------------------------------------------------------------- copies
  const bf16* kp = reinterpret_cast<const bf16*>(p.k) + (int64_t)s0 * p.ks + (int64_t)g * DK;
  const bf16* qp = reinterpret_cast<const bf16*>(p.q) + (int64_t)s0 * p.qs + (int64_t)g * DK;
  const bf16* vp = reinterpret_cast<const bf16*>(p.v) + (int64_t)s0 * p.vs + (int64_t)h * DV + c0;
  const bf16* dp = reinterpret_cast<const bf16*>(p.gate) + (int64_t)s0 * p.gs + h;
  // Rows have their 16-byte pieces swizzled so that those of a fragment spread over
  // the banks: piece pc of a row of 16 (K, Q; DK = 64: 8, as V) is at pc ^ swz(row).
  auto swz = [](int row, int ppr) {
    const int s = (row & 3) | ((row >> 1) & 12);
    return (ppr == 16 ? s : s >> 1) & (ppr - 1);
  };
  const uint32_t lds0 = lds_address(smem);
  // K and Q of a chunk of nt tokens into buffer buf (rows behind the end repeat the
  // last one: their weights are zeros, and what they give is not stored)
  auto copy = [&](int t0, int nt, int buf) {
    for (int c = wv; c < PPR; c += NW) {
      const int at = c * 64 + lane, row = at / PPR, pc = (at % PPR) ^ swz(row, PPR), r = row < nt ? row : nt - 1;
      const uint32_t to = lds0 + buf * PC * DK * 2 + c * 1024;
      copy16(uniform(kp + (int64_t)t0 * p.ks), (uint32_t)(r * p.ks * 2) + pc * 16, uniform(to + L::K));
      if (OUT) copy16(uniform(qp + (int64_t)t0 * p.qs), (uint32_t)(r * p.qs * 2) + pc * 16, uniform(to + L::Q));
    }
  };
  unsigned char* s_v = smem + L::V + wv * (L::V_BYTES + L::F_BYTES);
  float* s_f = reinterpret_cast<float*>(s_v + L::V_BYTES);      // L (upper and lower part), dt, weight, exp L, first wrong tokens
  u32x4 vr[8];
  float dr = 0.f;
  const uint32_t vo = (uint32_t)((lane >> 3) * p.vs * 2) + (lane & 7) * 16;
  // V, eight rows at a time, and dt, a token a lane.  Rows behind the end repeat the
  // last one: their dt is 0.
  auto fetch = [&](int t0, int nt) {
    const unsigned char* from = reinterpret_cast<const unsigned char*>(vp + (int64_t)t0 * p.vs);
    if (nt == PC) {
#pragma unroll
      for (int v = 0; v < 8; ++v) vr[v] = *reinterpret_cast<const u32x4*>(from + (int64_t)(16 * v) * p.vs + vo);
    } else {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const int row = 8 * v + (lane >> 3), r = row < nt ? row : nt - 1;
        vr[v] = *reinterpret_cast<const u32x4*>(from + (uint32_t)(r * p.vs * 2) + (lane & 7) * 16);
      }
    }
    const int r = lane < nt ? lane : nt - 1;
    dr = to_f32(*reinterpret_cast<const bf16*>(reinterpret_cast<const unsigned char*>(dp + (int64_t)t0 * p.gs) + (uint32_t)(r * p.gs * 2)));
    dr = lane < nt ? dr : 0.f;
  };

  // -------------------------------------------------------------- state
  f32x4s S[DB][NCB][2];                          // rows 32 kb + 8 hi + 4 e + r of column (tile cb, lane n)
  auto col = [&](int cb) { return 32 * (cb >> 1) + block_row(n, cb & 1); };
  float* Sg = p.S + ((size_t)b * p.H + h) * DK * DV + c0;
  auto seg_at = [&](int s) { return reinterpret_cast<f32x4s*>(p.seg + (((size_t)s * p.H + h) * UPH + c0 / SCAN_COLS) * UNIT) + lane; };
  auto each = [&](auto f) {
#pragma unroll
    for (int kb = 0; kb < DB; ++kb)
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
        for (int e = 0; e < 2; ++e) f(kb, cb, e);
  };
  each([&](int kb, int cb, int e) { S[kb][cb][e] = f32x4s{0.f, 0.f, 0.f, 0.f}; });
  if (active) {
    if (seg == 0 && !(OUT && !last)) {
      if (!p.has_state || p.has_state[i] != 0)
        each([&](int kb, int cb, int e) {
#pragma unroll
          for (int r = 0; r < 4; ++r) S[kb][cb][e][r] = Sg[(size_t)(32 * kb + 8 * hi + 4 * e + r) * DV + col(cb)];
        });
      if (!OUT) {
        f32x4s* to = seg_at(slot + slots - 1);
        each([&](int kb, int cb, int e) { to[((kb * NCB + cb) * 2 + e) * 64] = S[kb][cb][e]; });
      }
    } else if (OUT) {
      const f32x4s* from = seg_at(seg == 0 ? slot + slots - 1 : slot - 1);
      each([&](int kb, int cb, int e) { S[kb][cb][e] = from[((kb * NCB + cb) * 2 + e) * 64]; });
    }
    if (len > 0) fetch(0, len < PC ? len : PC);
  }
  if (len > 0) copy(0, len < PC ? len : PC, 0);
  const double rate = exp((double)p.A[h]) * -1.4426950408889634;
  double total = 0.;

  bf16* op = reinterpret_cast<bf16*>(p.o) + (int64_t)s0 * p.os + (int64_t)h * DV + c0;
  const uint32_t oo = (uint32_t)(n * p.os * 2) + hi * 16;

  // Byte addresses of a lane's fragments.  A fragment's rows differ by whole multiples
  // of what the swizzle looks at, or by such that change one bit of it, so that a few
  // registers and constant offsets cover all of them (checked below, at compile time).
  const int ti = n >> 2;
  constexpr int ROW = DK * 2;
  //  rows 16 rb + n of Q, piece 4 kb + hi: at kq[kb ^ swizzle bits of rb] + 16 rb ROW
  //  rows 32 kh + block_row(n, t) of K, piece 4 kb + hi: at kk[kb] + (32 kh + 4 t) ROW
  //  K^T, rows 32 kh + 8 hi + ti (+ 4), columns 32 db + 8 (n & 3) + 4 t: at kt[db] + (32 kh (+ 4)) ROW + 8 t
  //  V, rows as K^T's, columns 32 cp + 8 (n & 3) + 4 t: at va[cp] + (32 kh (+ 4)) 128 + 8 t
  int kq[DB], kk[DB], kt[DB], va[NCB / 2];
#pragma unroll
  for (int kb = 0; kb < DB; ++kb) {
    kq[kb] = n * ROW + ((4 * kb + hi) ^ swz(n, PPR)) * 16;
    kk[kb] = block_row(n, 0) * ROW + ((4 * kb + hi) ^ swz(block_row(n, 0), PPR)) * 16;
    kt[kb] = (8 * hi + ti) * ROW + ((4 * kb + (n & 3)) ^ swz(8 * hi + ti, PPR)) * 16;
  }
#pragma unroll
  for (int cp = 0; cp < NCB / 2; ++cp) va[cp] = (8 * hi + ti) * 128 + ((4 * cp + (n & 3)) ^ swz(8 * hi + ti, 8)) * 16;
  // rows of another rb: bits of the piece's number that the swizzle turns over
  constexpr int FLIP = PPR == 16 ? 2 : 1;
  auto frag_q = [&](const unsigned char* s, int rb, int kb) {
    return as_frag(*reinterpret_cast<const u32x4*>(s + kq[kb ^ (rb & 1) * FLIP] + 16 * rb * ROW));
  };
  auto frag_k = [&](const unsigned char* s, int kh, int t, int kb) {
    return as_frag(*reinterpret_cast<const u32x4*>(s + kk[kb] + (32 * kh + 4 * t) * ROW));
  };
  auto frag_kt = [&](const unsigned char* s, int db, int t, int kh) {
    const unsigned char* at = s + kt[db] + 32 * kh * ROW + 8 * t;
    return join(read_tr(at), read_tr(at + 4 * ROW));
  };
  // V^T (or V): columns of tile cb, tokens 32 kh + 8 hi ..
  auto frag_v = [&](int cb, int kh) {
    const unsigned char* at = s_v + va[cb >> 1] + 32 * kh * 128 + 8 * (cb & 1);
    return join(read_tr(at), read_tr(at + 4 * 128));
  };

  int buf = 0;
  for (int t0 = 0; t0 < len; t0 += PC, buf ^= 1) {
    const int nt = len - t0 < PC ? len - t0 : PC, left = len - t0 - PC;
    // the chunk's decays, a token a lane: L split so that a difference of two is exact
    // to fp32 (a decay of less than 2^-256 a token is zero)
    float decay = 0.f;
    bool wrong = false;
    if (active) {
      double l = (double)dr * rate;
      l = l < -256. ? -256. : l;
      const double at = wave_prefix(l), end = wave_last(at);
      const double hid = (at + 0x1.8p42) - 0x1.8p42;      // a multiple of 2^-10, |L| <= 2^14
      s_f[lane] = (float)hid;
      s_f[PC + lane] = (float)(at - hid);
      s_f[2 * PC + lane] = dr;
      s_f[3 * PC + lane] = exp2_of(end - at) * dr;
      s_f[4 * PC + lane] = exp2_of(at);
      decay = exp2_of(end);
      total += end;
      uint32_t top = 0;                          // the largest magnitudes, two values at a time
#pragma unroll
      for (int v = 0; v < 8; ++v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const u16x2 a = __builtin_bit_cast(u16x2, vr[v][e] & 0x7fff7fffu), m = __builtin_bit_cast(u16x2, top);
          top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, m));
        }
        const int row = 8 * v + (lane >> 3);
        *reinterpret_cast<u32x4*>(s_v + row * 128 + ((lane & 7) ^ swz(row, 8)) * 16) = vr[v];
      }
      wrong = OUT && __any((top & 0xffffu) >= 0x7f80u || top >= 0x7f800000u);
    }
    // this wave's copies for the chunk have landed, then everybody's; and
    // everybody has read the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (left > 0) copy(t0 + PC, left < PC ? left : PC, buf ^ 1);
    const unsigned char *s_k = smem + L::K + buf * PC * DK * 2, *s_q = smem + L::Q + buf * PC * DK * 2;

    if constexpr (OUT) {
      // the triangle of K Q^T: tile t of fragment f, rows j, columns i
      for (int c = wv; c < 2 * FRAGS; c += NW) {
        const int f = c >> 1, t = c & 1, rb = frag_rb(f), kh = frag_kh(f);
        const bool flip = (rb & 1) != 0;
        f32x4s a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < DB; ++kb)
          a = mm32(frag_k(s_k, kh, t, kb),
                   as_frag(*reinterpret_cast<const u32x4*>(s_q + (flip ? kq[kb ^ FLIP] : kq[kb]) + 16 * rb * ROW)), a);
        reinterpret_cast<f32x4s*>(smem + L::QK)[c * 64 + lane] = a;
      }
      __syncthreads();
      if (active) {
        f32x4s O[4][NCB];                        // columns 4 hi + r of tile cb, token 16 rb + n
#pragma unroll
        for (int rb = 0; rb < 4; ++rb)
#pragma unroll
          for (int cb = 0; cb < NCB; ++cb) O[rb][cb] = f32x4s{0.f, 0.f, 0.f, 0.f};
        // O = (Q S)^T
#pragma unroll
        for (int kb = 0; kb < DB; ++kb) {
          bf16x8 fq[4];
#pragma unroll
          for (int rb = 0; rb < 4; ++rb) fq[rb] = frag_q(s_q, rb, kb);
#pragma unroll
          for (int cb = 0; cb < NCB; ++cb) {
            float x[8];
            bf16x8 ss[3];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = S[kb][cb][e >> 2][e & 3];
            split8(x, ss);
#pragma unroll
            for (int v = 2; v >= 0; --v)
#pragma unroll
              for (int rb = 0; rb < 4; ++rb) O[rb][cb] = mm32(ss[v], fq[rb], O[rb][cb]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int rb = 0; rb < 4; ++rb) {
          const float a = s_f[4 * PC + 16 * rb + n];
#pragma unroll
          for (int cb = 0; cb < NCB; ++cb) O[rb][cb] *= a;
        }
        // values that are none: left out of the products (a zero of P would bring
        // them to earlier tokens) and put back behind them
        int* s_bad = reinterpret_cast<int*>(s_f + 5 * PC);
        if (wrong) {
          s_bad[lane] = NEVER;
          wave_lds_sync();
#pragma unroll
          for (int cb = 0; cb < NCB; ++cb)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
              const bf16x8 f = frag_v(cb, kh);
              int first = NEVER;
#pragma unroll
              for (int e = 7; e >= 0; --e) first = finite((float)f[e]) ? first : 32 * kh + 8 * hi + e;
              if (first != NEVER) atomicMin(s_bad + col(cb), first);
            }
          wave_lds_sync();
        }
        // O += (P V)^T
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          bf16x8 fv[NCB];
#pragma unroll
          for (int cb = 0; cb < NCB; ++cb) {
            fv[cb] = frag_v(cb, kh);
            if (wrong) {
#pragma unroll
              for (int e = 0; e < 8; ++e) fv[cb][e] = finite((float)fv[cb][e]) ? fv[cb][e] : (__bf16)0.f;
            }
          }
          float lh[8], ll[8], dt[8];
          ldn<8>(s_f + 32 * kh + 8 * hi, lh);
          ldn<8>(s_f + PC + 32 * kh + 8 * hi, ll);
          ldn<8>(s_f + 2 * PC + 32 * kh + 8 * hi, dt);
#pragma unroll
          for (int rb = 2 * kh; rb < 4; ++rb) {
            const float ih = s_f[16 * rb + n], il = s_f[PC + 16 * rb + n];
            float x[8];
            const f32x4s* qk = reinterpret_cast<const f32x4s*>(smem + L::QK) + frag_of(rb, kh) * 128 + lane;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const f32x4s a = qk[64 * t];
#pragma unroll
              for (int r = 0; r < 4; ++r) x[4 * t + r] = a[r];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float d = __builtin_amdgcn_exp2f((ih - lh[e]) + (il - ll[e]));
              const float y = x[e] * d * dt[e];
              x[e] = rb >= 2 * kh + 2 || 32 * kh + 8 * hi + e <= 16 * rb + n ? y : 0.f;
            }
            bf16x8 fp[3];
            split8(x, fp);
#pragma unroll
            for (int v = 2; v >= 0; --v)
#pragma unroll
              for (int cb = 0; cb < NCB; ++cb) O[rb][cb] = mm32(fv[cb], fp[v], O[rb][cb]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int rb = 0; rb < 4; ++rb)
#pragma unroll
          for (int cp = 0; cp < NCB / 2; ++cp) {
            bf16x8 w;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float y = O[rb][2 * cp + (e >> 2)][e & 3];
              if (wrong) y = 16 * rb + n >= s_bad[32 * cp + 8 * hi + e] ? __builtin_nanf("") : y;
              w[e] = (__bf16)y;
            }
            if (16 * rb + n < nt)
              *reinterpret_cast<bf16x8*>(reinterpret_cast<unsigned char*>(op + (int64_t)(t0 + 16 * rb) * p.os + 32 * cp) + oo) = w;
          }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (active) {
      if (left > 0) fetch(t0 + PC, left < PC ? left : PC);
      __builtin_amdgcn_sched_barrier(0);
      // S = exp(L_C) S + K^T (w V)
      each([&](int kb, int cb, int e) { S[kb][cb][e] *= decay; });
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        float w[8];
        ldn<8>(s_f + 3 * PC + 32 * kh + 8 * hi, w);
        bf16x8 fk[DB][2];
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int t = 0; t < 2; ++t) fk[db][t] = frag_kt(s_k, db, t, kh);
#pragma unroll
        for (int cb = 0; cb < NCB; ++cb) {
          const bf16x8 f = frag_v(cb, kh);
          float x[8];
          bf16x8 fw[3];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = w[e] * (float)f[e];
          split8(x, fw);
#pragma unroll
          for (int v = 2; v >= 0; --v)
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
              for (int t = 0; t < 2; ++t) S[db][cb][t] = mm32(fk[db][t], fw[v], S[db][cb][t]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  }
  if (!active) return;

  if (!OUT) {
    f32x4s* to = seg_at(slot);
    each([&](int kb, int cb, int e) { to[((kb * NCB + cb) * 2 + e) * 64] = S[kb][cb][e]; });
    if (lane == 0 && c0 == 0) p.seg_decay[(size_t)slot * p.H + h] = exp2_of(total);
    return;
  }
  if (!last) return;                             // (the state behind a segment is known already)
  each([&](int kb, int cb, int e) {
#pragma unroll
    for (int r = 0; r < 4; ++r) Sg[(size_t)(32 * kb + 8 * hi + 4 * e + r) * DV + col(cb)] = S[kb][cb][e][r];
  });
  if (!p.prime) return;
  const int off = p.sk.off[h], ranks = p.sk.off[h + 1] - off;
  if (ranks == 0) {                              // a dense-fallback head: the state copy
    int at = 0;
    while (at + 1 < p.sk.ndense && p.sk.dense_list[at] != h) ++at;
    bf16* C = reinterpret_cast<bf16*>(p.sk.Sc) + ((size_t)b * p.sk.ndense + at) * DK * DV + c0;
    each([&](int kb, int cb, int e) {
#pragma unroll
      for (int r = 0; r < 4; ++r) C[(size_t)(32 * kb + 8 * hi + 4 * e + r) * DV + col(cb)] = f32_to_bf16(S[kb][cb][e][r]);
    });
    return;
  }
  // u_j = S^T p_j in fp32: K-step (kb, e) of v_mfma_f32_16x16x4_f32 covers rows
  // 32 kb + 8 k + e; a lane's results are columns 4 hi + r of tile cb for j = n
  f32x4s U[NCB];
#pragma unroll
  for (int cb = 0; cb < NCB; ++cb) U[cb] = f32x4s{0.f, 0.f, 0.f, 0.f};
  const float* P = p.sk.Pt + (size_t)(off + (n < ranks ? n : 0)) * DK + 8 * hi;
#pragma unroll
  for (int kb = 0; kb < DB; ++kb) {
    float x[8];
    ldn<8>(P + 32 * kb, x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int cb = 0; cb < NCB; ++cb) U[cb] = mm4(S[kb][cb][e >> 2][e & 3], x[e], U[cb]);
  }
  if (n < ranks) {                               // (columns j >= ranks repeat row 0 and are dropped)
    bf16* Ug = reinterpret_cast<bf16*>(p.sk.U) + ((size_t)b * p.sk.R + off + n) * DV + c0;
#pragma unroll
    for (int cp = 0; cp < NCB / 2; ++cp) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = U[2 * cp + (e >> 2)][e & 3];
      stn<8>(Ug + 32 * cp + 8 * hi, x);
    }
  }
}

// The states between a prompt's segments: S behind segment s is g_s S + B_s,
// written over B_s.  Element by element (in whatever order the waves left them), so
// bound by memory; one lane a vector of four, the next segment's in flight.
constexpr int JOIN_THREADS = 256;
template <int DK, int DV>
__global__ void __launch_bounds__(JOIN_THREADS) scan_join_kernel(ScanParams p) {
  constexpr int VECS = DK * DV / 4, BLOCKS = VECS / JOIN_THREADS;
  const int tile = blockIdx.x / BLOCKS, x = tile / p.H, h = tile - x * p.H;
  int rank = 0;
  const int i = chunked_prompt(p, x, &rank);
  if (i < 0) return;
  const int s0 = p.start[i], len = p.start[i + 1] - s0;
  const int segs = (int)(((int64_t)len + (1 << p.seg_shift) - 1) >> p.seg_shift);
  if (prompt_wrong(p, i, p.seqs ? p.seqs[i] : i) || segs < 3) return;      // (reported by the others)
  const int first = first_slot(s0, rank, p.seg_shift);
  f32x4s* at = reinterpret_cast<f32x4s*>(p.seg + ((size_t)first * p.H + h) * DK * DV) + blockIdx.x % BLOCKS * JOIN_THREADS + threadIdx.x;
  const float* decay = p.seg_decay + (size_t)first * p.H + h;
  const size_t step = (size_t)p.H * VECS;
  f32x4s S = at[0], B = at[step];
  for (int s = 1; s + 1 < segs; ++s) {
    f32x4s next = B;
    if (s + 2 < segs) next = at[(s + 1) * step];
    S = decay[(size_t)s * p.H] * S + B;
    at[s * step] = S;
    B = next;
  }
}

template <int DK, int DV, bool OUT>
void launch_chunks(const ScanParams& p, hipStream_t st) {
  const unsigned tiles = (unsigned)(p.seg_shift ? p.nsegs : p.nchunked) * p.G;
  hipLaunchKernelGGL((scan_chunk_kernel<DK, DV, OUT>), dim3((tiles + 7) / 8 * 8 * p.parts), dim3(64 * p.waves),
                     (ScanLds<DK, OUT>::bytes(p.waves)), st, p);
}

template <int DK, int DV>
int launch(const ScanParams& p, hipStream_t st) {
  static_assert(ScanLds<DK, true>::bytes(SCAN_WAVES) <= 160 * 1024, "LDS of a CU");
  if (p.seg_shift) {
    launch_chunks<DK, DV, false>(p, st);
    hipLaunchKernelGGL((scan_join_kernel<DK, DV>), dim3((unsigned)p.nchunked * p.H * (DK * DV / 4 / JOIN_THREADS)), dim3(JOIN_THREADS), 0,
                       st, p);
  }
  launch_chunks<DK, DV, true>(p, st);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_scan_chunks(int dk, int dv, const ScanParams& p, hipStream_t st) {
  if (dk == 64 && dv == 64) return launch<64, 64>(p, st);
  if (dk == 128 && dv == 64) return launch<128, 64>(p, st);
  if (dk == 128 && dv == 128) return launch<128, 128>(p, st);
  return -2;
}

}  // namespace sk
