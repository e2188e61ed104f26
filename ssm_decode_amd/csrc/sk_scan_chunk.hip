// Prompts through the selective state space scan in chunks of 64 tokens.  With
// l_t = -dt_t exp(A_h), L_i the sum of a chunk's l up to token i, and S_0 the state
// before the chunk:
//   P_ij = exp(L_i - L_j) dt_j (q_i . k_j)   for j <= i, 0 above
//   O = diag(exp L) Q S_0 + P V
//   S = exp(L_C) S_0 + K^T diag(exp(L_C - L_j) dt_j) V
// The sums L run in 64 bits, so that a difference of two is that of the tokens
// between them, whatever came before.  P's factors are a quotient, exp(-L_j) dt_j on K Q^T and
// exp(L_i) on the outputs, where a chunk's decays together are 2^-NEAR_BITS or more and
// the factors so far from the type's end that no quotient overflows; elsewhere each is the
// exponential of a difference.
//
// Precision.  The state is fp32, and so is every product.  They run on the bf16 matrix
// cores with each fp32 operand (S_0, P, the weighted V) as an exact sum of three
// bf16 values, so a product with bf16 data (Q, V, K^T) takes three instructions.
//
// Layout.  A wave has 32 columns of one head's state, all rows, in registers, and a
// workgroup up to eight waves of one group, whose keys and queries it shares.  K, Q and
// V (64 columns for two waves) are in LDS twice: the next chunk's copy, straight from
// memory, is in flight over the present one.  The triangle of K Q^T is formed once a
// chunk, by all waves, and left in LDS as the operand that P V needs.  All products
// are the transposed ones, so that a lane's results are runs of columns of one token.
//
// Bound by the waves' instructions.  128 heads of 128 x 64 in 8 groups: one prompt of
// 16384 tokens 132 us without outputs, 11 between the segments and 342 with outputs, 24
// prompts of 15715 tokens together 371.  A wave's chunk of 64 tokens is 114 of the matrix
// instructions of 32 x 32 x 16 and about 2000 others, two waves to a SIMD (a lane's state,
// outputs and operands take 256 registers): over the last launch vector instructions take 56% of the time, the matrix cores 34%, and a
// wave waits 29% of its own for the other's issue and 31% at counters and barriers.  Its
// memory runs at 1.9 TB/s.  64 columns a wave halve the reads of K and Q and spill.
#include <type_traits>

#include "sk_prompt_chunk.hpp"
#include "sk_scan_device.hpp"

namespace sk {
namespace {

// (terms with V may pass 2^(128 - NEAR_BITS) only where they overflow on the way to an output)
constexpr int NEAR_BITS = 40;
constexpr uint32_t BIG_T = 0x5f800000u;          // 2^64: |K Q^T| from here on, and steps of 2^23 and more, take no quotient
constexpr float BIG_DT = 0x1p23f;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Operands of v_mfma_f32_32x32x16_bf16 (h = lane / 32, ln = lane % 32): row or column
// ln, eight of the 16 products' terms from 8 h on.  Register r of a result is row
// 8 (r / 4) + 4 h + r % 4 of column ln; row m stands for row swap23(m) of the block,
// so that registers 8 s .. 8 s + 7 are its rows 16 s + 8 h .. + 7: an operand of the
// next product as they stand, and runs of eight columns or tokens.
__device__ __forceinline__ int swap23(int m) { return (m & ~12) | (m & 4) << 1 | (m & 8) >> 1; }
__device__ __forceinline__ f32x16 mm16(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ void rows8(const f32x16& a, int s, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = a[8 * s + e];
}

template <int DK, bool OUT>
struct ScanLds {
  static constexpr int K = 0;                    // [2][64][DK]
  static constexpr int Q = K + 2 * PC * DK * 2;
  static constexpr int T = Q + (OUT ? 2 * PC * DK * 2 : 0);      // six fragments of K Q^T in fp32
  static constexpr int V = T + (OUT ? FRAGS * 2 * FRAG_BYTES : 0);      // two waves after two: [2][64][64]
  static constexpr int V_BYTES = PC * 2 * SCAN_COLS * 2, FACTORS = 7 * PC * 4;
  static constexpr int big(int waves) { return V + waves / 2 * 2 * V_BYTES + waves * FACTORS; }      // [2] whether K Q^T has a large element
  static constexpr int bytes(int waves) { return big(waves) + (OUT ? 16 : 0); }
};

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane((int)x); }
__device__ __forceinline__ const void* uniform(const void* x) {
  const uint64_t u = reinterpret_cast<uint64_t>(x);
  return reinterpret_cast<const void*>((uint64_t)uniform((uint32_t)(u >> 32)) << 32 | uniform((uint32_t)u));
}

// The f-th pair of 16 x 16 tiles of the triangle: columns (tokens i) 16 rb .., rows
// (tokens j) 32 kh ..; and its fragment of 32 columns of block ib, rows 16 s ..
__device__ __forceinline__ constexpr int frag_rb(int f) { return f < 2 ? f : 2 + (f - 2) / 2; }
__device__ __forceinline__ constexpr int frag_kh(int f) { return f < 2 ? 0 : (f - 2) & 1; }
__device__ __forceinline__ constexpr int frag_of(int ib, int s) { return ib == 0 ? s : 2 + s; }

// One workgroup per (segment or prompt, group, part of its heads).  Where prompts are
// cut into segments of 2^seg_shift tokens, three launches take the place of one:
//   1. without outputs, the segments but the last, at once: each from a zero state
//      (the first from the prompt's) its state behind it, B, and the product g of
//      its decays: the state behind a segment is g S + B;
//   2. scan_join_kernel: the states between the segments, in order (few segments: the
//      third launch's do that, each for itself);
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
  const int n = lane & 15, hi = lane >> 4, ln = lane & 31, hh = lane >> 5;
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
  const bf16* vp = reinterpret_cast<const bf16*>(p.v) + (int64_t)s0 * p.vs + (int64_t)h * DV + (c0 & -64);
  const bf16* dp = reinterpret_cast<const bf16*>(p.gate) + (int64_t)s0 * p.gs + h;
  // Rows have their 16-byte pieces swizzled so that those of a fragment spread over
  // the banks: piece pc of a row of PPR (16, DK = 64 and V: 8) is at pc ^ swz(row).
  auto swz = [](int row, int ppr) {
    const int s = (row & 3) | ((row >> 1) & 12);
    return ppr == 16 ? s : s >> 1;
  };
  const uint32_t lds0 = lds_address(smem);
  const int v_at = L::V + (wv >> 1) * 2 * L::V_BYTES;
  float* s_f = reinterpret_cast<float*>(smem + L::V + NW / 2 * 2 * L::V_BYTES + wv * L::FACTORS);      // L (upper and lower part), dt, weight, exp L; first wrong tokens
  float dr = 0.f;
  // dt (a token a lane) of a chunk of nt tokens, K and Q's pieces that this wave takes in
  // part `at` of `of` of a chunk's time, and eight of its half of V's rows, into buffer
  // buf.  (All at once they would stand in the way of each other, and of the wave: a
  // prompt of 16384 tokens spent 6500 of 32000 cycles a chunk on their issue.)  Rows
  // behind the end repeat the last one with a dt of 0: their weights are zeros, and
  // what they give is not stored.
  int fl = lane;
  auto fetch_dt = [&](int t0, int nt) {
    const int r = fl < nt - 1 ? fl : nt - 1;
    dr = to_f32(*reinterpret_cast<const bf16*>(reinterpret_cast<const unsigned char*>(dp + (int64_t)t0 * p.gs) + (uint32_t)(r * p.gs * 2)));
  };
  // (in a whole chunk a lane's offset from its unit's first row is the same for all
  // units, but for a turned bit or two of the swizzle)
  constexpr int RPU = 64 / PPR;                  // rows of a unit of K or Q
  auto copy_kq = [&](int t0, int buf, int at, int of) {
    for (int c = wv + NW * at; c < PPR; c += NW * of) {
      const uint32_t to = lds0 + buf * PC * DK * 2 + c * 1024, row = fl / PPR;
      const uint32_t x = ((fl % PPR) ^ (PPR == 16 ? fl >> 4 : (fl >> 4) & 1)) * 16 ^ (PPR == 16 ? (c & 6) * 32 : (c & 3) * 32);
      copy16(uniform(kp + (int64_t)(t0 + RPU * c) * p.ks), row * (uint32_t)(p.ks * 2) + x, uniform(to + L::K));
      if (OUT) copy16(uniform(qp + (int64_t)(t0 + RPU * c) * p.qs), row * (uint32_t)(p.qs * 2) + x, uniform(to + L::Q));
    }
  };
  auto copy_v = [&](int t0, int buf, int v) {
    const int first = 32 * (wv & 1) + 8 * v;
    copy16(uniform(vp + (int64_t)(t0 + first) * p.vs), (uint32_t)(fl >> 3) * (uint32_t)(p.vs * 2) + (((fl & 7) ^ ((fl >> 4) & 1)) * 16 ^ (v & 3) * 32),
           uniform(lds0 + v_at + buf * L::V_BYTES + first * 128));
  };
  // .. and all of them, of a chunk that may be the last
  auto copy_last = [&](int t0, int nt, int buf) {
#pragma unroll 1
    for (int c = wv; c < PPR; c += NW) {
      const int x = c * 64 + fl, row = x / PPR, pc = (x % PPR) ^ swz(row, PPR), r = row < nt - 1 ? row : nt - 1;
      const uint32_t to = lds0 + buf * PC * DK * 2 + c * 1024;
      copy16(uniform(kp + (int64_t)t0 * p.ks), (uint32_t)(r * p.ks * 2) + pc * 16, uniform(to + L::K));
      if (OUT) copy16(uniform(qp + (int64_t)t0 * p.qs), (uint32_t)(r * p.qs * 2) + pc * 16, uniform(to + L::Q));
    }
#pragma unroll 1
    for (int v = 0; v < 4 && active; ++v) {
      const int first = 32 * (wv & 1) + 8 * v, row = first + (fl >> 3), pc = (fl & 7) ^ swz(row, 8), r = row < nt - 1 ? row : nt - 1;
      copy16(uniform(vp + (int64_t)t0 * p.vs), (uint32_t)(r * p.vs * 2) + pc * 16, uniform(lds0 + v_at + buf * L::V_BYTES + first * 128));
    }
  };

  // -------------------------------------------------------------- state
  f32x16 S[DB];                                  // rows 32 db .., the wave's columns
  const int col = swap23(ln);                    // the lane's column
  float* Sg = p.S + ((size_t)b * p.H + h) * DK * DV + c0 + col;
  auto seg_at = [&](int s) { return reinterpret_cast<f32x4s*>(p.seg + (((size_t)s * p.H + h) * UPH + c0 / SCAN_COLS) * UNIT) + lane; };
  auto each = [&](auto f) {                      // f(block, register, row)
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) f(db, r, 32 * db + 16 * (r >> 3) + 8 * hh + (r & 7));
  };
  auto each4 = [&](auto f) {                     // f(block, four registers, place in a segment's workspace)
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int q = 0; q < 4; ++q) f(db, q, (db * 4 + q) * 64);
  };
  auto four = [&](int db, int q) { return f32x4s{S[db][4 * q], S[db][4 * q + 1], S[db][4 * q + 2], S[db][4 * q + 3]}; };
  if (len > 0) {
    const int nt = len < PC ? len : PC;
    copy_last(0, nt, 0);
    if (active) fetch_dt(0, nt);
  }
  each([&](int db, int r, int) { S[db][r] = 0.f; });
  if (active) {
    if (seg == 0 && !(OUT && !last)) {
      if (!p.has_state || p.has_state[i] != 0) each([&](int db, int r, int row) { S[db][r] = Sg[(size_t)row * DV]; });
      if (!OUT) {
        f32x4s* to = seg_at(slot + slots - 1);
        each4([&](int db, int q, int at) { to[at] = four(db, q); });
      }
    } else if (OUT) {
      // (joined: the state before it; few: the segments' from the first one's on)
      const bool chain = seg > 0 && !p.joined;
      const f32x4s* from = seg_at(seg == 0 ? slot + slots - 1 : chain ? slot - seg : slot - 1);
      each4([&](int db, int q, int at) {
        const f32x4s x = from[at];
#pragma unroll
        for (int r = 0; r < 4; ++r) S[db][4 * q + r] = x[r];
      });
      for (int s = slot - seg + 1; chain && s < slot; ++s) {
        const float g = p.seg_decay[(size_t)s * p.H + h];
        const f32x4s* B = seg_at(s);
        each4([&](int db, int q, int at) {
          const f32x4s x = B[at];
#pragma unroll
          for (int r = 0; r < 4; ++r) S[db][4 * q + r] = g * S[db][4 * q + r] + x[r];
        });
      }
    }
  }
  // (finite also where exp(A) is not, so that a step of zero takes nothing)
  const float rate_log = p.A[h];
  const double rate = wave_last(exp(rate_log > 700.f ? 700. : (double)rate_log) * -LOG2E);
  double total = 0.;

  bf16* op = reinterpret_cast<bf16*>(p.o) + (int64_t)s0 * p.os + (int64_t)h * DV + c0;
  const uint32_t oo = (uint32_t)((lane >> 2) * p.os * 2) + (lane & 3) * 16;

  // Byte addresses of a lane's fragments.  A fragment's rows differ by whole multiples
  // of what the swizzle looks at, or by such that change one bit of it, so that one
  // register, constant offsets and flipped bits cover all of a kind:
  //  tokens 32 tt + ln of Q, columns 32 db + 16 s + 8 h ..: (fq ^ 64 db ^ 32 s) + 32 tt ROW
  //  tokens 16 rb + n of Q, columns 32 kb + 8 hi .. (the triangle's tiles are 16 x 16): (q16 ^ 64 kb ^ flip of rb) + 16 rb ROW
  //  tokens 32 kh + block_row(n, t) of K, columns as those: (kk ^ 64 kb) + (32 kh + 4 t) ROW
  //  K^T, tokens 16 s + 8 h + ti (+ 4), the lane's run of four of rows 32 db ..: (kt ^ 64 db ^ flip of s) + (16 s (+ 4)) ROW
  //  V, tokens as K^T's, the lane's run of four columns: (va ^ 64 (s & 1)) + (16 s (+ 4)) 128
  constexpr int ROW = DK * 2, TFLIP = PPR == 16 ? 128 : 64;
  const int ti = n >> 2, run = n & 3, g0 = hi & 1, half = 4 * (c0 / SCAN_COLS & 1);      // the wave's first piece of V
  int fq = ln * ROW + (hh ^ swz(ln, PPR)) * 16;
  int q16 = n * ROW + (hi ^ swz(n, PPR)) * 16;
  int kk = block_row(n, 0) * ROW + (hi ^ swz(block_row(n, 0), PPR)) * 16;
  int kt = (8 * hh + ti) * ROW + ((2 * g0 + (run & 1)) ^ swz(8 * hh + ti, PPR)) * 16 + (run >> 1) * 8;
  int va = (8 * hh + ti) * 128 + ((half + 2 * g0 + (run & 1)) ^ swz(8 * hh + ti, 8)) * 16 + (run >> 1) * 8;
  auto frag = [](const unsigned char* s, int at) { return as_frag(*reinterpret_cast<const u32x4*>(s + at)); };

  asm volatile("s_waitcnt vmcnt(0)" : "+v"(dr)::"memory");
  int* s_big = reinterpret_cast<int*>(smem + L::big(NW));
  if (OUT && tid < 2) s_big[tid] = 0;
  int buf = 0;
  for (int t0 = 0; t0 < len; t0 += PC, buf ^= 1) {
    const int nt = len - t0 < PC ? len - t0 : PC, left = len - t0 - PC, next = left < PC ? left : PC;
    // (or every fragment's address would be made in front of the loop, and held)
    asm volatile("" : "+v"(fq), "+v"(q16), "+v"(kk), "+v"(kt), "+v"(va), "+v"(fl));
    // the chunk's decays, a token a lane: L split so that a difference of two is exact
    // to fp32 (a decay of less than 2^-256 a token is zero)
    float decay = 0.f;
    bool near_one = false;
    if (active) {
      const float d = lane < nt ? dr : 0.f;
      double l = (double)d * rate;
      l = l < -256. ? -256. : l;
      const double at = wave_prefix(l), end = wave_last(at);
      const double upper = (at + 0x1.8p42) - 0x1.8p42;      // a multiple of 2^-10, |L| <= 2^14
      s_f[lane] = (float)upper;
      s_f[PC + lane] = (float)(at - upper);
      near_one = end >= -NEAR_BITS && !__any(d >= BIG_DT);
      s_f[2 * PC + lane] = OUT && near_one ? exp2_of(-at) * d : d;
      s_f[3 * PC + lane] = exp2_of(end - at) * d;
      s_f[4 * PC + lane] = exp2_of(at);
      decay = exp2_of(end);
      if (!OUT) total += end;
    }
    // everybody's copies have landed, and everybody has read the other buffer
    __syncthreads();
    const unsigned char *s_k = smem + L::K + buf * PC * DK * 2, *s_q = smem + L::Q + buf * PC * DK * 2;
    if constexpr (OUT) {
      // The triangle: tile t of rows (tokens j) 32 kh .., columns (tokens i) 16 rb .., left
      // where a lane of the 32-column fragments finds it.
      uint32_t big = 0;
      for (int c = wv; c < 2 * FRAGS; c += NW) {
        const int f = c >> 1, t = c & 1, rb = frag_rb(f), kh = frag_kh(f), flip = (rb & 1) * TFLIP;
        f32x4s a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < DB; ++kb)
          a = mm32(frag(s_k, (kk ^ 64 * kb) + (32 * kh + 4 * t) * ROW), frag(s_q, (q16 ^ 64 * kb ^ flip) + 16 * rb * ROW), a);
        const int to = frag_of(rb >> 1, 2 * kh + (hi >> 1)) * 2 + t;
        reinterpret_cast<f32x4s*>(smem + L::T)[to * 64 + 32 * (hi & 1) + 16 * (rb & 1) + n] = a;
#pragma unroll
        for (int r = 0; r < 4; ++r) big = max(big, __float_as_uint(a[r]) & 0x7fffffffu);
      }
      if (tid == 0) s_big[buf ^ 1] = 0;          // (read behind the last chunk's triangle, set behind the next barrier)
      if (__any(big >= BIG_T) && lane == 0) s_big[buf] = 1;
    }
    if (!active) {
      if (left > 0) copy_last(t0 + PC, next, buf ^ 1);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      if (OUT) __syncthreads();
      continue;
    }
    if (left > 0) {
      fetch_dt(t0 + PC, next);
      if (left < PC) copy_last(t0 + PC, next, buf ^ 1);
    }
    unsigned char* s_v = smem + v_at + buf * L::V_BYTES;
    auto frag_v = [&](int s) {                   // V^T (or V): tokens 16 s + 8 h ..
      const unsigned char* at = s_v + (va ^ (s & 1) * 64) + 16 * s * 128;
      return join(read_tr(at), read_tr(at + 4 * 128));
    };
    int* s_bad = reinterpret_cast<int*>(s_f + 6 * PC);
    bool wrong = false;
    f32x16 O[2];                                 // outputs: columns, tokens 32 tt + ln

    if constexpr (OUT) {
      // O = (Q S)^T: in each of the steps the next one's fragments are read and its values
      // split between the matrix instructions.
      constexpr int STEPS = 2 * DB;
      bf16x8 fr[2][2], ss[2][3];
      auto load = [&](int st) {
        const int flip = 64 * (st >> 1) ^ 32 * (st & 1), u = st & 1;
        fr[u][0] = frag(s_q, fq ^ flip);
        fr[u][1] = frag(s_q, (fq ^ flip) + 32 * ROW);
      };
      auto split_s = [&](int st) {
        float x[8];
        rows8(S[st >> 1], st & 1, x);
        split8(x, ss[st & 1]);
      };
      load(0);
      split_s(0);
      __builtin_amdgcn_sched_barrier(0);
      uint32_t top = 0;                          // the largest magnitudes of V, two values at a time
      f32x16 zero;
#pragma unroll
      for (int r = 0; r < 16; ++r) zero[r] = 0.f;
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int u = st & 1;
        if (st + 1 < STEPS) {
          load(st + 1);
          split_s(st + 1);
        }
        if (st >= STEPS - 4) {
          const u32x4 w = __builtin_bit_cast(u32x4, frag_v(st - (STEPS - 4)));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, w[e] & 0x7fff7fffu),
                                                                       __builtin_bit_cast(u16x2, top)));
        }
#pragma unroll
        for (int v = 2; v >= 0; --v)
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) O[tt] = mm16(ss[u][v], fr[u][tt], st == 0 && v == 2 ? zero : O[tt]);
        region<6, 1, 9>();
        if (left >= PC) {
          copy_kq(t0 + PC, buf ^ 1, st, STEPS);
          if (st >= STEPS - 4) copy_v(t0 + PC, buf ^ 1, st - (STEPS - 4));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();                           // (the triangle is whole)
      if (near_one && __builtin_amdgcn_readfirstlane(s_big[buf])) {
        near_one = false;
        s_f[2 * PC + lane] = lane < nt ? to_f32(dp[(int64_t)(t0 + lane) * p.gs]) : 0.f;
        wave_lds_sync();
      }
      // Values that are none would come to earlier tokens by zeros of P: they are taken
      // out of V, with each column's first token that has one.
      if (__any((top & 0xffffu) >= 0x7f80u || top >= 0x7f800000u)) {
        wrong = true;
        if (lane < SCAN_COLS) s_bad[lane] = NEVER;
        wave_lds_sync();
        for (int c = lane; c < PC * SCAN_COLS; c += 64) {
          const int row = c / SCAN_COLS, cc = c % SCAN_COLS;
          bf16* at = reinterpret_cast<bf16*>(s_v + row * 128 + ((half + (cc >> 3)) ^ swz(row, 8)) * 16) + (cc & 7);
          if ((*at & 0x7f80) == 0x7f80) {
            *at = 0;
            atomicMin(s_bad + cc, row);
          }
        }
        wave_lds_sync();
      }
    }

    // Where P's factors are no quotient, they are taken one by one.
    if (OUT && !near_one) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) O[tt] *= s_f[4 * PC + 32 * tt + ln];
    }
    // S = exp(L_C) S + K^T (w V) and O = diag(exp L) (O + (P V)^T), in turn: the matrix
    // instructions of one with the reads, factors and splits of the other between.
    constexpr int FA = OUT ? 1 : 2;              // (with outputs K^T's next is read behind its last use)
    bf16x8 fa[FA][DB], fw[3], fp[2][3], fv[2];
    float wj[8], fj[8];
    auto load_k = [&](int s) {
      const int flip = (s & 1) * TFLIP;
#pragma unroll
      for (int db = 0; db < DB; ++db) {
        const unsigned char* at = s_k + (kt ^ (64 * db ^ flip)) + 16 * s * ROW;
        fa[s % FA][db] = join(read_tr(at), read_tr(at + 4 * ROW));
      }
    };
    // (factors are read one region before they are needed)
    auto load_w = [&](int s) { ldn<8>(s_f + 3 * PC + 16 * s + 8 * hh, wj); };
    auto load_f = [&](int s) { ldn<8>(s_f + 2 * PC + 16 * s + 8 * hh, fj); };
    auto prep_w = [&](int s) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = wj[e] * (float)fv[s & 1][e];
      split8(x, fw);
    };
    f32x4s tr[2][2];
    auto load_t = [&](int s) {
#pragma unroll
      for (int ib = s >> 1; ib < 2; ++ib)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          tr[ib][t] = reinterpret_cast<const f32x4s*>(smem + L::T)[(frag_of(ib, s) * 2 + t) * 64 + lane];
    };
    auto prep_p = [&](int ib, int s) {           // of P, columns (tokens i) 32 ib .., rows (tokens j) 16 s ..
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = tr[ib][e >> 2][e & 3] * fj[e];
        if (ib == s >> 1) x[e] = 16 * (s & 1) + 8 * hh + e <= ln ? x[e] : 0.f;
      }
      split8(x, fp[ib]);
    };
    auto far_factors = [&](int ib, int s) {      // (in place of T)
      const float ih = s_f[32 * ib + ln], il = s_f[PC + 32 * ib + ln];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = 16 * s + 8 * hh + e;
        tr[ib][e >> 2][e & 3] *= __builtin_amdgcn_exp2f((ih - s_f[j]) + (il - s_f[PC + j]));
      }
    };
    // columns of a token go through LDS (over V's, which are read), so that a store has
    // runs of 64 bytes
    auto store = [&](int tt) {
      if (near_one) O[tt] *= s_f[4 * PC + 32 * tt + ln];
      if (wrong) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * tt + ln >= s_bad[16 * (r >> 3) + 8 * hh + (r & 7)]) O[tt][r] = __builtin_nanf("");
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = (__bf16)O[tt][8 * s + e];
        const int row = 32 * tt + ln;
        *reinterpret_cast<bf16x8*>(s_v + row * 128 + ((half + 2 * s + hh) ^ swz(row, 8)) * 16) = w;
      }
      wave_lds_sync();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = 32 * tt + 16 * s + (lane >> 2);
        const u32x4 w = *reinterpret_cast<const u32x4*>(s_v + row * 128 + ((half + (lane & 3)) ^ swz(row, 8)) * 16);
        if (row < nt) *reinterpret_cast<u32x4*>(reinterpret_cast<unsigned char*>(op + (int64_t)(t0 + 32 * tt + 16 * s) * p.os) + oo) = w;
      }
    };
    fv[0] = frag_v(0);
    load_w(0);
    load_k(0);
    if (OUT) {
      load_f(0);
      load_t(0);
    }
#pragma unroll
    for (int db = 0; db < DB; ++db) S[db] *= decay;
    prep_w(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s + 1 < 4) {
        fv[(s + 1) & 1] = frag_v(s + 1);
        load_w(s + 1);
      }
      if (OUT) {
        if (!near_one) {
#pragma unroll
          for (int ib = s >> 1; ib < 2; ++ib) far_factors(ib, s);
        }
#pragma unroll
        for (int ib = s >> 1; ib < 2; ++ib) prep_p(ib, s);
      } else if (s + 1 < 4) {
        load_k(s + 1);
      }
#pragma unroll
      for (int v = 2; v >= 0; --v)
#pragma unroll
        for (int db = 0; db < DB; ++db) S[db] = mm16(fa[s % FA][db], fw[v], S[db]);
      region<3 * DB, 1, OUT ? 10 : 1>();
      if constexpr (OUT) {
        if (s + 1 < 4) {
          load_f(s + 1);
          load_t(s + 1);
          load_k(s + 1);
        }
#pragma unroll
        for (int v = 2; v >= 0; --v)
#pragma unroll
          for (int ib = s >> 1; ib < 2; ++ib) O[ib] = mm16(fv[s & 1], fp[ib][v], O[ib]);
      } else if (left >= PC) {
        copy_kq(t0 + PC, buf ^ 1, s, 4);
        copy_v(t0 + PC, buf ^ 1, s);
      }
      if (s + 1 < 4) prep_w(s + 1);
      if (OUT) {
        region<6, 2, 10>();
        if (s == 2) store(0);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // This wave's copies for the next chunk have landed: all but the last two of its
    // accesses to memory, which are the first tokens' outputs (of a chunk with a
    // next one).
    if (OUT) {
      asm volatile("s_waitcnt vmcnt(2)" : "+v"(dr)::"memory");
      store(1);
    } else {
      asm volatile("s_waitcnt vmcnt(0)" : "+v"(dr)::"memory");
    }
    if (wrong) {
      const float x = s_bad[col] == NEVER ? 0.f : __builtin_nanf("");
#pragma unroll
      for (int db = 0; db < DB; ++db) S[db] += x;
    }
  }
  if (!active) return;

  if (!OUT) {
    f32x4s* to = seg_at(slot);
    each4([&](int db, int q, int at) { to[at] = four(db, q); });
    if (lane == 0 && c0 == 0) p.seg_decay[(size_t)slot * p.H + h] = exp2_of(total);
    return;
  }
  if (!last) return;                             // (the state behind a segment is known already)
  each([&](int db, int r, int row) { Sg[(size_t)row * DV] = S[db][r]; });
  if (!p.prime) return;
  const int off = p.sk.off[h], ranks = p.sk.off[h + 1] - off;
  if (ranks == 0) {                              // a dense-fallback head: the state copy
    int at = 0;
    while (at + 1 < p.sk.ndense && p.sk.dense_list[at] != h) ++at;
    bf16* C = reinterpret_cast<bf16*>(p.sk.Sc) + ((size_t)b * p.sk.ndense + at) * DK * DV + c0 + col;
    each([&](int db, int r, int row) { C[(size_t)row * DV] = f32_to_bf16(S[db][r]); });
    return;
  }
  // u_j = S^T p_j in fp32: register r of v_mfma_f32_32x32x2_f32's operand is rows
  // 32 db + 16 (r / 8) + 8 k + r % 8; a lane's results are columns for j = ln
  f32x16 U;
#pragma unroll
  for (int r = 0; r < 16; ++r) U[r] = 0.f;
  const float* P = p.sk.Pt + (size_t)(off + (ln < ranks ? ln : 0)) * DK + 8 * hh;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float x[8];
      ldn<8>(P + 32 * db + 16 * s, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) U = __builtin_amdgcn_mfma_f32_32x32x2f32(S[db][8 * s + e], x[e], U, 0, 0, 0);
    }
  if (ln < ranks) {                              // (columns j >= ranks repeat row 0 and are dropped)
    bf16* Ug = reinterpret_cast<bf16*>(p.sk.U) + ((size_t)b * p.sk.R + off + ln) * DV + c0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float x[8];
      rows8(U, s, x);
      stn<8>(Ug + 16 * s + 8 * hh, x);
    }
  }
}

// The states between a prompt's segments: S behind segment s is g_s S + B_s,
// written over B_s.  Element by element (in whatever order the waves left them), so
// bound by memory; one lane a vector of four, the next four segments' in flight.
constexpr int JOIN_THREADS = 256, JOIN_AHEAD = 4;
template <int DK, int DV>
__global__ void __launch_bounds__(JOIN_THREADS) scan_join_kernel(ScanParams p) {
  constexpr int VECS = DK * DV / 4, BLOCKS = (VECS + JOIN_THREADS - 1) / JOIN_THREADS;
  const int tile = blockIdx.x / BLOCKS, x = tile / p.H, h = tile - x * p.H;
  int rank = 0;
  const int i = chunked_prompt(p, x, &rank);
  if (i < 0) return;
  const int s0 = p.start[i], len = p.start[i + 1] - s0;
  const int segs = (int)(((int64_t)len + (1 << p.seg_shift) - 1) >> p.seg_shift);
  if (prompt_wrong(p, i, p.seqs ? p.seqs[i] : i) || segs < 3) return;      // (reported by the others)
  const int first = first_slot(s0, rank, p.seg_shift), vec = blockIdx.x % BLOCKS * JOIN_THREADS + threadIdx.x;
  if (vec >= VECS) return;
  f32x4s* at = reinterpret_cast<f32x4s*>(p.seg + ((size_t)first * p.H + h) * DK * DV) + vec;
  const float* decay = p.seg_decay + (size_t)first * p.H + h;
  const size_t step = (size_t)p.H * VECS;
  f32x4s S = at[0], B[2][JOIN_AHEAD];
  float g[2][JOIN_AHEAD];
  auto fetch = [&](int s, int buf) {
#pragma unroll
    for (int u = 0; u < JOIN_AHEAD; ++u) {
      const int t = s + u < segs - 2 ? s + u : segs - 2;
      B[buf][u] = at[t * step];
      g[buf][u] = decay[(size_t)t * p.H];
    }
  };
  auto go = [&](int s, int buf) {
#pragma unroll
    for (int u = 0; u < JOIN_AHEAD; ++u) {
      if (s + u + 1 >= segs) return;
      S = g[buf][u] * S + B[buf][u];
      at[(s + u) * step] = S;
    }
  };
  fetch(1, 0);
  for (int s = 1; s + 1 < segs; s += 2 * JOIN_AHEAD) {
    if (s + JOIN_AHEAD + 1 < segs) fetch(s + JOIN_AHEAD, 1);
    go(s, 0);
    if (s + 2 * JOIN_AHEAD + 1 < segs) fetch(s + 2 * JOIN_AHEAD, 0);
    go(s + JOIN_AHEAD, 1);
  }
}

template <int DK, int DV, bool OUT>
void launch_chunks(const ScanParams& p, hipStream_t st) {
  const unsigned tiles = (unsigned)(p.seg_shift ? p.nsegs : p.nchunked) * p.G;
  hipLaunchKernelGGL((scan_chunk_kernel<DK, DV, OUT>), dim3((tiles + 7) / 8 * 8 * p.parts), dim3(64 * p.waves),
                     (ScanLds<DK, OUT>::bytes(p.waves)), st, p);
}

template <int DK, int DV>
int launch_join(const ScanParams& p, hipStream_t st) {
  constexpr unsigned BLOCKS = (DK * DV / 4 + JOIN_THREADS - 1) / JOIN_THREADS;
  hipLaunchKernelGGL((scan_join_kernel<DK, DV>), dim3((unsigned)p.nchunked * p.H * BLOCKS), dim3(JOIN_THREADS), 0, st, p);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

template <int DK, int DV>
int launch(const ScanParams& p, hipStream_t st) {
  static_assert(ScanLds<DK, true>::bytes(SCAN_WAVES) <= 160 * 1024, "LDS of a CU");
  if (p.seg_shift) {
    launch_chunks<DK, DV, false>(p, st);
    if (p.joined) launch_join<DK, DV>(p, st);
  }
  launch_chunks<DK, DV, true>(p, st);
  return hipGetLastError() == hipSuccess ? 0 : -5;
}

}  // namespace

int launch_scan_join(int dk, int dv, const ScanParams& p, hipStream_t st) {
  if (dk == 16 && dv == 32) return launch_join<16, 32>(p, st);
  if (dk == 64 && dv == 64) return launch_join<64, 64>(p, st);
  if (dk == 128 && dv == 64) return launch_join<128, 64>(p, st);
  if (dk == 128 && dv == 128) return launch_join<128, 128>(p, st);
  return -2;
}

int launch_scan_chunks(int dk, int dv, const ScanParams& p, hipStream_t st) {
  if (dk == 64 && dv == 64) return launch<64, 64>(p, st);
  if (dk == 128 && dv == 64) return launch<128, 64>(p, st);
  if (dk == 128 && dv == 128) return launch<128, 128>(p, st);
  return -2;
}

}  // namespace sk
