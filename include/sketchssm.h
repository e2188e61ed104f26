/*
 * sketchssm.h -- C ABI of the SketchSSM decode hot path on AMD Instinct
 * MI355X (gfx950).
 *
 * SketchSSM ("Write to the Full State, Read from a Compact Sketch",
 * arXiv 2609.33051) keeps the full recurrent state S of a linear-attention /
 * SSM head exact but reads it only once per window of W decode steps:
 *
 *   - flush (every W steps): read S once, apply the W buffered updates from
 *     the ring, build the sketch U = S^T P from the updated state with a fixed
 *     per-head basis P, write back S and U (project page, "02 / How to make a
 *     sketch", per-window flush panel; paper App. B);
 *   - read (the other W-1 steps): o = U (C q~) plus the exact contribution of
 *     the buffered updates, where q~ is the query pulled back through the
 *     buffered transitions; S is not read (project page, per-step non-flush
 *     panel; paper Sec. 3.2 and App. C.1).
 *
 * The coefficient map C is either a fixed per-head table the caller supplies
 * (the paper's fixed-coefficient rule, App. G) or the state-dependent map the
 * flush forms for every (sequence, head) tile from its new state,
 * C = (U^T U + lambda I)^{-1} U^T S^T with U the stored sketch (project page,
 * per-window flush panel; paper App. A.2.1-A.2.2).
 *
 * Two baselines share the layout: the standard full-state step (read and
 * write S every step; project page "01 / The idea", S_t = M_t S_{t-1} + B_t,
 * o_t = S_t^T q_t) and ReplaySSM (buffered writes, full-state read every
 * step; paper Sec. 1-2 and App. D).
 *
 * Families (per (sequence, head) tile; S is dk x dv, o = S^T q):
 *   SKSSM_MAMBA2: S <- a S + dt k v^T,  a = exp(-dt * exp(A_h)); q~ = (prod a) q
 *   SKSSM_GDN:    S <- alpha (I - beta k k^T) S + beta k v^T
 *   SKSSM_KDA:    S <- (I - beta k k^T) Diag(g) S + beta k v^T
 *
 * Memory and ownership
 *   - Every pointer inside sketchssm_buffers / sketchssm_step is a DEVICE
 *     pointer owned by the caller.  sketchssm_layer and its rank_offsets_host
 *     table are HOST memory, read during the call only and never retained.
 *   - The library allocates nothing, keeps no state between calls (except
 *     the per-device address of sketchssm_read_noalloc's scratch array) and
 *     never synchronises: every call only enqueues kernels on the caller's HIP
 *     stream (NULL = the default stream).  Buffers must not be reused until
 *     stream order guarantees completion.  Calls on different layers may run
 *     concurrently on different streams; calls on one layer must be ordered.
 *   - Calls are re-entrant; no C++ exception crosses the ABI.
 *
 * Errors
 *   - The return value is 0 on success or a negative SKSSM_E* code.
 *     Arguments are validated on the host, synchronously; on failure nothing
 *     is launched and nothing is written.
 *   - SKSSM_ELAUNCH reports a failed launch (hipGetLastError after it).
 *   - Semantic faults found by the kernels (a ring count outside [0, W], a
 *     read of a sequence whose window is already full, inconsistent counts
 *     within a Mamba-2 B/C group) leave that tile untouched and OR a
 *     SKSSM_ERRBIT_* bit into *err; the caller reads it after synchronising.
 *   - Device faults surface at the caller's next synchronisation.
 */
#ifndef SKETCHSSM_H
#define SKETCHSSM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* families */
#define SKSSM_MAMBA2 0
#define SKSSM_GDN 1
#define SKSSM_KDA 2

/* dtypes */
#define SKSSM_F32 0
#define SKSSM_BF16 1

/* coefficient maps */
#define SKSSM_COEF_FIXED 0 /* bufs->C: one fp32 map per head, shared by all sequences */
#define SKSSM_COEF_STATE 1 /* bufs->Cstate: one map per (sequence, head), written by the flush */

/* evaluation of the effective query and the buffered term at a non-flush
 * read (GDN and KDA; a Mamba-2 effective query is a decay only, and Mamba-2
 * ignores the choice) */
#define SKSSM_PULLBACK_SERIAL 0 /* one buffered transition at a time, newest first */
#define SKSSM_PULLBACK_WY 1     /* every buffered slot's coefficient from one triangular
                                   system over the slots (paper App. C.1), then q~ and
                                   the buffered term as sums over the slots */
#define SKSSM_PULLBACK_PROJ 2   /* the coefficients of SKSSM_PULLBACK_WY, with C q~ formed
                                   from per-slot factors projected through the coefficient
                                   map (paper App. C.2): the read that appends slot l stores
                                   P_l = C_h (Gamma_l (.) k_l) in bufs->ring_pc (Gamma_l:
                                   the product of the decays of slots 0..l), and
                                   C q~ = C_h (Gamma_n0 (.) q) - sum_l beta_l d_l P_l.
                                   Every non-flush step of such a layer is a
                                   sketchssm_read (replay steps do not store factors). */

/* flush flags */
#define SKSSM_FLUSH_DUE 0 /* flush tiles whose ring holds W entries */
#define SKSSM_FLUSH_ALL 1 /* flush every tile (prime U, or retire sequences) */
#define SKSSM_FLUSH_DUE_SCAN 2 /* as SKSSM_FLUSH_DUE, with the due sequences first listed
                                  on the device (in bufs->work), so that a ragged window
                                  phase launches workgroups for the due tiles only */
#define SKSSM_FLUSH_CLOSE 3 /* the step that closes every tile's window, in place of
                               sketchssm_read then SKSSM_FLUSH_DUE at that step: tiles
                               whose ring holds W - 1 entries take the step's own entry
                               as the W-th */

/* return codes */
#define SKSSM_OK 0
#define SKSSM_EINVAL -1  /* NULL or misaligned pointer (16-byte alignment) */
#define SKSSM_EDIM -2    /* unsupported shape, W, ranks or rank table */
#define SKSSM_EDTYPE -3  /* unsupported dtype combination */
#define SKSSM_EFLAG -4   /* unknown flag or coefficient-map mode */
#define SKSSM_ELAUNCH -5 /* kernel launch failed */
#define SKSSM_ESCRATCH -6 /* sketchssm_read_noalloc: the layer needs more scratch than the
                             library's array holds (SKSSM_NOALLOC_SCRATCH_BYTES) */

/* size of the device array that sketchssm_read_noalloc uses as its workspace
 * (16 MiB; one per GPU the library runs on, held until the process ends) */
#define SKSSM_NOALLOC_SCRATCH_BYTES 16777216

/* bits OR-ed into *err by the kernels */
#define SKSSM_ERRBIT_COUNT 1  /* count outside [0, W] (or == W at a read) */
#define SKSSM_ERRBIT_GROUP 2  /* Mamba-2 heads of one B/C group disagree on count */
#define SKSSM_ERRBIT_SEQ 4    /* sketchssm_flush_seqs, _prefill, _scan, _conv, _state_save,
                                 _state_load: a listed index outside [0, batch), or a sequence
                                 listed twice (flush_seqs: a tile claimed twice); _prefill, _scan,
                                 _conv: a list of first tokens that falls, or leaves [0, tokens];
                                 _reorder: a parent outside its group */
#define SKSSM_ERRBIT_SLOT 8   /* sketchssm_state_save/_load: a cache slot outside [0, slots), or
                                 a slot that an earlier entry of a save's list has */
#define SKSSM_ERRBIT_LOGIT 16 /* sketchssm_beam_select: a logit or a score that is a NaN or a
                                 positive infinity */

/* activations of sketchssm_group_norm */
#define SKSSM_ACT_NONE 0
#define SKSSM_ACT_SILU 1    /* x / (1 + exp(-x)) */
#define SKSSM_ACT_SIGMOID 2 /* 1 / (1 + exp(-x)) */

/* Supported shapes: (dk, dv) in {(16,32), (64,64), (128,64), (128,128)};
 * 1 <= W <= 32; 0 <= r_h <= min(dk, 16), except r_h <= dk when dk == 16
 * (r_h = 0: a dense-fallback head, paper App. D, which keeps a copy of its
 * state in the sketch dtype and reads it at non-flush steps; at most 64 per
 * layer);
 * heads % qk_groups == 0 (qk_groups == heads for GDN/KDA). */
typedef struct {
  int32_t family;            /* SKSSM_MAMBA2 | SKSSM_GDN | SKSSM_KDA */
  int32_t batch;             /* B sequences */
  int32_t heads;             /* H state heads */
  int32_t qk_groups;         /* G: Mamba-2 B/C groups (heads h in group h / (H/G)); GDN/KDA: = H */
  int32_t dk, dv;            /* state is dk x dv per (sequence, head) */
  int32_t window;            /* W: one flush every W steps */
  int32_t act_dtype;         /* dtype of q, k, v, o, Mamba-2 dt and the ring's k, v, dt */
  int32_t sketch_dtype;      /* dtype of U */
  const int32_t* rank_offsets_host; /* [H+1] host copy: exclusive prefix sum of r_h; r_h = 0
                                marks a dense-fallback head (no sketch: a state copy) */
  int32_t coef_map;          /* SKSSM_COEF_FIXED or SKSSM_COEF_STATE */
  float coef_ridge;          /* SKSSM_COEF_STATE: ridge relative to the mean eigenvalue of
                                the sketch's Gram matrix, lambda = coef_ridge * trace(G) / r_h;
                                finite and > 0 (ignored for SKSSM_COEF_FIXED) */
  int32_t pullback;          /* SKSSM_PULLBACK_SERIAL, _WY or _PROJ (non-flush reads) */
} sketchssm_layer;

typedef struct {
  float* S;                  /* [B][H][dk][dv] fp32, dv fastest */
  void* U;                   /* [B][R][dv] sketch dtype, R = offsets[H]; rows
                                off_h..off_h+r_h-1 hold u_j = S^T p_j of head h */
  const float* Pt;           /* [R][dk] fp32: row off_h + j = column j of P_h */
  const float* C;            /* SKSSM_COEF_FIXED: [R][dk] fp32: row off_h + j = row j of C_h
                                (r_h x dk); NULL allowed for SKSSM_COEF_STATE */
  const int32_t* rank_offsets; /* [H+1] device copy of rank_offsets_host */
  void* ring_k;              /* [B][G][W][dk] act dtype */
  void* ring_v;              /* [B][H][W][dv] act dtype */
  void* ring_gate;           /* Mamba-2: dt [B][H][W] act dtype; GDN: alpha [B][H][W] fp32;
                                KDA: g [B][H][W][dk] fp32 */
  float* ring_beta;          /* GDN/KDA: [B][H][W] fp32; NULL for Mamba-2 */
  int32_t* count;            /* [B][H]: entries buffered in tile (b,h) since its last flush,
                                0..W; every head of a sequence advances together */
  const float* A;            /* Mamba-2: [H] fp32; NULL otherwise */
  int32_t* err;              /* [1] device error word (SKSSM_ERRBIT_*), never cleared here */
  void* work;                /* workspace of sketchssm_workspace_bytes(layer) bytes (16-byte
                                aligned; may be NULL when that is 0); scratch that a call
                                overwrites, so calls sharing one workspace must be ordered */
  void* Cstate;              /* SKSSM_COEF_STATE: [B][R][dk] sketch dtype; rows off_h..off_h+r_h-1
                                of sequence b hold the map of tile (b, h), written by every
                                flush of that tile (NULL allowed for SKSSM_COEF_FIXED) */
  void* Scopy;               /* [B][D][dk][dv] sketch dtype, D = number of dense-fallback heads
                                (r_h = 0, at most 64), in head order: their state copies,
                                written by their flush, read by their non-flush reads.  NULL
                                allowed when D = 0.  (Compact: a [B][H] layout would put the
                                few dense tiles at strides that load a few memory channels.) */
  float* ring_pc;            /* GDN/KDA with SKSSM_PULLBACK_PROJ: [B][H][W][16] fp32, slot l
                                of tile (b, h) holds P_l (r_h entries); NULL otherwise */
} sketchssm_buffers;

typedef struct {             /* one decode step */
  const void* q;             /* [B][G][dk] act dtype */
  const void* k;             /* [B][G][dk] act dtype */
  const void* v;             /* [B][H][dv] act dtype */
  const void* gate;          /* Mamba-2: dt [B][H] act dtype; GDN: alpha [B][H] fp32;
                                KDA: g [B][H][dk] fp32 */
  const float* beta;         /* GDN/KDA: [B][H] fp32; NULL for Mamba-2 */
  void* o;                   /* [B][H][dv] act dtype (output) */
} sketchssm_step;

/* Non-flush sketched read (project page, per-step non-flush panel: c = C q~,
 * o^ = U c, plus the exact buffered contribution; paper Sec. 3.2 and
 * App. C.1 for q~).  For every tile: append the step's (k, v, gate, beta) at
 * ring slot count, count += 1; if count < W write o = U (C q~) + o_buf
 * (a dense-fallback head: o = Scopy^T q~ + o_buf), otherwise leave o for
 * sketchssm_flush.  Never reads S.  C is bufs->C
 * (SKSSM_COEF_FIXED) or the tile's own map in bufs->Cstate, as its last
 * flush wrote it (SKSSM_COEF_STATE).  Mamba-2 layers, and GDN/KDA layers
 * with dense-fallback heads, need bufs->work (sketchssm_workspace_bytes). */
int sketchssm_read(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                   const sketchssm_step* step, void* hip_stream);

/* Flush (paper App. B; project page per-window flush panel: U = S^T Omega,
 * fused into the update).  For every tile with count == W (flags =
 * SKSSM_FLUSH_DUE) or every tile (SKSSM_FLUSH_ALL): apply the count buffered
 * entries to S in order, write S, write U = S^T P from the updated state,
 * set count = 0 and, if step != NULL, write the exact output o = S^T q.
 * A dense-fallback head (r_h = 0) writes its state copy to bufs->Scopy
 * (rounded to the sketch dtype) instead of a sketch.
 * FLUSH_ALL with count == 0 primes U from the current state.
 * SKSSM_COEF_STATE: also write the tile's map to bufs->Cstate, solved in
 * fp32 from the sketch rows as stored (rounded to the sketch dtype) and the
 * updated state: G = U_h U_h^T (r_h x r_h), Y = U_h S^T (r_h x dk),
 * C = (G + lambda I)^{-1} Y, lambda = coef_ridge * trace(G) / r_h, stored in
 * the sketch dtype (C = 0 when the sketch is zero).
 * SKSSM_FLUSH_DUE_SCAN (paper App. B: each sequence flushes when its own
 * window fills): the same result as SKSSM_FLUSH_DUE for callers that do not
 * track window phases, given that every head of a sequence holds the same
 * count (sketchssm_read appends, and the flushes reset, all heads of a
 * sequence together).  A first launch (one workgroup) lists, in sequence
 * order, the sequences whose head-0 count is W in bufs->work
 * (sketchssm_workspace_bytes; 16-byte aligned) and reports head-0 counts
 * outside [0, W] (SKSSM_ERRBIT_COUNT).  The flush then runs a grid of one
 * workgroup per tile of min(batch, 2 * ceil(batch / W) + 8) sequences
 * (about twice what a ragged phase brings due at a step) over the tiles of
 * the listed sequences, each workgroup taking further tiles in turn when
 * the list is longer (an aligned phase), so that a ragged phase does not
 * pay a workgroup per tile of the batch.  A listed tile whose count is
 * below W is left alone; the counts of the other heads are
 * checked in listed sequences only.
 * SKSSM_FLUSH_CLOSE (paper App. B: the flush step applies the window's W
 * entries, its own included, and its output comes from the updated state):
 * for a step at which every sequence closes its window (an aligned phase),
 * called instead of sketchssm_read followed by SKSSM_FLUSH_DUE, with the
 * same results in S, U, count, the maps and o.  step is required (k, v,
 * gate, beta as for sketchssm_read; q and o for the output).  Each tile's
 * ring must hold W - 1 entries: the W - 1 buffered entries are applied,
 * then the step's own, and count becomes 0; a tile with any other count
 * sets SKSSM_ERRBIT_COUNT and is left untouched (the caller's phase was not
 * aligned: such a step needs sketchssm_read and SKSSM_FLUSH_DUE).  This
 * saves the read's launches at the closing step, which only append. */
int sketchssm_flush(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                    const sketchssm_step* step /* NULL: no output */, int32_t flags,
                    void* hip_stream);

/* Flush of listed sequences: sketchssm_flush with SKSSM_FLUSH_DUE, launched
 * for the tiles of the nseq sequences in seqs only (paper App. B: each
 * sequence flushes when its own window fills).  For callers that know which
 * sequences close their window at this step: under a ragged window phase
 * about batch / W sequences are due per step, and the due-flag flush pays
 * for a workgroup per tile of the whole batch.  seqs: DEVICE array of nseq
 * distinct sequence indices (int32, 4-byte aligned), 0 <= nseq <= batch.
 * A listed tile whose count is in [0, W) is left alone; a count outside
 * [0, W] sets SKSSM_ERRBIT_COUNT; an index outside [0, batch) sets
 * SKSSM_ERRBIT_SEQ and is skipped.  Each tile is claimed before it is
 * flushed (its count goes from W to W + 1 until the flush stores 0), so a
 * sequence listed twice is flushed once, and the second claim of a tile
 * that is still being flushed sets SKSSM_ERRBIT_SEQ.  nseq = 0 launches
 * nothing. */
int sketchssm_flush_seqs(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                         const sketchssm_step* step /* NULL: no output */, const int32_t* seqs,
                         int32_t nseq, void* hip_stream);

/* Standard full-state step (project page "01 / The idea": S_t = M_t S_{t-1}
 * + B_t, o_t = S_t^T q_t): S <- M S + B and o = S^T q for every tile.
 * Ignores the ring, count, U, Pt and C. */
int sketchssm_full_step(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                        const sketchssm_step* step, void* hip_stream);

/* ReplaySSM step (paper Sec. 1-2 and App. D: buffer writes for W steps,
 * read the full state every step).  Append as sketchssm_read; if count < W
 * write the exact o = S0^T q~ + o_buf reading S in full; if count == W apply
 * the W entries, write S, o = S^T q, count = 0.  Does not touch U. */
int sketchssm_replay_step(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                          const sketchssm_step* step, void* hip_stream);

/* Bytes of the workspace bufs->work for this layer, or a negative SKSSM_E*
 * code for an invalid layer: the larger of what sketchssm_read and
 * sketchssm_flush with SKSSM_FLUSH_DUE_SCAN need (a call uses the workspace
 * only while it runs, and calls on one layer are ordered, so both share it).
 * The read needs it (and checks bufs->work) only for these layers:
 * Mamba-2, for what the heads of a B/C group share at a step: the query's
 * coordinates in every head's sketch basis, C_h q (B x R fp32; the decay
 * factor of the pulled-back query is applied afterwards), the dot products
 * of the query with the group's buffered keys (B x G x W fp32) and the
 * group's checked ring fill (B x G int32); GDN and KDA with dense-fallback
 * heads: per (sequence, dense head) the pulled-back query (dk fp32), the
 * buffered term (dv fp32) and a flag (int32), passed from the read's main
 * launch to the launch that reads the state copies.  The scan flush lists
 * the due sequences: their number (int32 at byte 0), then from byte 256
 * their indices (batch int32, rounded up to 64).  The caller allocates it; the library never
 * does. */
int64_t sketchssm_workspace_bytes(const sketchssm_layer* layer);

/* sketchssm_read for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid allocation.
 * Same arguments, semantics, kernels and results as sketchssm_read, except
 * that bufs->work is ignored: the workspace is a device array of the library
 * (SKSSM_NOALLOC_SCRATCH_BYTES, one per GPU, resolved on the first call on
 * each device).  The call allocates nothing and never synchronises.
 * Returns SKSSM_ESCRATCH, launching nothing, when sketchssm_workspace_bytes
 * of the layer exceeds SKSSM_NOALLOC_SCRATCH_BYTES (at dk = 128 this holds,
 * e.g., a Mamba-2 layer of 1024 sequences with 2048 sketch rows and W = 32).
 * Every call on one GPU shares that GPU's array, whatever the layer or
 * stream: calls that may overlap on one GPU (two streams, two threads) race
 * and must be ordered by the caller.  The array keeps the last call's
 * contents; every value a call reads from it is written earlier in the same
 * call, so nothing needs clearing. */
int sketchssm_read_noalloc(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                           const sketchssm_step* step, void* hip_stream);

/* Prompts of the gated delta rule: token rows of nseq prompts, one behind the
 * other.  Rows are [H][dk] or [H][dv] elements in a row; the strides are the
 * elements from one token's row to the next (rows may be slices of one
 * projection's output), at least a row, at most 2^25, and a multiple of 16
 * bytes for q, k, v and o. */
typedef struct {
  const void* q;             /* [tokens][H][dk] act dtype */
  const void* k;             /* [tokens][H][dk] act dtype */
  const void* v;             /* [tokens][H][dv] act dtype */
  const float* gate;         /* alpha [tokens][H] fp32 */
  const float* beta;         /* [tokens][H] fp32 */
  void* o;                   /* [tokens][H][dv] act dtype (output); overlaps no input */
  int64_t q_stride, k_stride, v_stride, gate_stride, beta_stride, o_stride;
  int32_t tokens;            /* rows of q, k, v, gate, beta and o */
  int32_t nseq;              /* prompts, at most layer->batch */
  const int32_t* seq_start;  /* DEVICE [nseq + 1]: prompt i holds the tokens from seq_start[i] up to
                                seq_start[i + 1]; 0 <= seq_start[i] <= seq_start[i + 1] <= tokens */
  const int32_t* seqs;       /* DEVICE [nseq]: the sequence of prompt i, distinct; NULL: sequence i */
  const int32_t* has_state;  /* DEVICE [nseq]: 0: prompt i starts from a zero state (its sequence's
                                is not read); NULL: every prompt goes on from its state */
  int32_t prime;             /* 1: also write the sketch U = S^T P (a dense-fallback head's state copy)
                                of the new states; 0: leave the sketch as it is */
  void* work;                /* workspace of sketchssm_prefill_workspace_bytes (16-byte aligned; may be
                                NULL when that is 0), overwritten by the call */
  int64_t work_bytes;        /* bytes at work */
} sketchssm_prompts;

/* Prompts through the gated delta rule (SKSSM_GDN): for each of a prompt's
 * tokens in order, as sketchssm_full_step,
 *   S <- alpha (I - beta k k^T) S + beta k v^T,  o = S^T q,
 * and, with prime, the sketch that sketchssm_read starts from.  A sequence's
 * ring must be empty (count 0): a tile with buffered entries sets
 * SKSSM_ERRBIT_COUNT and is left untouched (flush it first).  A sequence
 * outside the batch sets SKSSM_ERRBIT_SEQ and its prompt is skipped; where one
 * is listed twice, the first prompt has it.  A seq_start that falls anywhere or
 * leaves [0, tokens] sets SKSSM_ERRBIT_SEQ and nothing is written.  A prompt of
 * no tokens leaves its state (or writes the zero state), with prime its sketch
 * too.  Token rows that no prompt holds are neither read nor written.
 * Sums run in fp32; longer prompts (dk >= 64) go in chunks of 64
 * tokens, whose products are those of fp32 operands.  An infinity or a NaN
 * in a token's row or in the state reaches what the recurrence brings it to
 * (as one or the other) and no earlier token.  An overflow of finite numbers,
 * the square of a key's norm among them, may in a chunk reach its head's
 * outputs from the chunk's start on.  Other
 * families return SKSSM_EDIM; prime with SKSSM_COEF_STATE is SKSSM_EFLAG (a
 * state-dependent map is formed by sketchssm_flush with SKSSM_FLUSH_ALL).
 * nseq = 0 launches nothing. */
int sketchssm_prefill(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                      const sketchssm_prompts* prompts, void* hip_stream);

/* Bytes of prompts->work that sketchssm_prefill needs for up to this many
 * tokens and prompts, or a negative SKSSM_E* code (the same that the call would
 * return: at most 2^22 - 1 chunks of 64 tokens, or prompts, times heads).  A
 * workspace for more tokens or prompts need not do for fewer: ask for the sizes
 * of the call.  Calls that may overlap need a workspace each. */
int64_t sketchssm_prefill_workspace_bytes(const sketchssm_layer* layer, int32_t tokens, int32_t nseq);

/* A pool of slots that each hold the states of one sequence's heads in 8 or
 * 4 bits.  32 consecutive values of a state row (along dv) share a scale:
 * scale = max|x| / 127 (8 bits) or / 7 (4 bits), code = x / scale rounded to
 * nearest even, and a code stands for code * scale (the scale is rounded down
 * where code * scale would overflow).  A block whose largest
 * magnitude is under 2^-100 is held as zeros; one with an infinity or a NaN
 * reads back as NaN. */
typedef struct {
  void* codes;               /* DEVICE [slots][H][dk][dv] two's complement codes of `bits` bits (4 bits:
                                two to a byte, the lower column in the low half) */
  float* scale;              /* DEVICE [slots][H][dk][dv / 32] */
  int32_t slots;
  int32_t bits;              /* 8 or 4, otherwise SKSSM_EDTYPE */
} sketchssm_state_cache;

/* Quantise the states of sequences seqs[0..n) into cache slots slots[0..n)
 * (DEVICE int32 arrays, 4-byte aligned; any family).  A sequence may be
 * saved to several slots.  The ring must be empty: a tile with buffered
 * entries sets SKSSM_ERRBIT_COUNT and its part of the slot is left as it was
 * (flush it first).  An index out of range sets SKSSM_ERRBIT_SEQ or
 * SKSSM_ERRBIT_SLOT and the entry is skipped; of entries with the same slot
 * the first is taken.  n = 0 launches nothing. */
int sketchssm_state_save(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                         const sketchssm_state_cache* cache, const int32_t* seqs,
                         const int32_t* slots, int32_t n, void* hip_stream);

/* Read cache slots slots[0..n) back into the states of sequences seqs[0..n)
 * (distinct; a slot may be read into several sequences), empty their rings
 * (count 0) and, with prime (0 or 1), write their sketches as
 * sketchssm_prefill does.  Errors as sketchssm_state_save; of entries with
 * the same sequence the first is taken. */
int sketchssm_state_load(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                         const sketchssm_state_cache* cache, const int32_t* seqs,
                         const int32_t* slots, int32_t n, int32_t prime, void* hip_stream);

/* Group norm of rows whose channels come last, with an activation and a gate
 * (what the layers apply to o behind the state read).  For each row and each
 * group of `width` channels, with a = the activation:
 *   x' = gate_first ? x * a(gate) : x       (gate NULL: x' = x)
 *   n  = (x' - mean) / sqrt(var + eps)      (centred 0: mean = 0, var = the mean of squares)
 *   y  = n * weight + bias,  then  y * a(gate) where the gate comes after,
 *        a(y) where there is no gate.
 * Statistics and arithmetic are fp32, rounded once to y. */
typedef struct {
  const void* x;             /* [rows][groups][width] */
  const void* gate;          /* [rows][groups][width], or NULL */
  void* y;                   /* [rows][groups][width]; may be x or gate itself */
  const float* weight;       /* [groups][width], or [width] for every group; NULL: 1 */
  const float* bias;         /* as weight; NULL: 0 */
  int64_t x_stride, gate_stride, y_stride; /* elements from a row to the next: at least a row, at most
                                2^25, a multiple of 16 bytes */
  int64_t rows;
  const int32_t* first;      /* DEVICE, or NULL (0): only the rows from *first ..            */
  const int32_t* end;        /* DEVICE, or NULL (rows): .. up to *end, within [0, rows), are read
                                and written (prompts' seq_start and its last entry) */
  int32_t groups;            /* 1 to 65535 */
  int32_t width;             /* 8 to 8192, a multiple of 8 */
  int32_t dtype;             /* of x, gate and y: SKSSM_F32 or SKSSM_BF16 */
  int32_t group_weights;     /* 1: weight and bias are [groups][width]; 0: [width] */
  int32_t centred;           /* 0 or 1 */
  int32_t activation;        /* SKSSM_ACT_* */
  int32_t gate_first;        /* 0 or 1 */
  float eps;                 /* finite, >= 0 */
} sketchssm_norm;
int sketchssm_group_norm(const sketchssm_norm* norm, void* hip_stream);

/* Prompts of the selective state space scan (SKSSM_MAMBA2): token rows of nseq
 * prompts, one behind the other, as sketchssm_prompts, with the queries and keys of
 * the layer's groups (all strides but dt's a multiple of 16 bytes). */
typedef struct {
  const void* q;             /* [tokens][G][dk] act dtype */
  const void* k;             /* [tokens][G][dk] act dtype */
  const void* v;             /* [tokens][H][dv] act dtype */
  const void* dt;            /* [tokens][H] act dtype, as sketchssm_read takes it; 0 or more */
  void* o;                   /* [tokens][H][dv] act dtype (output); overlaps no input */
  int64_t q_stride, k_stride, v_stride, dt_stride, o_stride;
  int32_t tokens;            /* rows of q, k, v, dt and o */
  int32_t nseq;              /* prompts, at most layer->batch */
  const int32_t* seq_start;  /* as sketchssm_prompts */
  const int32_t* seqs;
  const int32_t* has_state;
  int32_t prime;
  void* work;                /* workspace of sketchssm_scan_workspace_bytes (16-byte aligned; may be
                                NULL when that is 0), overwritten by the call */
  int64_t work_bytes;
} sketchssm_scan_prompts;

/* Prompts through the selective state space scan: for each of a prompt's tokens
 * in order, as sketchssm_full_step,
 *   S <- a S + dt k v^T,  a = exp(-dt exp(A_h)),  o = S^T q,
 * with bufs->A, and, with prime, the sketch that sketchssm_read starts from.  Rings,
 * lists, empty prompts, errors and the workspace as for sketchssm_prefill.  Sums run
 * in fp32, and products are those of fp32 operands; the decays' logarithms are
 * summed in 64 bits.  An infinity or a NaN in a token's row or in the state reaches
 * what the recurrence brings it to (as one or the other) and no earlier token.  (In
 * bf16, terms dt_j (q_i . k_j) v_j of 2^87 and more, and factors q_i . k_j or
 * dt_j (q_i . k_j) of 2^127 and more whatever v_j is, may overflow on the way to an
 * output that they would not.)
 * Other families return SKSSM_EDIM; prime with SKSSM_COEF_STATE is SKSSM_EFLAG. */
int sketchssm_scan(const sketchssm_layer* layer, const sketchssm_buffers* bufs,
                   const sketchssm_scan_prompts* prompts, void* hip_stream);

/* Bytes of prompts->work that sketchssm_scan needs for this many tokens and
 * prompts, or a negative SKSSM_E* code, as sketchssm_prefill_workspace_bytes. */
int64_t sketchssm_scan_workspace_bytes(const sketchssm_layer* layer, int32_t tokens, int32_t nseq);

/* Part of a convolution's channels, written to rows of their own. */
typedef struct {
  void* y;                   /* [tokens][channels of the piece]; overlaps no input and no other piece */
  int64_t y_stride;          /* elements from a token's row to the next: as sketchssm_prompts */
  int32_t channels;          /* 0 (the piece is left out) or more, a multiple of 8 */
  int32_t unit;              /* 0, or the width of the heads that are brought to unit length:
                                16, 64 or 128, of which channels is a multiple */
} sketchssm_conv_piece;

/* The short causal convolution of the rows that a layer's queries, keys and
 * values come from, with the inputs that each sequence holds:
 *   y_t = a(bias + sum_j weight_j x_(t - taps + 1 + j)),  j = 0 .. taps - 1,
 * for each channel, with a = the activation; x before a prompt's first token is what
 * its sequence holds (has_state 0: zeros).  A unit piece's heads are divided by
 * sqrt(sum of their squares + eps) behind the activation.  Afterwards the sequence
 * holds its last taps - 1 inputs.  Sums are fp32, rounded once to y. */
typedef struct {
  const void* x;             /* [tokens][channels] */
  int64_t x_stride;
  const float* weight;       /* [channels][taps]; the last tap is the token's own */
  const float* bias;         /* [channels], or NULL */
  void* state;               /* [batch][taps - 1][channels]: the sequences' last inputs, oldest first */
  sketchssm_conv_piece piece[3]; /* the channels in order, the channels of a row together */
  int32_t taps;              /* 2 to 8 */
  int32_t dtype;             /* of x, y and state: SKSSM_F32 or SKSSM_BF16 */
  int32_t activation;        /* SKSSM_ACT_* */
  float eps;                 /* finite, >= 0 */
  int32_t batch;             /* sequences of state */
  int32_t tokens;            /* rows of x and of the pieces */
  int32_t nseq;              /* prompts, at most batch */
  const int32_t* seq_start;  /* as sketchssm_prompts; NULL: one token to each (tokens = nseq), a decode step */
  const int32_t* seqs;       /* as sketchssm_prompts */
  const int32_t* has_state;  /* as sketchssm_prompts */
  int32_t* err;              /* [1] device error word (SKSSM_ERRBIT_SEQ), never cleared here */
} sketchssm_convolution;

/* Lists and errors as for sketchssm_prefill: a list that falls or leaves [0, tokens]
 * is refused whole, a sequence outside the batch or listed before refuses its
 * prompt; a prompt of no tokens leaves what its sequence holds (has_state 0: zeros).
 * Rows that no prompt holds are neither read nor written. */
int sketchssm_conv(const sketchssm_convolution* conv, void* hip_stream);

/* Selection of beams.  Sequences are in groups of `beams` consecutive ones (a
 * request's beams).  From each group the best `beams` candidates of
 *   score_b + x_bj - log sum_j' exp(x_bj')
 * over its sequences b and the vocabulary j are taken, in falling order of that
 * number, ties to the lowest b * vocab + j.  A logit of minus infinity rules its
 * token out, a score of minus infinity its beam (as the second and further beams of a
 * first step).  An ended beam has one candidate: end_token at its own score.  A NaN or
 * a positive infinity sets SKSSM_ERRBIT_LOGIT and takes its beam out.  Where a group has
 * too few candidates, the places behind them are empty: parent the sequence itself,
 * token -1, score minus infinity, not ended.  Scores are formed in 64 bits from sums
 * of exponentials in fp32, and rounded once. */
typedef struct {
  const void* logits;        /* [groups * beams][vocab], rows at any alignment of an element */
  int64_t stride;            /* elements from a row to the next: at least vocab, at most 2^31 - 1 */
  const float* scores;       /* [groups * beams] sums of the logarithms so far */
  const int32_t* ended;      /* [groups * beams] not 0: the beam has ended; NULL: none has */
  float* new_scores;         /* [groups * beams]; may be scores */
  int32_t* new_ended;        /* [groups * beams]; may be ended.  1 where a parent had ended or the
                                token is end_token */
  int32_t* parents;          /* [groups * beams]: the sequence that each goes on from */
  int32_t* tokens;           /* [groups * beams] */
  int32_t* err;              /* [1] device error word, never cleared here */
  int32_t groups, beams;     /* beams: 1 to 16 */
  int32_t vocab;             /* 1 to 2^24 */
  int32_t dtype;             /* of the logits: SKSSM_F32 or SKSSM_BF16 */
  int32_t end_token;         /* -1 (none) to vocab - 1 */
  void* work;                /* workspace of sketchssm_beam_workspace_bytes (16-byte aligned) */
  int64_t work_bytes;
} sketchssm_beams;
int sketchssm_beam_select(const sketchssm_beams* beams, void* hip_stream);

/* Bytes of beams->work, or a negative SKSSM_E* code. */
int64_t sketchssm_beam_workspace_bytes(int32_t groups, int32_t beams, int32_t vocab, int32_t dtype);

/* Rows of sequences besides a layer's buffers, such as a convolution's state. */
typedef struct {
  void* data;                /* DEVICE [batch] rows, 16-byte aligned */
  int64_t row_bytes;         /* a multiple of 16 */
} sketchssm_rows;

/* Behind a selection of beams: within each group of `beams` (1 to 16) consecutive
 * sequences, sequence b becomes a copy of sequence parents[b] (DEVICE [batch], 4-byte
 * aligned, each within the group) in every buffer of the layer that holds something
 * of a sequence (S, U, the ring with its counts, maps, state copies and factors, as
 * the layer has them) and in nextra (0 to 4) further ones, which overlap neither those
 * nor each other (SKSSM_EINVAL), in place.  A group with a parent outside it sets
 * SKSSM_ERRBIT_SEQ and is left as it is.  layer->batch is a multiple of beams. */
int sketchssm_reorder(const sketchssm_layer* layer, const sketchssm_buffers* bufs, const sketchssm_rows* extra,
                      int32_t nextra, const int32_t* parents, int32_t beams, void* hip_stream);

/* Library version (major * 10000 + minor * 100 + patch). */
int sketchssm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SKETCHSSM_H */
