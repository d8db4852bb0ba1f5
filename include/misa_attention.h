/*
 * misa_attention.h -- C ABI of the attention side of libmisa (B200, sm_100a):
 * what a program does with the tokens that the indexer of misa.h selected.
 *
 *   misa_rope_phases, misa_apply_rope   rotary positions of index queries and
 *                                       keys, attention queries and keys
 *   misa_append_kv                      the attention cache written (rotated
 *                                       and quantised) as tokens arrive
 *   misa_read_kv                        that cache read back at listed tokens
 *   misa_attend                         attention over each query's selected
 *                                       tokens or its whole prefix, with a
 *                                       tree of drafted tokens behind it
 *
 * The pages behind misa.h describe the selection only ("the top-k tokens go
 * to the main attention"); the operations here have no counterpart there and
 * are written from their formulas, given at each declaration.
 *
 * Conventions are those of misa.h: device memory owned by the caller, no
 * allocation, calls asynchronous on `stream`, arguments validated on the host
 * before any launch, MISA_ERR_* statuses with misa_last_error(),
 * MISA_DEV_* bits OR-ed into the cache's status word for what only the device
 * sees, misa_debug_fail_next for injected failures.  A workspace may be used
 * by one call at a time: calls in stream order (graphs replayed on one stream
 * among them) may share one, calls that can overlap need one each.
 */
#ifndef MISA_ATTENTION_H
#define MISA_ATTENTION_H

#include "misa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MISA_MAX_DRAFT 1024      /* drafted tokens per sequence */
#define MISA_MAX_ROPE_GROUPS 4   /* tensors rotated by one misa_apply_rope call */

/*
 * Attention cache of n_seq sequences.
 *   k, v     [n_seq][L_cap][H_kv][d]  bf16 bit patterns or e4m3 codes, 16-byte
 *                                     aligned
 *   k_scale, v_scale [n_seq][L_cap][H_kv] fp32 dequantisation scales of 0 to
 *                                     2^100 of each row of d elements; NULL for bf16,
 *                                     non-NULL for e4m3
 *   seq_len  [n_seq]                  int32 committed tokens per sequence
 *   status   [1] uint32 or NULL       device error bits (MISA_DEV_*)
 * dtype is a misa_key_dtype.  Supported: d = 64 or 128, 1 <= H_kv <= 128,
 * L_cap <= MISA_MAX_L.  Keys and values have the same width d: a cache of one
 * latent row per token, whose values are a part of wider keys, is not supported.
 */
typedef struct {
  void *k;
  void *v;
  float *k_scale;
  float *v_scale;
  int32_t *seq_len;
  uint32_t *status;
  int32_t n_seq;
  int32_t L_cap;
  int32_t H_kv;
  int32_t d;
  int32_t dtype;
} misa_kv;

/*
 * Rotary positions.  The rot elements from `first` on of a row form rot/2
 * pairs (a, b); at position p pair i becomes
 *     (amplitude * (a cos t - b sin t), amplitude * (b cos t + a sin t)),
 *     t = 2 pi * p * phase[i] / 2^64,
 * in fp32, rounded once to the output's type.  The other elements are kept.
 *   phase  [rot/2] uint64, device memory (misa_rope_phases fills a host array).
 *          The product p * phase[i] wraps modulo 2^64, that is modulo whole
 *          turns, and its fraction of a turn is rounded to fp32: an angle is
 *          off by at most 2^-26 turns, at every position.
 *   layout MISA_ROPE_HALF: pair i = elements (first + i, first + rot/2 + i);
 *          MISA_ROPE_INTERLEAVED: (first + 2i, first + 2i + 1).
 */
#define MISA_ROPE_HALF 0
#define MISA_ROPE_INTERLEAVED 1
typedef struct {
  const uint64_t *phase;
  int32_t rot;
  int32_t first;
  int32_t layout;
  float amplitude;
} misa_rope;

/*
 * Phase increments of misa_rope from the usual parameters (host only, `phases`
 * is HOST memory).  f_i = base^(-2i/rot) radians per position, then
 *   MISA_ROPE_NONE    f_i
 *   MISA_ROPE_LINEAR  f_i / factor (positions interpolated)
 *   MISA_ROPE_NTK     f_i of base * factor^(rot/(rot-2))
 *   MISA_ROPE_YARN    f_i (1 - r_i) + (f_i / factor) r_i with the ramp r_i from
 *                     0 at the pair that turns beta_fast times in orig_len
 *                     positions to 1 at the one that turns beta_slow times
 *                     (both rounded outwards to whole pairs)
 * Errors: MISA_ERR_INVALID for a NULL array, rot odd or < 2, base <= 0 or not
 * finite, factor or orig_len not positive where used, beta_fast < beta_slow
 * or either not positive, an unknown scaling.
 */
#define MISA_ROPE_NONE 0
#define MISA_ROPE_LINEAR 1
#define MISA_ROPE_NTK 2
#define MISA_ROPE_YARN 3
MISA_API misa_status misa_rope_phases(uint64_t *phases, int32_t rot, double base, int32_t scaling, double factor,
                                      double orig_len, double beta_fast, double beta_slow);

/*
 * A tensor of rows to rotate: x and y are bf16 bit patterns [n][H][d] with the
 * given strides in elements between rows and between heads (the d elements of
 * a head are consecutive); pos [n] int32, any value, is each row's position.
 * y may be x with equal strides (in place); other overlaps are refused: rows of
 * y that share memory with one another, with rows of x or with another group's
 * rows.  Interleaved slices of one projection do not.
 */
typedef struct {
  const uint16_t *x;
  uint16_t *y;
  const int32_t *pos;
  int64_t x_row, x_head;
  int64_t y_row, y_head;
  int32_t n;
  int32_t H;
  int32_t d;
} misa_rope_rows;

/*
 * Rotate up to MISA_MAX_ROPE_GROUPS tensors in one launch (a step's index
 * queries, its new index keys, its attention queries).  Rows that start on 16
 * bytes with rot a multiple of 16 and first and d multiples of 8 go through
 * 16-byte accesses; others are handled element by element.
 * Errors: MISA_ERR_INVALID for n or H < 0, rot odd or outside [2, d - first],
 * first < 0, an unknown layout, a non-finite amplitude, a group count outside
 * [1, MISA_MAX_ROPE_GROUPS], and in groups that have rows NULL pointers, in place
 * with other strides, rows of y whose strides let them meet, or that share
 * memory with rows of x or of another group; MISA_ERR_UNSUPPORTED for d > 1024.
 */
MISA_API misa_status misa_apply_rope(const misa_rope *rope, const misa_rope_rows *groups, int32_t n_groups,
                                     misa_stream stream);

/*
 * New keys and values: bf16 bit patterns [n_seq][count][H_kv][d] with the
 * given strides in elements (the d elements of a head are consecutive; every
 * row starts on 16 bytes).  They may be slices of a fused projection.
 */
typedef struct {
  const uint16_t *k;
  const uint16_t *v;
  int64_t k_seq, k_tok, k_head;
  int64_t v_seq, v_tok, v_head;
} misa_new_kv;

/*
 * Write `count` new tokens per sequence in one pass.  For every s with
 * new_pos[s] >= 0, token j goes to position new_pos[s] + j: its key rows are
 * rotated (rope non-NULL) by rope_pos[s][j] ([n_seq][count] int32), or by the
 * position written when rope_pos is NULL.  Into an e4m3 cache each row x of d
 * elements is written as
 *     scale = amax_e |x_e| / 448   (1 for a row of zeros),
 *     code_e = e4m3(x_e / scale)   rounded to nearest even, saturated,
 * in fp32 with IEEE division (the rotated key is not rounded before); into a
 * bf16 cache rounded once.  commit != 0 sets seq_len[s] = new_pos[s] + count;
 * with commit 0 (drafted tokens) seq_len stays.  new_pos[s] < 0 leaves
 * sequence s untouched; a write past L_cap skips the sequence and sets
 * MISA_DEV_APPEND_RANGE.  Writing the same rows again is idempotent, so the
 * drafted tokens that are accepted are written again at their places.
 * new_pos may be seq_len itself (the tokens go behind what is there); it is
 * then updated by a second launch, after the write that reads it.
 * A row that holds a NaN or infinity keeps it as far as its type can (NaN
 * codes in e4m3).
 * Errors: those of the cache and rope; MISA_ERR_INVALID for count < 1 or
 * above L_cap, NULL new_kv/k/v/new_pos, rows not on 16 bytes (pointers, and
 * strides not multiples of 8), commit with a new_pos that overlaps seq_len
 * without being it.
 */
MISA_API misa_status misa_append_kv(const misa_kv *kv, const misa_new_kv *new_kv, const int32_t *new_pos,
                                    int32_t count, const misa_rope *rope, const int32_t *rope_pos, int32_t commit,
                                    misa_stream stream);

/*
 * Read rows back: k_out[i][j] = the dequantised key rows [H_kv][d] of token
 * tok[i][j] of sequence seq[i], rounded once to bf16; v_out the values.
 *   seq [n] int32, tok [n][k] int32 (-1 entries give rows of zeros; so do
 *   tokens outside [0, L_cap) and sequences outside the cache, which set
 *   MISA_DEV_BAD_POSITION)
 *   k_out, v_out [n][k][H_kv][d] bf16 bit patterns, 16-byte aligned; one of
 *   them may be NULL
 * Tokens at and beyond seq_len (drafted ones) are read as they are.
 * Errors: those of the cache; MISA_ERR_INVALID for n < 0, k < 1, (n > 0) NULL seq
 * or tok, both outputs NULL or overlapping; MISA_ERR_UNSUPPORTED for k >
 * MISA_MAX_L.
 */
MISA_API misa_status misa_read_kv(const misa_kv *kv, const int32_t *seq, const int32_t *tok, int32_t n, int32_t k,
                                  uint16_t *k_out, uint16_t *v_out, misa_stream stream);

/*
 * Attention queries.
 *   q     [n_q][H][d] bf16 bit patterns, 16-byte aligned; H a multiple of the
 *         cache's H_kv, head j reads key/value head j / (H / H_kv)
 *   q_seq [n_q] int32 sequence of each query
 *   q_pos [n_q] int32 last position of its prefix 0..q_pos (-1: none)
 *   scale factor of q . k (normally 1 / sqrt(d))
 * Queries of one sequence should be adjacent: without a list they share the
 * reads of its tokens.
 */
typedef struct {
  const uint16_t *q;
  const int32_t *q_seq;
  const int32_t *q_pos;
  int32_t n_q;
  int32_t H;
  float scale;
} misa_attend_queries;

/*
 * Drafted tokens: slot j (0 <= j < n <= MISA_MAX_DRAFT) of sequence s sits in
 * the cache at position start[s] + j (written with misa_append_kv, commit 0).
 *   start [n_seq] int32
 *   mask  [n_q][ceil(n/32)] uint32: bit j % 32 of word j / 32 says whether the
 *         query sees slot j.  A node of a tree sets itself and its ancestors.
 * Slots should lie behind the query's prefix (a token inside both counts
 * twice).  Slots outside [0, L_cap) are not seen and, where a mask asks for
 * one, set MISA_DEV_BAD_POSITION.
 */
typedef struct {
  const int32_t *start;
  const uint32_t *mask;
  int32_t n;
} misa_draft;

/*
 * Attention of every query and head over the tokens T_i that the query sees:
 *     s_t = scale * q . k_t,   out = sum_t exp(s_t) v_t / sum_t exp(s_t),
 *     lse = ln sum_t exp(s_t)
 * with T_i = the query's list, or its prefix when topk is NULL, together with
 * the drafted slots of its mask (draft non-NULL).
 *   topk [n_q][k] int32, as the top-k calls of misa.h write it (any order;
 *        -1 entries and tokens outside the query's prefix are ignored; a
 *        token listed twice counts twice), or NULL with k = 0
 *   out  [n_q][H][d] bf16 bit patterns, 16-byte aligned
 *   lse  [n_q][H] fp32 or NULL
 * A query that sees nothing gets out = 0 and lse = -inf.  What a query does
 * not see does not reach its output, be it NaN or infinite.  A query whose
 * sequence or position is outside the cache gets nothing or the clamped
 * prefix and sets MISA_DEV_BAD_POSITION.
 * Numbers: products of the stored values with fp32 sums; softmax statistics
 * in fp32.  bf16 caches: the weights exp(s_t - ref), ref a running maximum of
 * s_t, are rounded to bf16 before they meet the values.  e4m3 caches: the
 * codes are exact in f16; each row of q is scaled by a power of two of its own
 * (elements down to 2^-23 of the row's largest stay exact) and
 * exp(s_t - ref) v_scale_t, ref 7 ln 2 below a running maximum of
 * s_t + ln v_scale_t (v_scale_t held within 2^-93 and 2^100 there), is rounded to
 * f16: contributions below 2^-21 of a row's largest are off by up to 2^-32 of it.
 * Workspace: misa_attend_workspace_bytes(kv, qs, k, draft ? draft->n : 0),
 * 16-byte aligned.  Results do not depend on what it held.
 * Errors: those of the cache; MISA_ERR_INVALID for n_q outside [0, 65535], H not
 * a positive multiple of H_kv, a non-finite scale, k < 1 with a list, a draft of
 * n < 1, and with n_q > 0 NULL q/q_seq/q_pos/out, k != 0 without a list, a draft
 * with NULL pointers, out, lse or the workspace that overlap one another or q;
 * MISA_ERR_UNSUPPORTED for H > MISA_MAX_H, k > MISA_MAX_L, draft->n
 * > MISA_MAX_DRAFT; MISA_ERR_WORKSPACE for a short workspace.
 */
MISA_API misa_status misa_attend(const misa_kv *kv, const misa_attend_queries *qs, const int32_t *topk, int32_t k,
                                 const misa_draft *draft, uint16_t *out, float *lse, void *ws, size_t ws_bytes,
                                 misa_stream stream);

/* Workspace bytes of misa_attend for these shapes (0 may be the need; also 0
 * on invalid arguments).  Host-only, launches nothing. */
MISA_API size_t misa_attend_workspace_bytes(const misa_kv *kv, const misa_attend_queries *qs, int32_t k,
                                            int32_t n_draft);

#ifdef __cplusplus
}
#endif

#endif /* MISA_ATTENTION_H */
