/*
 * orpo_decode.h — C ABI of one beam-search step on the quantised head, for one GB300 GPU (sm_103a).
 *
 * The pairs the head trains on are responses that were generated; on-policy pairs come from the
 * same head, in the same quantised format.  These entry points are that other direction, one
 * decode step in three calls on one stream:
 *
 *   orpo_head_logits_q   logits of a few rows of h (the beams' last positions) out of the
 *                        affine group-quantised head that orpo_head_fwd_q reads
 *   orpo_beam_select     log-softmax over the vocabulary and the n best continuations over
 *                        beams x vocabulary, per batch entry
 *   orpo_beam_reorder    the beams' states (key/value caches, recurrent states) follow their
 *                        parents, in place
 *
 * The mlx-bun documentation pages leave generation out ("Training — design" starts from given
 * chosen / rejected responses); the weight format and the softcap are those of their head (§5.1
 * tier 4), the rest is the textbook definition written out below.
 *
 * Conventions are those of orpo_head.h: device pointers, caller-owned buffers and workspace, no
 * allocation, asynchronous and stream-ordered calls, ORPO_ERR_* return codes before any launch,
 * ORPO_STATUS_* bits OR-ed into the device word `status`, capturable in a CUDA graph.  A call
 * whose sizes make it empty (M, batch, outer ... = 0) launches nothing.
 */
#ifndef ORPO_DECODE_H
#define ORPO_DECODE_H

#include "orpo_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most beams per batch entry, and most continuations selected per batch entry. */
#define ORPO_MAX_BEAMS 64
#define ORPO_MAX_SELECT 64

/*
 * Logits of M rows under the quantised head.
 *   W[v, j] = bf16(scales[v, j/group] * q[v, j] + biases[v, j/group]), product and sum rounded once.  (orpo_head_fwd_q
 *   rounds to fp32 and then to bf16: its weights are these but where the exact value lies within fp32's rounding
 *   of the middle between two bf16 values, and there one bf16 unit off at most.)
 *   z[m, v] = sum_j h[m, j] W[v, j]       (products of bf16 values, fp32 accumulation: the tensor core's adds truncate
 *   within 512 columns, and those sums are added with rounding; off by about 3e-7 of the largest logit)
 *   logits[m, v] = softcap * tanh(z / softcap) if softcap > 0, else z; rounded once when bf16
 * h: bf16 [M, d], rows ld_h elements apart (ld_h >= d, a multiple of 8; e.g. the last positions of
 * [M, T, d] hidden states are h + (T-1) d with ld_h = T d), 16-byte aligned.  wq, scales, biases,
 * bits, group: as for orpo_head_fwd_q.  logits: fp32 (logits_bf16 = 0, 4-byte aligned) or bf16
 * (logits_bf16 = 1, 2-byte aligned), rows ld_logits >= V elements apart; columns V .. ld_logits-1
 * are not touched.  Each row depends on its own row of h only: infinities and NaN go into that
 * row's logits and no other.  The sum's order depends on the sizes alone, so results repeat bit
 * for bit.
 * Meant for few rows: the quantised weights are read once per 64 rows of h.
 * Workspace: orpo_head_logits_q_workspace_bytes(M, d, bits) bytes, 16-byte aligned; 0 (workspace may be
 * NULL) where h fits on chip (up to 16 rows of d <= 3328, 32 of d <= 1536, 64 or passes of 64 of d <= 768), else
 * about 2 M d: a copy of h in the order the kernel takes it.
 * Limits: 0 <= M <= 2^31 - 2^16, 1 <= V <= 2^31 - 2^16, 8 <= d < 2^20, d a multiple of 8.
 */
size_t orpo_head_logits_q_workspace_bytes(int64_t M, int64_t d, int bits);
int orpo_head_logits_q(const void* h_bf16, int64_t ld_h, const uint8_t* wq, const void* scales_bf16,
                       const void* biases_bf16, int bits, int group, int64_t M, int64_t V, int64_t d,
                       float softcap, void* logits, int64_t ld_logits, int logits_bf16,
                       void* workspace, size_t ws_bytes, int32_t* status, void* stream);

/*
 * The n best continuations of each of `batch` entries with `beams` beams.
 * Row r = b * beams + k of logits (fp32, or bf16 when logits_bf16 = 1; rows ld_logits >= V elements
 * apart) belongs to beam k of entry b, whose score (sum of log-probabilities so far) is score[r].
 *   lse_r = log sum_v exp(x[r, v]);   value(k, v) = score[r] + (x[r, v] - lse_r)   in fp32, with lse_r as m + log s
 *   (m the row's largest logit, s = sum exp(x - m)) and the value as score + ((x - m) - log s),
 *   and value = -inf where x[r, v] = -inf, where lse_r is not finite (every logit masked, or one
 *   is +inf) or where score[r] is NaN.  A NaN logit counts as -inf.
 * A live beam proposes its n largest logits, the lowest token first among equal ones.  A beam with
 * finished[r] != 0 proposes token eos at its own score, then n - 1 times eos at -inf; its logits
 * are not read.  (finished = NULL: every beam is live.)
 * Of the beams * n proposals, the n of greatest value are written in descending order; among equal
 * values the lower beam comes first, and within a beam its own order holds.
 *   out_score  fp32  [batch, n]  value
 *   out_parent int32 [batch, n]  beam within the entry, 0 .. beams-1
 *   out_token  int32 [batch, n]
 *   out_finished uint8 [batch, n] (may be NULL): 1 where the parent was finished or token == eos
 * When n == beams, out_score may be score itself and out_finished may be finished itself.
 * eos: a token in [0, V), or -1 for none (finished must then be NULL).
 * Device errors: ORPO_STATUS_NONFINITE (a NaN or +inf logit of a live beam, or a NaN score; masked
 * logits, -inf or any finite value, are no error; -inf is the cheap one, a finite value on all but a few tokens costs
 * about ten times as much).
 * Results do not depend on run-to-run scheduling.
 * Limits: batch >= 0, 1 <= beams <= ORPO_MAX_BEAMS, 1 <= n <= min(ORPO_MAX_SELECT, V),
 * batch * beams <= 2^20, V <= 2^31 - 2^16.  The workspace (16-byte aligned) must hold
 * orpo_beam_select_workspace_bytes(batch, beams, V, n), which is never more than
 * 16 * batch * beams * (n + 1) * ceil(V / 1024) + 4096; 0 for invalid sizes.
 */
size_t orpo_beam_select_workspace_bytes(int64_t batch, int beams, int64_t V, int n);
int orpo_beam_select(const void* logits, int64_t ld_logits, int logits_bf16, const float* score,
                     const uint8_t* finished, int32_t eos, int64_t batch, int beams, int64_t V, int n,
                     float* out_score, int32_t* out_parent, int32_t* out_token, uint8_t* out_finished,
                     void* workspace, size_t ws_bytes, int32_t* status, void* stream);

/*
 * Reorder per-beam states by parent, in place, as if every beam's state were read before any is
 * written:
 *   state[o, b * beams + k, r, t, :] <- state[o, b * beams + parent[b, k], r, t, :],  t < length[b]
 * state: contiguous bytes [outer, batch * beams, rows, capacity, unit_bytes] of any element type:
 * e.g. outer = 2 * layers, rows = heads, capacity = positions allocated, unit_bytes = head size *
 * element size.  length: int32 [batch], positions in use, 0 .. capacity (NULL: all of them);
 * positions from length[b] on keep what they hold.  parent: int32, rows ld_parent >= beams
 * elements apart, so the first `beams` columns of orpo_beam_select's [batch, n] output serve as
 * they are.  A beam that is its own parent is not written, and only parents of others are read.
 * Device errors: ORPO_STATUS_PARENT (a parent outside [0, beams) or a length outside [0, capacity];
 * that entry's state is left as it is).
 * Limits: 1 <= beams <= ORPO_MAX_BEAMS; outer, batch, rows, capacity, unit_bytes >= 0, batch * rows
 * <= 2^30 and the state's size in bytes below 2^62.
 */
int orpo_beam_reorder(void* state, const int32_t* parent, int64_t ld_parent, const int32_t* length,
                      int64_t outer, int64_t batch, int beams, int64_t rows, int64_t capacity,
                      int64_t unit_bytes, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ORPO_DECODE_H */
