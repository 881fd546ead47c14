/*
 * specverify_draft.h -- the drafter's side of libspecverify: operators that a
 * user of the verification entry points (specverify.h) needs around them to
 * train a drafter and to draft with it.
 *
 *   sv_teacher_topk              the verifier's rows -> its top logits and the
 *                                mass outside them (a distillation target)
 *   sv_distill_topk              loss of a drafter's rows against such a
 *                                target, and optionally its gradient
 *   sv_distill_topk_backward     the gradient alone, from what the loss kept
 *   sv_beam_select               one step of beam search over beams and
 *                                vocabulary
 *   sv_beam_reorder              the beams' states follow that step
 *
 * The nearer a drafter's q lies to the verifier's p, the larger the acceptance
 * rate sum_v min(p(v), q(v)); the beams' tokens are deterministic drafts,
 * which the point-mass entry points (sv_verify_chain_pm, sv_verify_tree_pm)
 * accept without loss.
 *
 * The conventions of specverify.h hold: device pointers owned by the caller,
 * the caller's workspace (of the same layout, so one workspace serves every
 * entry point of both headers, one call at a time) and stream, asynchronous
 * calls that allocate nothing and may be captured in a graph, argument checks
 * on the host before anything is enqueued, input errors found on the device as
 * bits of the workspace's error word.  Logit rows are SV_BF16 or SV_F32, unit
 * stride along V, 16-byte aligned rows; -inf logits mean probability 0; NaN
 * and +inf are outside the contract.  Results do not depend on the launch's
 * timing: the same call gives the same bits.
 *
 * Calls that overlap in time (two streams, two captured graphs that may be
 * replayed together) need a workspace each; a captured graph needs the one of
 * its capture for as long as it is replayed.
 */
#ifndef SPECVERIFY_DRAFT_H
#define SPECVERIFY_DRAFT_H

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t sv_draft_op;
enum {
  SV_DRAFT_TEACHER = 0,
  SV_DRAFT_DISTILL = 1,   /* sv_distill_topk and sv_distill_topk_backward */
  SV_DRAFT_BEAM = 2,
  SV_DRAFT_REORDER = 3
};

#define SV_MAX_TEACHER 256     /* teacher tokens per row of a distillation call */
#define SV_MAX_ROWS 65536      /* rows (teacher, distillation) per call; B * W of a beam call */
#define SV_MAX_BEAMS 64        /* beams per sequence */

/* Device error-word bit of these entry points, beside SV_DERR_TOKEN and
 * SV_DERR_ROW. */
#define SV_DERR_RANGE 32       /* a parent beam or a length out of range */

/*
 * Workspace bytes for one call.  `rows` is R (teacher, distillation) or B
 * (beam select); W the beams per sequence (beam select); k the teacher's
 * tokens per row or, for beam select, N.  SV_DRAFT_REORDER takes the fixed
 * part only and reads none of the sizes.  SV_EINVAL / SV_EUNSUPPORTED for
 * shapes that the call would reject.
 */
sv_status sv_draft_workspace_size(sv_draft_op op, sv_dtype dt, int32_t rows, int32_t W, int32_t V, int32_t k,
                                  size_t* bytes);

/*
 * The k largest logits of each row, ordered by value descending and index
 * ascending on ties (the fan-out's order), and the logarithm of the mass they
 * leave: rest = log sum over the other v of exp(z_v / T).
 *   logits [R, V]; 1 <= k <= SV_MAX_FANOUT
 *   out_ids [R, k] (-1 padded where k > V), out_vals [R, k] raw logits (-inf
 *   padded), out_rest [R] (natural logarithm; -inf if nothing is left)
 * The teacher's probabilities at temperature T follow from these alone:
 * p_i = exp(vals_i / T) / Z with Z = sum_i exp(vals_i / T) + exp(rest).  The
 * mass outside is summed by itself, never as a difference, so it keeps its
 * digits where the top tokens hold nearly everything.
 *
 * Streams each row once and reads parts of it again, each by the wave of 64
 * threads that owns it (a thread owns every 256th or 512th 16-byte vector):
 * the vectors of a thread that holds more than one value near the k-th best;
 * of those the ones with listed values once more; all of these if more than
 * 512 values pass for the k best at first; and the wave's whole share where
 * the values it sums lie too far apart (2^100 in exp(z / T)) or their sum is
 * small against what the list took out of it.  Unordered rows of 128256 bf16
 * logits read 2% again for 16 values, 26% for 64.
 */
sv_status sv_teacher_topk(const void* logits, sv_dtype dt, int64_t stride, int32_t R, int32_t V, int32_t k, float T,
                          int32_t* out_ids, float* out_vals, float* out_rest, void* ws, size_t ws_bytes, void* stream);

/*
 * Distillation from a teacher's top logits: the Kullback-Leibler divergence
 * KL(p || q) of the drafter's q = softmax(z / T) over the teacher's k tokens I
 * and one class for all others,
 *   loss = sum_{i in I} p_i log(p_i / q_i) + p_0 log(p_0 / q_0),
 *   q_0 = sum_{v not in I} q_v,
 * with p_i, p_0 as at sv_teacher_topk (p_0 = exp(rest) / Z).  Its gradient is
 *   dz_v = (g / T) (q_v - p_v)                 v in I
 *   dz_v = (g / T) q_v (1 - p_0 / q_0)         otherwise.
 * Without `rest` (NULL) p_0 = 0: the teacher is renormalised over I and every
 * other token's q counts against the loss.
 *   z [R, V] the drafter's logits
 *   t_ids [R, k], t_vals [R, k] (values at which exp(t / T) is meant: logits,
 *     or log-probabilities times T), t_rest [R] or NULL; 1 <= k <=
 *     SV_MAX_TEACHER.  An id of -1 is absent.  An id outside [-1, V) or one
 *     that stands in its row already sets SV_DERR_TOKEN and counts as absent.
 *   grad_loss [R] the loss's upstream gradient g, or NULL (all 1)
 * A row without teacher mass (no id with a value above -inf, rest NULL or
 * -inf), as padding has it, may hold anything: loss, stat and gradient are 0.  A row
 * with teacher mass and no finite logit sets SV_DERR_ROW and gives the same
 * zeros.  A token with p_i > 0 and q_i = 0 makes the loss +inf; its gradient
 * is finite (q_i - p_i), and so is that of the others (q_v / q_0 is formed
 * without q_0, which may underflow; where every logit outside I is -inf their
 * gradient is 0).
 * Outputs:
 *   out_loss [R]
 *   out_stat [R, 4] what the backward pass needs: m, the row's largest logit;
 *     s = sum_v exp((z_v - m) / T); and m_0, s_0, the same of the tokens
 *     outside I (-inf and 0 if there are none)
 *   out_grad [R, V] of z's type, or NULL: loss only.  Its rows are like z's
 *     (grad_stride >= V, 16-byte aligned); it may be z itself (the same
 *     pointer and stride: the gradient takes the logits' place) but must not
 *     overlap z otherwise.  What lies between the rows is not written.
 * Reads each row once for the loss; with the gradient, rows of up to 196608
 * bf16 or 98304 fp32 logits once in all, longer ones (and up to some 100 rows
 * of more than 80000 or 52000) twice.  The gradient of a row may therefore
 * differ in its last bits between calls with different numbers of rows.
 */
sv_status sv_distill_topk(const void* z, sv_dtype dt, int64_t stride, int32_t R, int32_t V, const int32_t* t_ids,
                          const float* t_vals, const float* t_rest, int32_t k, float T, const float* grad_loss,
                          float* out_loss, float* out_stat, void* out_grad, int64_t grad_stride, void* ws,
                          size_t ws_bytes, void* stream);

/*
 * The gradient of sv_distill_topk from the out_stat of a call with the same
 * z, teacher and T (rows whose s is 0 give 0).  out_grad as there; with
 * out_grad = z the logits are overwritten, so it is the last reader of them.
 */
sv_status sv_distill_topk_backward(const void* z, sv_dtype dt, int64_t stride, int32_t R, int32_t V,
                                   const int32_t* t_ids, const float* t_vals, const float* t_rest, int32_t k, float T,
                                   const float* stat, const float* grad_loss, void* out_grad, int64_t grad_stride,
                                   void* ws, size_t ws_bytes, void* stream);

/*
 * One step of beam search: of all continuations (w, v) of a sequence's beams,
 * the N with the largest score
 *   scores[b, w] + z_{w,v} / T - log sum_u exp(z_{w,u} / T),
 * ordered by score descending, then w ascending; within a beam by logit
 * descending, then v ascending (so also where the scores' rounding makes
 * different logits equal: a beam at -1e30 continues with its best tokens).
 *   logits [B, W, V], row (b, w) at b*W + w; 1 <= W <= SV_MAX_BEAMS
 *   scores [B, W] the beams' log-probabilities; a beam at -inf has no
 *     continuation (at the first step all but one)
 *   finished [B, W] int32 or NULL: a beam with a non-zero flag has one
 *     continuation, pad_tok, at its own score
 *   1 <= N <= SV_MAX_FANOUT
 * Outputs: out_beam, out_tok [B, N] (-1 padded), out_score [B, N] (-inf
 *   padded): fewer than N where fewer have a score above -inf.
 * Scores are formed and compared in 64 bits.  A row's logarithm is that of a
 * sum of 32-bit exponentials, within 1e-5 of the exact one and mostly within
 * 2e-7: beams of the same row and score tie, continuations of different beams
 * whose scores are nearer than that may change places.  A live row without a
 * finite logit sets SV_DERR_ROW and has no continuation.  Rows of dead and
 * finished beams are not read, the others as by sv_teacher_topk.
 */
sv_status sv_beam_select(const void* logits, sv_dtype dt, int64_t stride, const float* scores, const int32_t* finished,
                         int32_t B, int32_t W, int32_t V, float T, int32_t pad_tok, int32_t N, int32_t* out_beam,
                         int32_t* out_tok, float* out_score, void* ws, size_t ws_bytes, void* stream);

/*
 * The beams' states follow a selection: for every layer l, sequence b, beam n
 * with parent w = parent[b, n], segment h (a head, say),
 *   dst[l, b, n, h, 0 .. len_b) = src[l, b, w, h, 0 .. len_b)
 * in units of positions of pos_bytes bytes.  lens [B] int32 or NULL (every
 * position up to S); what lies behind a sequence's length is left as it was.
 *   src [L, B, W, H, S], dst [L, B, N, H, S]; positions of a segment are
 *     adjacent; the other strides are in bytes: src_stride / dst_stride point
 *     to 4 host values (layer, sequence, beam, segment)
 *   parent [B, N]: -1 leaves a beam's state as it is
 * dst may be src (the same pointer and strides, N <= W): the call then works
 * in place, and a beam that follows itself costs nothing.  Otherwise they must
 * not overlap, first byte to last.  What is written (in place: all W beams'
 * states) must not overlap itself, and its strides must nest: each at least
 * what the smaller ones span.  SV_EINVAL otherwise.
 * A parent outside [-1, W) or a length outside [0, S] sets SV_DERR_RANGE; that
 * beam, or that whole sequence, is left as it was.  Any alignment is taken.
 * One beam's states hold fewer than 2^32 places of 16 bytes (8 or 4 where more than
 * 16 or 32 beams move in place; every segment takes multiples of 256 places);
 * SV_EUNSUPPORTED beyond.
 */
sv_status sv_beam_reorder(const void* src, const int64_t* src_stride, void* dst, const int64_t* dst_stride,
                          const int32_t* parent, const int32_t* lens, int32_t L, int32_t B, int32_t W, int32_t N,
                          int32_t H, int64_t S, int64_t pos_bytes, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_DRAFT_H */
