/*
 * moe_learner.h -- C ABI of the operators a learner needs around the expert
 * layer of moe_nvfp4.h, in the same library (libmoe_nvfp4.so):
 *
 *   - in front of the layer, the residual add + RMS norm, whose BF16 output
 *     feeds the router and the experts and whose 8-bit output feeds dense
 *     block-scaled products (forward and backward);
 *   - behind the last layer, the token losses on the logits: log-probabilities
 *     of given tokens with entropy and top alternatives, and distillation from
 *     a teacher's top logits (forward, backward, and the distillation step in
 *     one call).
 *
 * Conventions are those of moe_nvfp4.h: device pointers owned by the caller,
 * every call enqueued on `stream`, no allocation, no synchronisation, return
 * codes checked on the host before anything is enqueued, `status` an optional
 * device int that receives MOE_STATUS_* bits, results deterministic bit for
 * bit.  Host threads may call them at the same time.  Differences:
 *   - logits and their gradients need only the alignment of their element
 *     (rows of any length and stride); every other 16-bit and byte tensor is
 *     16-byte aligned, int32 and float vectors 4-byte aligned (the stats of
 *     moe_distill_topk, rows of four floats, 16-byte aligned);
 *   - logits are MOE_DTYPE_BF16 or MOE_DTYPE_F32; all statistics and sums are
 *     FP32, the softmax statistics held about the row's maximum.
 * Strides are in elements; T times a stride stays below 2^46.
 * MOE_ERR_SHAPE is also returned for a size or a number outside the limits an
 * entry point states.  T = 0 does nothing (moe_add_rmsnorm_backward: dw = 0).
 */
#ifndef MOE_LEARNER_H
#define MOE_LEARNER_H

#include "moe_nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_F32  1

/* device status bit (others: moe_nvfp4.h) */
#define MOE_STATUS_BAD_TOKEN 0x20 /* a token id >= V, or listed twice for a row */

#define MOE_LOGPROBS_MAX_TOP 32   /* most alternatives per row */
#define MOE_DISTILL_MAX_K    256  /* most teacher entries per row */
#define MOE_DISTILL_MAX_V    (1 << 20)

/* ---------------------------------------------------------------------- */
/* Residual add + RMS norm.                                                 */
/* ---------------------------------------------------------------------- */

/* Bytes of the scale buffer of `rows` rows of d 8-bit values (one byte per 32
 * values in the 128 x 4 tile layout of moe_nvfp4.h, kgroups = d/128); 0 where
 * d % 128 != 0. */
size_t moe_mx8_sf_bytes(int64_t rows, int d);

/* h = BF16(x + res);  rstd = 1 / sqrt(mean_i h_i^2 + eps);  y_i = h_i rstd w_i
 * in FP32 from the rounded h (the value that the residual stream keeps and
 * the backward reads), rounded once to each output:
 *   x     bf16 [T] rows ldx elements apart
 *   res   bf16 [T] rows ldr apart, or NULL: h = x, and then h may be NULL
 *   w     bf16 [d]
 *   h     bf16 [T][d] (out); may be x or res itself where that is contiguous
 *   y     bf16 [T][d] (out), or NULL
 *   y8    u8 [T][d] E4M3 codes (out), y8_sf moe_mx8_sf_bytes(T, d) scale
 *         bytes (out), or both NULL.  The scale of 32 consecutive values is
 *         2^(byte - 127), the smallest power of two with max|y_i| / scale <=
 *         448 (byte 0 at least), and a code is E4M3_RNE(y_i / scale): no value
 *         saturates.  Scale bytes of rows >= T are untouched.
 *   rstd  f32 [T] (out), or NULL
 * Needs d % 16 == 0 (y8: d % 128 == 0), 16 <= d <= 16384, ldx, ldr >= d and
 * multiples of 8, 0 <= eps <= 1e30.  Non-finite values of h set
 * MOE_STATUS_NONFINITE_X (the row's outputs are then unspecified).  The sum of
 * squares is FP32: rows whose sum exceeds its range (|h| about 1e18 and more)
 * give y = 0; with eps = 0, rows whose squares all underflow (|h| below about
 * 1e-23) give infinities, and NaN for their zeros.  One launch. */
int moe_add_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* res,
                    int64_t ldr, const uint16_t* w, float eps, int T, int d,
                    uint16_t* h, uint16_t* y, uint8_t* y8, uint8_t* y8_sf,
                    float* rstd, int* status, void* stream);

/* Workspace of moe_add_rmsnorm_backward: the per-block parts of dw. */
size_t moe_add_rmsnorm_backward_workspace_bytes(int T, int d);

/* The gradients of moe_add_rmsnorm, with n_i = h_i rstd:
 *   dx_i = rstd (dy_i w_i - n_i mean_j(dy_j w_j n_j)) + dh_i
 *   dw_i = sum_t dy_i n_i
 * dx is the gradient of x and of res alike.
 *   dy    bf16 [T][d] gradient of y
 *   dh    bf16 [T][d] gradient of h from the residual stream, or NULL for 0
 *   h, rstd, w  the forward's
 *   dx    bf16 [T][d] (out); may be dy or dh itself
 *   dw    f32 [d] (out), or NULL (then ws is not read).  Summed in a fixed
 *         order.
 * A dx that is no finite BF16 number (a non-finite dy, dh, h, rstd or w, or an
 * overflow) sets MOE_STATUS_NONFINITE_X; the other rows' dx are as without it.
 * Needs d % 16 == 0, 16 <= d <= 16384.  Two launches (one without dw). */
int moe_add_rmsnorm_backward(const uint16_t* dy, const uint16_t* dh,
                             const uint16_t* h, const float* rstd,
                             const uint16_t* w, int T, int d, uint16_t* dx,
                             float* dw, void* ws, size_t ws_bytes, int* status,
                             void* stream);

/* ---------------------------------------------------------------------- */
/* Token losses.  z = logits * inv_temperature; p = softmax(z).             */
/* A logit of -inf (a masked id) has p = 0 and enters no sum.  A row of      */
/* nothing but -inf has no distribution: see each entry point.  A row with a */
/* NaN or +inf gives NaN and sets MOE_STATUS_NONFINITE_LOGITS.               */
/* Needs 1 <= V <= 2^30, ld >= V, 1e-6 <= inv_temperature <= 1e6.            */
/* ---------------------------------------------------------------------- */

/* Log-probabilities of given tokens, entropy and top alternatives, in one
 * pass over the logits:
 *   logits  [T] rows of V, ld elements apart
 *   targets i32 [T], or NULL.  A negative id is no target (logprob 0); an id
 *           >= V sets MOE_STATUS_BAD_TOKEN and counts as none.
 *   n_top   alternatives per row, 0 <= n_top <= MOE_LOGPROBS_MAX_TOP
 *   logprob f32 [T] (out) z_target - lse(z), or NULL
 *   entropy f32 [T] (out) -sum p ln p, or NULL
 *   stats   f32 [T][2] (out) m = max logit and l = ln sum exp((logit - m)
 *           inv_temperature), so lse = m inv_temperature + l; or NULL
 *   top_ids i32 [T][n_top], top_logprob f32 [T][n_top] (out): the ids by
 *           (logit desc, id asc); ids of -inf logits are not listed, places
 *           left over hold -1 and -inf.  NULL where n_top = 0.
 * A row without a distribution: logprob -inf (0 without a target), entropy 0,
 * stats (-inf, 0), no alternatives.  One launch. */
int moe_token_logprobs(const void* logits, int dtype, int64_t ld, int T, int V,
                       const int32_t* targets, float inv_temperature, int n_top,
                       float* logprob, float* entropy, float* stats,
                       int32_t* top_ids, float* top_logprob, int* status,
                       void* stream);

/* Gradient of moe_token_logprobs:
 *   dlogits_v = inv_temperature (g_logprob (1[v = target] - p_v)
 *                                - g_entropy p_v (ln p_v + H))
 *   stats, entropy  the forward's (entropy only where g_entropy is given)
 *   g_logprob, g_entropy  f32 [T] gradients of logprob and entropy, or NULL
 *           for 0 (not both); g_logprob counts on rows with a target only
 *   dlogits [T] rows of V, ldd elements apart, of the logits' type (out); may
 *           be the logits themselves (same ld).  Columns past V are untouched.
 * Rows without a distribution, and rows whose gradients are both 0, get
 * zeros; the logits of the latter are not read.  Fastest where logits and
 * dlogits rows share their alignment within 16 bytes.  One launch. */
int moe_token_logprobs_backward(const void* logits, int dtype, int64_t ld,
                                int T, int V, const int32_t* targets,
                                float inv_temperature, const float* stats,
                                const float* entropy, const float* g_logprob,
                                const float* g_entropy, void* dlogits,
                                int64_t ldd, int* status, void* stream);

/* Distillation from a teacher's top logits: per row the teacher's K ids c_i
 * with its logits a_i, and the KL divergence of the student from the teacher
 *   loss = sum_i q_i (ln q_i - ln p_{c_i}) + r (ln r - ln s)
 *   teacher_lse given: q_i = exp(a_i inv_temperature - teacher_lse), the
 *     teacher's mass r = max(0, 1 - sum q_i) off the list and the student's
 *     mass s = sum of p off the list compared as one outcome.  r counts as 0
 *     up to 2^-23 (8 + 2 |teacher_lse|), what rounding leaves of 1 - sum q_i
 *     where the list holds all of the teacher's mass
 *   teacher_lse NULL: q = softmax over the listed a_i inv_temperature, r = 0
 *   teacher_ids     i32 [T][K], in any order.  A negative id is an empty
 *                   place.  An id >= V, or one listed before in its row, sets
 *                   MOE_STATUS_BAD_TOKEN and counts as an empty place.
 *   teacher_logits  f32 [T][K]; teacher_lse f32 [T] or NULL
 *   loss            f32 [T] (out)
 *   stats           f32 [T][4] (out) or NULL: max logit and ln-sum (as
 *                   moe_token_logprobs) of the whole row, then of the part
 *                   off the list ((-inf, 0) where that has no mass)
 * s is summed off the list alone, not as 1 minus the rest, so it keeps its
 * precision when the student is peaked.  q_i > 0 with p = 0 (or ln p below
 * FP32's range) gives +inf, and so does r > 0 with s = 0; a row with no teacher entry and no teacher_lse gives
 * 0; a row without a distribution gives +inf (0 where the teacher has no
 * mass).  NaN or +inf in the teacher's numbers gives NaN and
 * MOE_STATUS_NONFINITE_LOGITS.
 * Needs 1 <= K <= MOE_DISTILL_MAX_K, V <= MOE_DISTILL_MAX_V.  One launch. */
int moe_distill_topk(const void* logits, int dtype, int64_t ld, int T, int V,
                     const int32_t* teacher_ids, const float* teacher_logits,
                     const float* teacher_lse, int K, float inv_temperature,
                     float* loss, float* stats, int* status, void* stream);

/* Gradient of moe_distill_topk from its stats, with g = f32 [T] the gradient
 * of each row's loss:
 *   dlogits_v = g inv_temperature (p_v Q - q_v)          on the list,
 *               g inv_temperature t_v (s Q - r)          off it, t_v = p_v / s
 * with Q = sum q_i + r (1, or 0 for a row without teacher entries).  dlogits
 * as in moe_token_logprobs_backward.  Rows without a distribution, and rows
 * with g = 0 whatever their numbers hold, get zeros (the numbers of a row with
 * g = 0 still set status bits).  One launch. */
int moe_distill_topk_backward(const void* logits, int dtype, int64_t ld, int T,
                              int V, const int32_t* teacher_ids,
                              const float* teacher_logits,
                              const float* teacher_lse, int K,
                              float inv_temperature, const float* stats,
                              const float* g, void* dlogits, int64_t ldd,
                              int* status, void* stream);

/* moe_distill_topk and its gradient in one call, for weights g that are known
 * beforehand (a mean over tokens, a mask): loss as the forward gives it, not
 * multiplied by g.  Zeros where moe_distill_topk_backward gives them.  dlogits
 * may be the logits themselves.  One launch. */
int moe_distill_topk_train(const void* logits, int dtype, int64_t ld, int T,
                           int V, const int32_t* teacher_ids,
                           const float* teacher_logits,
                           const float* teacher_lse, int K,
                           float inv_temperature, const float* g, float* loss,
                           void* dlogits, int64_t ldd, int* status,
                           void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LEARNER_H */
