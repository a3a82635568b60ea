/*
 * moe_tokens.h -- C ABI of the operators at a model's token ends, in the same
 * library (libmoe_nvfp4.so):
 *
 *   - the embedding: the table's rows that given tokens name, scaled, and the
 *     gradient of the table;
 *   - the draw of the next token from the logits of each row, with temperature,
 *     top-k, top-p and min-p and a random number that the caller gives.  The
 *     drawn token and its log-probability are those that moe_token_logprobs
 *     (moe_learner.h) scores in the learner.
 *
 * Conventions are those of moe_nvfp4.h and moe_learner.h: device pointers
 * owned by the caller, every call enqueued on `stream`, no allocation, no
 * synchronisation, return codes checked on the host before anything is
 * enqueued, `status` an optional device int that receives MOE_STATUS_* bits,
 * results deterministic bit for bit.  Host threads may call them at the same
 * time.  16-bit tensors, tables and gradients are 16-byte aligned, logits by
 * their element, int32 and float vectors 4-byte aligned.  Strides are in
 * elements; rows times a stride stay below 2^46.  No output overlaps an input or
 * another output.  T = 0 does nothing (but see moe_embed_tokens_backward).
 */
#ifndef MOE_TOKENS_H
#define MOE_TOKENS_H

#include "moe_learner.h"

#ifdef __cplusplus
extern "C" {
#endif

/* device status bit (others: moe_nvfp4.h, moe_learner.h) */
#define MOE_STATUS_BAD_SAMPLING 0x40 /* a row's sampling numbers are out of range */

#define MOE_EMBED_MAX_V  (1 << 24)
#define MOE_EMBED_MAX_D  16384
#define MOE_SAMPLE_MAX_V (1 << 20)

/* ---------------------------------------------------------------------- */
/* Embedding.                                                               */
/* ---------------------------------------------------------------------- */

/* out_t = BF16(scale * table[ids_t]), the product in FP32:
 *   ids    i32 [T].  A negative id (padding) gives a row of zeros, and so does
 *          an id >= V, which sets MOE_STATUS_BAD_TOKEN.
 *   table  [V] rows of d, ldt elements apart, MOE_DTYPE_BF16 or MOE_DTYPE_F32
 *   out    bf16 [T] rows of d, ldo elements apart (out)
 * Needs d % 8 == 0, 8 <= d <= MOE_EMBED_MAX_D, 1 <= V <= MOE_EMBED_MAX_V,
 * ldt, ldo >= d and multiples of 8, a finite scale.  One launch. */
int moe_embed_tokens(const int32_t* ids, const void* table, int dtype,
                     int64_t ldt, int T, int V, int d, float scale,
                     uint16_t* out, int64_t ldo, int* status, void* stream);

/* Workspace of moe_embed_tokens_backward: the tokens sorted by id, a bit map of
 * the ids, and the parts of the sums of ids that many tokens name.  0 for sizes
 * out of range.  Calls that may run at the same time need their own. */
size_t moe_embed_tokens_backward_workspace_bytes(int T, int V, int d);

/* The gradient of moe_embed_tokens with respect to the table:
 *   dtable_v = scale * sum over the t with ids_t = v of dy_t  (+ dtable_v)
 * summed in FP32 in an order that follows from the sizes and the ids alone, and
 * multiplied by scale once.
 *   dy      bf16 [T] rows of d, ldy elements apart
 *   ids     as in the forward: negative ids and ids >= V contribute nothing,
 *           the latter set MOE_STATUS_BAD_TOKEN
 *   accumulate  0: all V rows are written, zeros where no token names the row
 *           (T = 0: all zeros).  1: added to the rows that tokens name, the
 *           others are neither read nor written.
 *   dtable  f32 [V][d]
 *   ws      moe_embed_tokens_backward_workspace_bytes(T, V, d) bytes
 * Limits as moe_embed_tokens; T <= 2^24, ldy >= d and a multiple of 8.  One
 * launch up to 1024 tokens, four to six beyond. */
int moe_embed_tokens_backward(const uint16_t* dy, int64_t ldy,
                              const int32_t* ids, int T, int V, int d,
                              float scale, int accumulate, float* dtable,
                              void* ws, size_t ws_bytes, int* status,
                              void* stream);

/* ---------------------------------------------------------------------- */
/* The draw of a token.                                                     */
/* ---------------------------------------------------------------------- */

/* Per row, with z = logits * inv_temperature and the weight w = e^(z - max z),
 * counted as 0 where it is below 2^-42 (such an id is never drawn):
 *   1. of the ids in the order (logit descending, id ascending) the first
 *      top_k are kept; ids of -inf logits never are;
 *   2. of these the shortest leading part that holds at least top_p of their
 *      weight (the first id always);
 *   3. of these the ones with w >= min_p;
 *   4. the token is the first kept id, in the order of the ids, up to which
 *      the kept weight is above u times all of it.
 * The token is the one of these formulas in exact arithmetic unless a border
 * lies within some 2^-33 of the row's weight: FP32 weights decide where their
 * error bound allows it, and weights of that precision where it does not.  Equal
 * logits have equal weights, and sums of weights 1 are exact.
 *   logits   [T] rows of V, ld elements apart, MOE_DTYPE_BF16 or MOE_DTYPE_F32
 *   inv_temperature  f32 [T], each 1e-6 to 1e6, or NULL for 1
 *   top_k    i32 [T], or NULL; < 1 or >= V: off
 *   top_p    f32 [T], or NULL; >= 1: off; <= 0 keeps the first id
 *   min_p    f32 [T], or NULL; <= 0: off; > 1 counts as 1
 *   u        f32 [T] random numbers, 0 <= u < 1
 *   tokens   i32 [T] (out)
 *   logprob  f32 [T] (out) ln p of the token under softmax(z), as
 *            moe_token_logprobs gives it, or NULL
 *   kept_logprob  f32 [T] (out) its logarithm under what was kept: ln of the
 *            probability with which it was drawn, or NULL
 * A row of nothing but -inf gives token -1 and -inf twice; a row with a NaN or
 * +inf token -1, NaN twice and MOE_STATUS_NONFINITE_LOGITS; a row whose
 * inv_temperature or u is out of range or whose top_p or min_p is NaN token
 * -1, NaN twice and MOE_STATUS_BAD_SAMPLING.
 * A row's token does not depend on the other rows, unless a border lies within the
 * distance above: T decides which launch takes the row, and their weights differ
 * below it.  The log-probabilities may differ in their last bits with T and with the
 * alignment of a row's address, along whose 16-byte vectors FP32 sums are formed.  Between
 * its launches the call marks rows in tokens, which nothing else may write or read
 * meanwhile.
 * Needs 1 <= V <= MOE_SAMPLE_MAX_V, ld >= V.  One launch for few rows (a cluster
 * of blocks each), else two: the second decides rows that the first leaves open,
 * which are few where the weight of each row lies in few ids and top_k is off or
 * 1024 at most.  A top_k above that (above 1536 where rows are long or few) leaves
 * its row open however the weight lies, unless min_p, with top_p off, keeps few;
 * such a row costs what a flat one does. */
int moe_sample_tokens(const void* logits, int dtype, int64_t ld, int T, int V,
                      const float* inv_temperature, const int32_t* top_k,
                      const float* top_p, const float* min_p, const float* u,
                      int32_t* tokens, float* logprob, float* kept_logprob,
                      int* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_TOKENS_H */
