/*
 * Rules on rows of logits before a token is drawn from them (libattn.so; C ABI):
 * biases, penalties for tokens that the request has seen, grammar masks; and the
 * table of seen tokens that the penalties go by.
 *
 * The code walkthrough's section 4.3 draws tokens from the logits of a batch
 * (attn_sample_tokens, sample.h); these calls go before and after it:
 *   attn_logits_adjust -> attn_sample_tokens -> attn_tokens_seen
 *
 * All device memory is the caller's; the calls are asynchronous on `stream`, allocate
 * nothing and may be recorded by stream capture.
 */
#ifndef GB300_LOGITS_H
#define GB300_LOGITS_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The table of seen tokens: uint16 [num_rows, ld], ld >= V, 16-byte aligned, ld a
 * multiple of 8.  Word v of a row: bit 15 is set if token v is in the request's
 * prompt, bits 0 .. 14 say how many times it was generated (at most 32767, where it
 * stays).  Rows outlive a batch: a request keeps its row while it runs, and the calls
 * name the rows of the batch. */
enum { ATTN_SEEN_PROMPT = 1, ATTN_SEEN_CLEAR = 2 };

/* Rules for the B rows of a call (host struct holding device pointers; a pointer
 * that may be NULL leaves its rule out).
 * Each logit x of token v in row b goes through
 *   1. x + (the sum of the row's biases for v, in list order), where it has any;
 *   2. if v was seen (its word is not 0): x / r where x > 0, else x * r, with
 *      r = repetition[b]; an r that is not > 0 leaves x;
 *   3. if v was generated, count times: x - frequency[b] * count, then
 *      x - presence[b];
 *   4. -inf if the row's mask has no bit for v;
 * each operation in fp32, rounded to nearest even. */
typedef struct attn_logits_rules {
  const uint16_t* seen;      /* [seen_rows, seen_ld], or NULL: no penalties */
  int64_t seen_ld;
  int32_t seen_rows;
  const int32_t* seen_row;   /* [B]: row b's row of the table (outside the table: nothing seen); NULL: b */
  const float* repetition;   /* [B], each may be NULL */
  const float* presence;
  const float* frequency;
  const int32_t* bias_start; /* [B + 1], or NULL: no biases.  Row b's entries: bias_start[b] .. bias_start[b + 1] - 1 */
  const int32_t* bias_token; /* [num_biases]; tokens outside [0, V) are skipped */
  const float* bias_value;   /* [num_biases] */
  int32_t num_biases;        /* entries of bias_start outside [0, num_biases) are skipped */
  const uint32_t* mask;      /* [mask_rows, mask_ld], bit v % 32 of word v / 32: token v is allowed; NULL: no masks */
  int64_t mask_ld;           /* words per row, >= ceil(V / 32) */
  int32_t mask_rows;
  const int32_t* mask_row;   /* [B]: row b's mask (outside [0, mask_rows): every token is allowed); NULL: b */
} attn_logits_rules_t;

/* out [B, ld_out] (fp32) = the rules applied to logits [B, ld], V logits per row; out
 * may be logits itself with ld_out == ld (else the two must not overlap).  A row
 * whose mask allows nothing comes out as -inf throughout (attn_sample_tokens wants one
 * finite logit).  ATTN_EINVAL: NULL rules, NULL logits or out with B != 0, B < 0, V < 1,
 * V > 2^23, ld or ld_out < V, out == logits with another ld, a misaligned pointer, a table
 * or mask with a row shorter than V or without rows, seen_ld not a multiple of 8,
 * bias_start with num_biases < 0, or > 0 without bias_token and bias_value. */
ATTN_API int attn_logits_adjust(const float* logits, int32_t B, int32_t V, int64_t ld,
                                const attn_logits_rules_t* rules, float* out, int64_t ld_out, void* stream);

/* Tokens enter the table: those of request b, tokens[cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1] (cu_seqlens NULL: tokens[b], N == B), into row rows[b]
 * (NULL: b).  Without ATTN_SEEN_PROMPT the generated counts rise by one per token
 * listed, with it the prompt bit is set.  ATTN_SEEN_CLEAR empties the rows of the
 * call first.  Rows outside [0, num_rows) and tokens outside [0, V) are skipped; a row
 * may be named more than once.  ATTN_EINVAL: NULL seen, NULL tokens with N != 0, negative sizes,
 * V < 1, V > 2^23, ld < V or not a multiple of 8, num_rows < 1, a misaligned
 * pointer, cu_seqlens NULL with N != B, other flags, ATTN_SEEN_CLEAR with
 * B * ceil(ld / 8192) above 2^31 - 1. */
ATTN_API int attn_tokens_seen(uint16_t* seen, int64_t ld, int32_t num_rows, int32_t V, const int32_t* rows,
                              const int32_t* cu_seqlens, const int32_t* tokens, int32_t B, int32_t N,
                              int32_t flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_LOGITS_H */
