/*
 * sdv_sample.h -- sampling under each request's own settings: temperature,
 * top-k, top-p and min-p from given uniforms, and the distribution that they
 * leave.
 *
 * The verify step (sdv.h) samples from the plain softmax.  A request with
 * settings of its own takes these instead: its rows' filtered distributions are
 * what sdv_accept reads as target probabilities, what a draft model hands over
 * as draft_probs beside the tokens drawn from them, and a row without drafts
 * takes its next token directly.
 *
 * Conventions are those of sdv.h: device pointers owned by the caller, work
 * only enqueued on `stream`, host-visible errors returned at once with nothing
 * enqueued, device-visible ones in the status word.  A nonzero *status on entry
 * makes a call a no-op; after a call that set it the outputs hold nothing meaningful.
 */
#ifndef SDV_SAMPLE_H
#define SDV_SAMPLE_H

#include "sdv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows to sample, all device pointers.
 *  logits [rows, vocab], x_format 0 = bf16, 1 = fp32, row r at r * stride
 *                   elements (aligned to its type; any stride >= vocab).  -inf: never
 *                   drawn and counted by no setting; +inf: shares the row's whole mass
 *                   with its likes.
 *  row_request [rows] or NULL: the request whose settings row r takes (NULL:
 *                   row r is request r).  Negative: the row's outputs are left as they are.
 *  temperature, top_p, min_p fp32, top_k int [requests], each may be NULL (1, 1,
 *                   0, 0).  temperature 0 takes the largest logit (the first of equals); else
 *                   1e-30 .. 1e30.  top_k 0: off.  top_p in (0, 1], 1: off.  min_p in [0, 1], 0: off.
 *  uniforms [rows]  fp32 in [0, 1); may be NULL when tokens is.
 *  tokens [rows] int or NULL, probs fp32 [rows, probs_stride] or NULL, not both NULL.  They overlap
 *                   no input.  probs and logits that do are refused (SDV_ERR_INVALID_ARG): their address
 *                   ranges are apart, or they are columns of rows equally far apart in bytes.
 *
 * In order (logit descending, index ascending): the first top_k stay; of those
 * the shortest run whose sum of w = exp((z - max) / temperature) reaches top_p times theirs;
 * of those the ones with w >= min_p.  probs is w / (sum of those left), 0
 * elsewhere; the token is the first index whose running sum, by index, exceeds uniform * sum.
 * Both bounds are met on exact sums of integers: w in steps of 2^-42, within 2^-34 of itself down to 2^-13 of the
 * largest and 2^-33 of the largest below (what lies under 2^-43 of it adds nothing to a sum).  So which token is the last to stay, or the
 * one drawn, does not depend on an order of summation.
 * probs is that quotient in fp32, within 2^-20.8 of itself or 2^-149, and 0 for tokens below 2^-126 of the largest, though they stay.
 *
 * Device errors (SDV_ERR_BAD_INPUT): a setting or uniform out of range, a request
 * not below `requests`, a row with a NaN or with nothing above -inf. */
typedef struct {
  const void *logits;
  int x_format;
  long long stride;
  int rows, vocab, requests;
  const int *row_request;
  const float *temperature;
  const int *top_k;
  const float *top_p, *min_p;
  const float *uniforms;
  int *tokens;
  float *probs;
  long long probs_stride;
} sdv_sample_rows;

/* Sample (tokens) and / or filter (probs) the rows.  Needs no workspace; calls
 * may overlap.  vocab up to 2^20, else SDV_ERR_UNSUPPORTED; rows up to 2^20. */
sdv_status sdv_sample(const sdv_sample_rows *rows, int *status, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SDV_SAMPLE_H */
