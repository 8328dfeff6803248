/*
 * sdv_adapter.h -- low-rank adapters of many requests at once beside a shared
 * projection.
 *
 * The projections of a batch are shared (sdv_linear); a request with an adapter
 * of its own adds scale * (x A^T) B^T to its rows.  One call serves all
 * requests of a ragged batch, whichever adapters they have.
 *
 * Conventions are those of sdv.h: device pointers owned by the caller, work
 * only enqueued on `stream`, host-visible errors returned at once with nothing
 * enqueued, device-visible ones in the status word.  A nonzero *status on entry
 * makes a call a no-op; after a call that set it the outputs hold nothing meaningful.
 */
#ifndef SDV_ADAPTER_H
#define SDV_ADAPTER_H

#include "sdv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A pool of adapters of one projection [n, k] (as sdv_linear's [N, K]): k, n and rank multiples of 8, rank at
 * most 128 (an adapter of a smaller rank has zeros behind it).
 *  a [count, rank, k], b [count, n, rank] bf16, scales [count] fp32 (device, 16-byte
 *  aligned, read-only; valid for the handle's life, what they hold may be exchanged between calls). */
typedef struct {
  int k, n, rank, count;
  const void *a, *b;
  const float *scales;
} sdv_adapter_config;

typedef struct sdv_adapters sdv_adapters;

/* Create a handle on the current device for calls of up to max_rows rows of max_slots (<= 1024) requests.  It needs no
 * workspace: calls may overlap.  They are made with the handle's device current. */
sdv_status sdv_adapters_create(const sdv_adapter_config *cfg, int max_rows, int max_slots, sdv_adapters **out);
void sdv_adapters_destroy(sdv_adapters *adapters);

/* Rows of a batch.
 *  B, T (host)         requests, at least one; rows that the buffers hold.
 *  row_offsets [B+1] (device) row_offsets[0] = 0, non-decreasing, row_offsets[B] <= T: request b owns rows
 *                      [row_offsets[b], row_offsets[b+1]).  Rows behind the last request's are not touched.
 *  adapter_ids [B] (device) the request's adapter, below `count`; negative: none, its rows of out are base's.
 *  x [T, k]            x_format 0 = bf16, 1 = fp32, rows x_stride elements apart.
 *  base, out [T, n]    y_format 0 = bf16, 1 = fp32; out may be base, else it shares no memory with base; with x it never does
 *                      (refused: SDV_ERR_INVALID_ARG; rows of unlike pitches have address ranges apart).
 * Pointers 16-byte aligned, strides multiples of 16 bytes.
 * out = base + scale * (x A^T) B^T: products of the values as they are (fp32 x as a sum of three bf16, the rank values of three for an
 * fp32 out and two for a bf16 one), sums in fp32, rounded once to out's format.  Infinities and NaN do what fp32 arithmetic does with
 * them (0 * inf and inf - inf are NaN), in their own rows only; finite values take part whatever their size. */
typedef struct {
  int B, T;
  const int *row_offsets, *adapter_ids;
  const void *x;
  int x_format;
  long long x_stride;
  const void *base;
  void *out;
  int y_format;
  long long base_stride, out_stride;
} sdv_adapter_rows;

sdv_status sdv_adapters_apply(sdv_adapters *adapters, const sdv_adapter_rows *rows, int *status, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SDV_ADAPTER_H */
