/*
 * sdv_cache.h -- the paged KV cache beside the verify step: filling it with a
 * chunk of new tokens, attention of the chunk over it, and reading it back.
 *
 * The verify step writes and reads a bf16 cache for a handful of rows per
 * sequence; these entry points serve what happens around it -- prompts and
 * pieces of prompts, next tokens, a cache held in 8 bits -- on the same pages,
 * page tables and status word (sdv.h).  All three take one description of a
 * ragged chunk (sdv_chunk).
 *
 * Conventions are those of sdv.h: device pointers owned by the caller, work
 * only enqueued on `stream`, host-visible errors returned at once with nothing
 * enqueued, device-visible ones in the status word.  A nonzero *status on entry
 * makes a call a no-op.  Offsets and lengths that contradict one another are
 * found before anything is written; a page id outside the pool is found when
 * its turn comes, its page is neither read nor written, and the rest of that
 * call's outputs hold nothing meaningful.
 */
#ifndef SDV_CACHE_H
#define SDV_CACHE_H

#include "sdv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How the cache holds keys and values.
 * SDV_CACHE_BF16: kv_pool bf16 [pages, n_kv, 2 (K then V), 16, head_dim], the
 *   verify step's layout.
 * SDV_CACHE_E4M3: kv_pool e4m3 codes [pages, n_kv, 2, 16, head_dim] and
 *   kv_scales bytes [pages, n_kv, 2, 16], one scale 2^e per (position, head, key
 *   or value), held as e + 127.  e is the smallest exponent in [-15, 7] with
 *   max|x| <= 448 * 2^e (-15 for a row of zeros); the code is x * 2^-e rounded
 *   to nearest even.  Magnitudes above 57344 saturate to it, infinities among
 *   them; a NaN stays a NaN and does not enter the maximum.  The value
 *   code * 2^e is exact in bf16 and in fp16. */
enum { SDV_CACHE_BF16 = 0, SDV_CACHE_E4M3 = 1 };

/* n_q <= 65536, a multiple of n_kv; head_dim 64 or 128; page_size 16; rope_theta 0 or >= 1:
 * the rotary base of sdv_cache_append (0: keys and queries are not rotated). */
typedef struct {
  int n_q, n_kv, head_dim, page_size;
  int cache_format;
  float rope_theta;
} sdv_cache_config;

/* A ragged chunk of new tokens.
 *  B, T (host)      sequences, at least one; rows that the caller's row buffers hold.  With T = 0 a
 *                   call enqueues nothing and its row pointers may be null.
 *  max_q (host)     an upper bound of every sequence's rows.  It picks sdv_cache_attention's kernels (a
 *                   captured call keeps them): one that is far too large costs time, a step of next tokens up to
 *                   twice its own, and no result.
 *  row_offsets [B+1] (device) row_offsets[0] = 0, non-decreasing, row_offsets[B] <= T:
 *                   sequence b owns rows [row_offsets[b], row_offsets[b+1]).
 *                   Rows behind the last sequence's are not touched.
 *  kv_lens [B] (device) positions of sequence b in the cache, the chunk's own
 *                   among them: row i of n sits at position kv_lens[b] - n + i.  A
 *                   row whose position is below 0 is empty: nothing is stored
 *                   for it, it sees nothing, and its output is 0.
 *  kv_pool, kv_scales, num_pool_pages   the cache (kv_scales NULL for bf16).
 *  page_table [B, max_pages_per_seq] (device) pool page of each block of 16
 *                   positions.  Only the blocks that a call needs are read: an
 *                   entry for positions before the window may be anything.
 *  window (host)    0: row at position p sees positions 0..p; w > 0: the last w of
 *                   them, p - w + 1 .. p (attention only). */
typedef struct {
  int B, T, max_q;
  const int *row_offsets, *kv_lens;
  void *kv_pool;
  void *kv_scales;
  int num_pool_pages;
  const int *page_table;
  int max_pages_per_seq;
  int window;
} sdv_chunk;

typedef struct sdv_cache sdv_cache;

/* Bytes of device workspace (partial results of key ranges cut between thread
 * blocks, and their counters) for chunks of up to max_rows rows (max_rows * n_q
 * below 2^30) and max_slots (<= 1024) sequences.  0 on an invalid configuration. */
size_t sdv_cache_workspace_size(const sdv_cache_config *cfg, int max_rows, int max_slots);

/* Create a handle on the current device.  `workspace` (device, caller-owned, >=
 * sdv_cache_workspace_size bytes, 256-byte aligned) has its counters cleared here, on `stream`, which
 * is synchronised (so not inside a capture); it is used by every sdv_cache_attention of this handle, so those calls must not overlap in
 * time; graphs captured on one handle must not run at the same time either.
 * Calls are made with the handle's device current. */
sdv_status sdv_cache_create(const sdv_cache_config *cfg, void *workspace, size_t workspace_bytes, int max_rows,
                            int max_slots, void *stream, sdv_cache **out);
void sdv_cache_destroy(sdv_cache *cache);

/* Rows of a chunk for sdv_cache_append.  Row r's heads are contiguous, head h at
 * r * stride + h * head_dim (strides in elements, so the rows of one fused
 * projection serve as they are).  Pointers 16-byte aligned, strides a multiple
 * of 16 bytes.
 *  k, v  [T, n_kv, head_dim]; x_format 0 = bf16, 1 = fp32.
 *  q     [T, n_q, head_dim] in the same format or NULL; q_out bf16: q at its
 *        positions, rotated when the handle rotates (rows of empty positions
 *        are not written). */
typedef struct {
  const void *k, *v, *q;
  long long k_stride, v_stride, q_stride;
  int x_format;
  void *q_out;
  long long q_out_stride;
} sdv_append_rows;

/* Write the chunk's keys and values at their positions: rotated (rotate-half,
 * angle = position * theta^(-2j/head_dim), keys only) when the handle has a rope_theta, then
 * rounded once to the cache's format. */
sdv_status sdv_cache_append(sdv_cache *cache, const sdv_chunk *chunk, const sdv_append_rows *rows, int *status,
                            void *stream);

/* Attention of the chunk's rows over their own sequences' cached positions, the
 * chunk's own (already appended) among them: scale 1/sqrt(head_dim), query head
 * h reads key head h / (n_q / n_kv).  q and out bf16 [T, n_q, head_dim] with row strides in
 * elements (16-byte aligned, strides multiples of 8).  Scores, the softmax's maximum and
 * sum and the output are held in 32 bits; the weights enter the second product
 * in 16 bits (bf16 over a bf16 cache; fp16 over codes, where a small weight is rounded to a multiple of at most
 * 2^-15 of what the keys beside it add up to).  Positions behind a sequence's end are never used, whatever they hold; the cached
 * values that the chunk's rows see are taken to be finite. */
sdv_status sdv_cache_attention(sdv_cache *cache, const sdv_chunk *chunk, const void *q, long long q_stride, void *out,
                               long long out_stride, int *status, void *stream);

/* Read the chunk's positions back: k_out / v_out [T, n_kv, head_dim] (either
 * may be NULL), out_format 0 = bf16, 1 = fp32, both exact.  Empty rows read as 0.  With row_offsets
 * that give a sequence as many rows as it has positions, all of it is read. */
sdv_status sdv_cache_read(sdv_cache *cache, const sdv_chunk *chunk, void *k_out, long long k_stride, void *v_out,
                          long long v_stride, int out_format, int *status, void *stream);

/* The tables of a step, made on the device from the requests' lengths.
 *  B, T (host)      requests, 1 .. 1024; entries that the row outputs hold, up to 2^30.
 *  new_rows [B], lens [B] (device) rows that request b brings to this step, and its positions in the cache
 *                   with them (both may be 0; a request with more rows than
 *                   positions has empty rows, as in a chunk).
 *  page_table [B, max_pages_per_seq], page_counts [B], free_pages [num_pool_pages], num_free (device,
 *                   all updated in place): the first page_counts[b] entries of row b are the
 *                   request's pages; the first *num_free entries of free_pages are the free stack, its
 *                   top last.
 *  row_offsets [B+1], row_request [T], positions [T], slots [T], last_rows [B] (device, outputs;
 *                   the last four may be NULL): request b's rows are [row_offsets[b],
 *                   row_offsets[b+1]), the i-th of n at position lens[b] - n + i; slots: page * 16 +
 *                   position % 16, -1 for an empty row; last_rows: the request's last row, -1 for
 *                   none.  Entries of row_request, positions and slots behind the last row are -1.
 *  max_B (host)     0, or the requests that row_offsets [max_B+1] and last_rows [max_B] have room for, B .. 1024: those
 *                   behind the B have no rows in this step (their offsets are the last one, their last
 *                   rows -1), so that a chunk of max_B sequences serves steps of any B.
 * row_offsets, lens, page_table are what a chunk (above) takes, row_request and
 * row_offsets what sampling (sdv_sample.h) and adapters (sdv_adapter.h) take. */
typedef struct {
  int B, T;
  const int *new_rows, *lens;
  int *page_table;
  int max_pages_per_seq;
  int *page_counts;
  int *free_pages;
  int num_pool_pages;
  int *num_free;
  int *row_offsets, *row_request, *positions, *last_rows;
  long long *slots;
  int max_B;
} sdv_cache_tables;

/* Give every request the ceil(lens[b] / 16) pages that its length needs and describe the step's rows.
 * Pages past that (a request that ended has length 0, one that was rewound a smaller one) are pushed
 * first, in the order of requests and of their blocks, their entries becoming -1; then missing pages are
 * popped in the same order.  Needs no handle and no workspace; calls on the same tables must not overlap.
 * Device errors, nothing written: SDV_ERR_BAD_INPUT (a negative count or length, more
 * than T rows, page_counts or *num_free out of range, a stack that the pushed
 * pages do not fit), SDV_ERR_CAPACITY (too few pages, a request of more than max_pages_per_seq).
 * SDV_ERR_PAGE_RANGE: a popped or pushed page id, or the page of a row, outside the pool: it is
 * handed on as it is (its rows' slots are -1). */
sdv_status sdv_cache_plan(const sdv_cache_tables *tables, int *status, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SDV_CACHE_H */
