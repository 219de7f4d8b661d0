/*
 * kvpage: which request holds which pages of a cache, on one NVIDIA GB300
 * (sm_103a): pages are given out, shared, copied when they are written, given
 * back and brought together, all on the device, so that a decode step with them
 * is a CUDA graph.
 *
 * The state is the caller's, three int32 arrays in device memory:
 *     refs [pages]                 how many requests hold a page; 0: it is free
 *     table [requests, columns]    pages of a request in order, -1 from held on
 *     held [requests]              how many it holds
 * Copies of them are snapshots, and written back they are the state.  Counts and
 * numbers below 0 or past the end are never followed.  All results are whole
 * numbers and do not depend on an order of threads.  Calls on one plan share its
 * workspace and must be ordered; arrays must not overlap.
 */
#ifndef KVPAGE_H
#define KVPAGE_H

#include "q4kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvpage_s *kvpage_plan_t;

typedef struct {
    int32_t *refs;
    int32_t *table;  /* request b's row at table + b * columns */
    int32_t *held;
} kvpage_state_t;

/* pages 1 .. 2^28, page_size 1 .. 65536, requests 1 .. 65535, columns 1 .. 2^24, requests * columns <= 2^28 */
q8mv_status_t kvpage_plan(kvpage_plan_t *out, int64_t pages, int32_t page_size, int32_t requests, int32_t columns,
                          int device);

/*
 * Pages for tokens[b] (below 0: 0) tokens past lengths[b] (below 0: 0).  With P =
 * page_size, columns lengths / P .. ceil((lengths + tokens) / P) - 1 get a fresh page
 * if they are past held (and so do any between held and lengths / P), or if the page
 * there is shared (refs > 1): the other requests keep it.  If the first of them already has tokens (lengths % P > 0) and was
 * shared, its page has to be copied: src[b] -> dst[b], both -1 for a request
 * without.  Fresh pages are the lowest that were free before the call, in order of
 * request, then column.  ok[b] = 1, or 0 for a request that would pass the columns,
 * or for which, with all before it, there are not enough free pages: it stays as it
 * was.  slots[b * width + t] is the slot of token lengths[b] + t, -1 from tokens[b] on
 * and where ok is 0.
 */
q8mv_status_t kvpage_extend(kvpage_plan_t plan, const kvpage_state_t *state, const int32_t *lengths,
                            const int32_t *tokens, int32_t width, int64_t *slots, int32_t *src, int32_t *dst,
                            int32_t *ok, cudaStream_t stream);

/*
 * Request b becomes what request parents[b] was before the call, holding the same
 * pages (shared now), all at once, so any map is fine; it gives back the pages that it
 * held.  parents[b] = b changes nothing, a parent outside 0 .. requests - 1 leaves b
 * without pages.
 */
q8mv_status_t kvpage_fork(kvpage_plan_t plan, const kvpage_state_t *state, const int32_t *parents,
                          cudaStream_t stream);

/* Request b keeps the pages of its first lengths[b] tokens (0: none) and gives the others back. */
q8mv_status_t kvpage_free(kvpage_plan_t plan, const kvpage_state_t *state, const int32_t *lengths,
                          cudaStream_t stream);

/*
 * The L pages with refs > 0 become pages 0 .. L - 1: the i-th page past them that is
 * held moves to the i-th free one among them, src[i] -> dst[i] for i < count[0], -1
 * behind, with src and dst [pages / 2].  refs and the table follow; copy the pages of
 * every cache next.
 */
q8mv_status_t kvpage_compact(kvpage_plan_t plan, const kvpage_state_t *state, int32_t *src, int32_t *dst,
                             int32_t *count, cudaStream_t stream);

/* Synchronises the plan's device, then releases its workspace.  NULL is accepted. */
q8mv_status_t kvpage_destroy(kvpage_plan_t plan);

/*
 * Page dst[i] becomes a copy of page src[i], codes and scales of every head, for i < n,
 * or i < min(n, count[0]) with count in device memory.  Pairs with a page outside the
 * cache are skipped; a page may be the source of several, no destination may be
 * another's source or destination.  0 <= n < 2^31.
 */
q8mv_status_t kvpage_copy_q8(const q8kv_cache_t *cache, int64_t n, const int32_t *src, const int32_t *dst,
                             const int32_t *count, cudaStream_t stream);
q8mv_status_t kvpage_copy_q4(const q4kv_cache_t *cache, int64_t n, const int32_t *src, const int32_t *dst,
                             const int32_t *count, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KVPAGE_H */
