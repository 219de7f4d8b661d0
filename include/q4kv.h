/*
 * q4kv: a Q4_0 key/value cache on one NVIDIA GB300 (sm_103a): 4.5 bits an
 * element where q8kv's takes 9, and the same operators on it: writing, reading
 * and moving rows, and attention of a tree of drafted tokens over it (a single
 * token is a tree of one).
 *
 * Calls, statuses, streams and plans are q8kv.h's, and so are pages, slots and
 * the numbering of rows: row (page, head, place) is
 *     r = page * stride_page + head * stride_head + place * stride_token.
 * A row holds NB blocks of 32 elements, NB the least of 2, 3, 4, 6 and 8 that
 * hold head_dim.  It starts at byte r * 16 * NB of the codes and element r * SB of
 * the scales, SB = 2, 4, 4, 8, 8 for those NB (columns at and past NB are not
 * used).  Element e = 32 b + i has a code c of 0 .. 15 and stands for
 *     x[e] = (c - 8) * d[b],   d an f16.
 * In its block's 16 bytes it is in byte i / 2, in the low half if i is even.  A
 * row keeps units of U bytes (4 for keys, 2 for values) of all its blocks side by
 * side: byte U u + j of block b is byte U (u NB + b) + j of the row.  So a lane of
 * the attention finds what it needs of all blocks in one place.
 * Codes and scales are 16-byte aligned device memory; head_dim is a multiple of
 * 16, at most 256.
 */
#ifndef Q4KV_H
#define Q4KV_H

#include "q8kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    uint8_t *k_codes;
    uint16_t *k_scales;   /* bits of f16 */
    uint8_t *v_codes;
    uint16_t *v_scales;
    int64_t pages;        /* >= 0; pages * page_size < 2^40 */
    int32_t page_size;    /* 1 .. 65536 */
    int32_t heads;        /* 1 .. 65535 */
    int32_t head_dim;     /* 16 .. 256, a multiple of 16 */
    int32_t reserved;     /* 0 */
    int64_t stride_page;  /* in rows, each >= 1 */
    int64_t stride_head;
    int64_t stride_token;
} q4kv_cache_t;

/*
 * Quantise n tokens' keys and values into the cache; arguments as q8kv_cache_write.
 * Per block, on the inputs' f32 values and every step rounded:
 *     top = the largest of max x and max -x, with its sign (the positive one of two alike)
 *     d = f16(top * -1/8),  c = clamp(rint(x * (1 / d)) + 8, 0, 15)
 * (ties to even; c = 8 where d = 0; elements past head_dim count as 0).  NaN
 * elements do not count in top and get code 8.  A block whose d leaves f16 (|top| of
 * 524160 or more, an infinity) has codes 8 and reads back as NaN.
 */
q8mv_status_t q4kv_cache_write(const q4kv_cache_t *cache, int64_t n, const void *k, const void *v, int32_t type,
                               int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                               const int64_t *slots, cudaStream_t stream);

/* As q8kv_cache_read: (c - 8) * d in f32, which is exact, rounded once to `type`. */
q8mv_status_t q4kv_cache_read(const q4kv_cache_t *cache, int64_t n, const int64_t *slots, void *k_out, void *v_out,
                              int32_t type, cudaStream_t stream);

/* As q8kv_cache_move. */
q8mv_status_t q4kv_cache_move(const q4kv_cache_t *cache, int64_t batch, int64_t path, const int64_t *src,
                              const int64_t *dst, cudaStream_t stream);

/*
 * As q8kv_attend, with the same arguments, masks, limits and results for what is
 * not seen.  Arithmetic: codes are exact in f16; queries as there; each block's
 * products accumulate in f32 with the 8 taken off, its scale is folded in f32, the
 * softmax runs in f32, and its weights times the values' scales enter the second
 * product as two f16 parts (f32 and f16 outputs) or one (bf16 outputs), each of them
 * to 2^-24 of the row's largest weight times the largest scale near it, whatever the
 * values' size.  With more than 48 bf16 query rows a request and kv head (head_dim up
 * to 128), and page tables long enough, keys enter the first product exactly and values
 * the second with f16's 11 bits.  A scale that is not finite makes all of a row that
 * sees its key NaN.
 */
typedef struct q4kv_attend_s *q4kv_attend_plan_t;

q8mv_status_t q4kv_attend_plan(q4kv_attend_plan_t *out, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                               int32_t max_requests, int64_t max_rows, int device);
q8mv_status_t q4kv_attend(q4kv_attend_plan_t plan, const q4kv_cache_t *cache, const q8kv_attend_args_t *args,
                          cudaStream_t stream);
/* As q8kv_attend_check and q8kv_attend_set_wait. */
q8mv_status_t q4kv_attend_check(q4kv_attend_plan_t plan, int32_t *device_error);
q8mv_status_t q4kv_attend_set_wait(q4kv_attend_plan_t plan, uint64_t wait_ns);
/* Synchronises the plan's device, then releases its workspace.  NULL is accepted. */
q8mv_status_t q4kv_attend_destroy(q4kv_attend_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* Q4KV_H */
