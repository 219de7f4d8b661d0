/*
 * kvrope: rotary positions of queries and keys on one NVIDIA GB300 (sm_103a),
 * and their fused form that rotates q and k and writes k and v to a Q8_0 or Q4_0
 * cache.
 *
 * The first rotary_dim elements of a head are rotary_dim / 2 pairs: (2 i, 2 i + 1)
 * when interleaved, else (i, i + rotary_dim / 2); the rest stays.  At position p
 * pair i turns by p * turns[i] units of 2^-64 of a whole turn, modulo 2^64 as
 * unsigned integers, so that no position is too far for the angle to be exact:
 *     c = f32(cos) * factor,  s = f32(sin) * factor
 *     y[a] = x[a] c - x[b] s,  y[b] = x[b] c + x[a] s     (a, b the pair)
 * in f32, every step rounded.  cos and sin are within 2^-42 of the angle's before
 * their rounding to f32.  A frequency f, in radians a position, has turns
 * round(f / (2 pi) * 2^64).  Frequencies that are scaled for long contexts, by any
 * rule, are other turns.
 */
#ifndef KVROPE_H
#define KVROPE_H

#include "q4kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvrope_s *kvrope_plan_t;

/* head_dim 2 .. 65536, rotary_dim even, 2 .. min(head_dim, 512); turns[rotary_dim / 2] on the host. */
q8mv_status_t kvrope_plan(kvrope_plan_t *out, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
                          const uint64_t *turns, float factor, int device);

/*
 * out = x rotated by positions[n] (inverse != 0: by the transpose, which is the
 * gradient's way, and back but for the square of a factor that is not 1).  Row r, head h at x + r * x_row + h * x_head elements, the last
 * axis contiguous, any alignment of the type; out may be x itself with its strides.
 * Else it must not overlap x or positions, nor its own rows one another: calls whose
 * memory does, or whose rows are differently far apart in the same stretch of it, are
 * refused.  Negative positions turn the other way.  0 <= n < 2^31.
 */
q8mv_status_t kvrope_apply(kvrope_plan_t plan, int64_t n, int32_t heads, int32_t type, const void *x, int64_t x_row,
                           int64_t x_head, const int64_t *positions, void *out, int64_t out_row, int64_t out_head,
                           int32_t inverse, cudaStream_t stream);

/*
 * One call for a layer's step: out = q rotated (heads_q = 0: no q), k rotated and,
 * without a rounding to its type between, quantised with v into slots, as
 * q8kv_cache_write or q4kv_cache_write would.  A slot outside the cache skips its
 * token's k and v, not its q.  The plan's head_dim is the cache's.  out is refused as
 * in kvrope_apply where it overlaps q (unless it is q), k, v, positions or slots; it may
 * lie between them, as q's part of one tensor that holds all three.
 */
typedef struct {
    const void *q, *k, *v;
    void *out;                /* q's shape; may be q with its strides */
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
    const int64_t *positions; /* [n] */
    const int64_t *slots;     /* [n] */
    int64_t n;
    int32_t heads_q;
    int32_t type;             /* Q8KV_* of q, k, v and out */
} kvrope_write_args_t;

q8mv_status_t kvrope_write_q8(kvrope_plan_t plan, const q8kv_cache_t *cache, const kvrope_write_args_t *args,
                              cudaStream_t stream);
q8mv_status_t kvrope_write_q4(kvrope_plan_t plan, const q4kv_cache_t *cache, const kvrope_write_args_t *args,
                              cudaStream_t stream);

/* Synchronises the plan's device, then releases its tables.  NULL is accepted.  Calls of one plan may overlap. */
q8mv_status_t kvrope_destroy(kvrope_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* KVROPE_H */
