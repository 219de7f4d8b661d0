/*
 * q8kv: a Q8_0 key/value cache on one NVIDIA GB300 (sm_103a), and the decode
 * operators that work on it: writing, reading and moving rows, attention of a
 * tree of drafted tokens over the cache (a single token is a tree of one), and
 * the verification of drafted tokens against the target's probabilities.
 *
 * The calls live in libq8mv.so beside the Q8_0 products of q8mv.h and follow
 * the same rules: plain pointers and sizes, q8mv_status_t results, arguments
 * checked on the host before anything is launched, asynchronous on the given
 * stream, no allocation outside a plan's creation, one plan per concurrent
 * stream.
 *
 * The cache.  A page holds page_size tokens.  Token slot s (0 <= s < pages *
 * page_size) is place s % page_size of page s / page_size.  For each slot and
 * kv head there is one row of head_dim int8 codes c and ceil(head_dim / 32)
 * f32 scales d for the keys, and one for the values; element e stands for
 *     x[e] = c[e] * d[e / 32].
 * Row (page, head, place) starts at element
 *     r * head_dim of the codes and r * ceil(head_dim / 32) of the scales,
 *     r = page * stride_page + head * stride_head + place * stride_token,
 * so a page may keep a head's tokens together (stride_token = 1) or a token's
 * heads together (stride_head = 1).  Rows must not overlap.  Codes and scales
 * are 16-byte aligned device memory; head_dim is a multiple of 16, at most 256.
 *
 * Slots, page numbers, lengths, masks, tokens and parents are device memory
 * that the host does not read.  A slot or page outside the cache is never
 * followed: each call says what it does instead.
 */
#ifndef Q8KV_H
#define Q8KV_H

#include "q8mv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { Q8KV_F32 = 0, Q8KV_F16 = 1, Q8KV_BF16 = 2 };

typedef struct {
    int8_t *k_codes;
    float *k_scales;
    int8_t *v_codes;
    float *v_scales;
    int64_t pages;        /* >= 0; pages * page_size < 2^40 */
    int32_t page_size;    /* 1 .. 65536 */
    int32_t heads;        /* 1 .. 65535 */
    int32_t head_dim;     /* 16 .. 256, a multiple of 16 */
    int32_t reserved;     /* 0 */
    int64_t stride_page;  /* in rows, each >= 1 */
    int64_t stride_head;
    int64_t stride_token;
} q8kv_cache_t;

/*
 * Quantise n tokens' keys and values into the cache.  Token i, head h is read
 * from k + i * k_row + h * k_head and v + i * v_row + h * v_head (strides in
 * elements, >= 0; the last axis is contiguous; any alignment of the type), and
 * written to slots[i].  Per 32-element block of a row (the last may be
 * shorter), in IEEE f32 arithmetic on the inputs' f32 values, every step rounded:
 *     amax = max |x|,  d = amax / 127,  c = rint(x * (127 * (1 / amax)))
 * (ties to even; c = 0 when amax = 0; +-127 where the factor overflows), as
 * q8mv_quantize_rows but for the factor, which that rounds once: a code may be one
 * apart where x is halfway between two.  NaN elements do not count in amax and get
 * code 0 unless amax is infinite; a block with an infinity has d = inf and
 * codes 0, and reads back as NaN.  Slots outside the cache are skipped; the
 * slots of one call must differ.  0 <= n < 2^31, here and in q8kv_cache_read.
 */
q8mv_status_t q8kv_cache_write(const q8kv_cache_t *cache, int64_t n, const void *k, const void *v, int32_t type,
                               int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head,
                               const int64_t *slots, cudaStream_t stream);

/*
 * Read n slots back: k_out and v_out [n, heads, head_dim], contiguous,
 * 16-byte aligned, each element c * d in f32 rounded once to `type`.  A slot
 * outside the cache gives zeros.
 */
q8mv_status_t q8kv_cache_read(const q8kv_cache_t *cache, int64_t n, const int64_t *slots, void *k_out, void *v_out,
                              int32_t type, cudaStream_t stream);

/*
 * Move rows inside the cache: for each request b < batch and i = 0 .. path-1
 * in this order, slot dst[b * path + i] becomes a copy of slot
 * src[b * path + i] (codes and scales of every head).  A pair with a slot
 * outside the cache is skipped.  A later pair of the same request may read
 * what an earlier one wrote, as with the accepted nodes of a draft tree that
 * move up to follow their prefix; slots of different requests must not meet.
 * batch <= 65535, path < 2^31.
 */
q8mv_status_t q8kv_cache_move(const q8kv_cache_t *cache, int64_t batch, int64_t path, const int64_t *src,
                              const int64_t *dst, cudaStream_t stream);

/*
 * Attention of draft trees over the cache.  Request b has T_b query rows
 * ("nodes": the newest token and the tokens drafted after it), and P_b =
 * lengths[b] cached tokens before them; node j's own key and value are in the
 * cache at position P_b + j (write them first).  Position p of request b is
 * place p % page_size of page table[b * table_row + p / page_size].  Node i
 * sees every position below P_b, and node j of its request if bit j % 32 of
 * word mask[(row of i) * mask_row + j / 32] is set (mask = NULL: if j <= i, a
 * chain; bits of nodes at or past 32 * mask_words are 0).  For query head a,
 * kv head a / (heads_q / heads_kv):
 *     s[j] = scale * q . k[j]      over what the node sees
 *     out  = sum_j exp(s[j]) v[j] / sum_j exp(s[j])
 *     lse  = log sum_j exp(s[j])
 * and out = 0, lse = -inf for a node that sees nothing.  Positions in columns
 * at or past table_cols, or whose page is outside the cache, are not seen;
 * whatever their memory holds has no effect.
 *
 * Arithmetic: codes are exact in f16.  The f32 queries are split into two f16
 * parts (bf16 and f16 queries are exact in one) after a power-of-two scale per
 * row; products accumulate in f32, each block's scale is folded in f32, the
 * softmax runs in f32, and its weights times the values' scales enter the
 * second product as two f16 parts (f32 and f16 outputs) or one (bf16 outputs,
 * whose own rounding is eight times coarser).  With more than 32 bf16 query rows
 * a request and kv head (head_dim up to 128), and page tables long enough, keys
 * may enter the first product with 22 bits and values the second with f16's 11;
 * a value that is not finite then makes all of a row that sees it NaN.  Sums are
 * split over the GPU by the call's shape and the lengths alone and joined in a
 * fixed order: same inputs, same bits.
 * Limits here: rows of the cache, (pages - 1) * stride_page + (heads - 1) *
 * stride_head + (page_size - 1) * stride_token, below 2^32 - 1, and positions,
 * table_cols * page_size, below 2^31 - 512.
 */
typedef struct q8kv_attend_s *q8kv_attend_plan_t;

typedef struct {
    const void *q;          /* row r, head a at q + r * q_row + a * q_head (elements) */
    void *out;              /* row r, head a at out + r * out_row + a * out_head, the type of q */
    float *lse;             /* [rows, heads_q], natural logarithm; NULL = not wanted */
    int32_t type;           /* Q8KV_* of q and out */
    int32_t requests;       /* B >= 0 */
    int64_t rows;           /* R: all requests' nodes */
    int64_t q_row, q_head, out_row, out_head; /* >= 0; rows of `out` must not overlap */
    const int32_t *starts;  /* [B + 1], request b's rows are starts[b] .. starts[b+1]-1; NULL: R / B each */
    const int32_t *lengths; /* [B] tokens before the nodes (below 0 counts as 0) */
    const int32_t *table;   /* [B, table_row] page numbers */
    int64_t table_row;
    int32_t table_cols;
    int32_t mask_words;
    const uint32_t *mask;   /* [R, mask_row], or NULL */
    int64_t mask_row;
    float scale;
} q8kv_attend_args_t;

/* out and lse must not overlap the inputs or one another.  heads_q a multiple of heads_kv, at most max_requests requests and max_rows
 * rows in a call (max_requests <= 65536, max_rows <= 2^20).  device -1 = current. */
q8mv_status_t q8kv_attend_plan(q8kv_attend_plan_t *out, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                               int32_t max_requests, int64_t max_rows, int device);
q8mv_status_t q8kv_attend(q8kv_attend_plan_t plan, const q8kv_cache_t *cache, const q8kv_attend_args_t *args,
                          cudaStream_t stream);
/*
 * Calls with many bf16 query rows a request run on a kernel that waits on
 * shared-memory barriers; every wait is bounded (about 2 s).  A call in which one
 * runs out ends with an undefined output; the plan's other calls, checked or not,
 * are as without it.  Synchronises the plan's device, reports in *device_error
 * whether one ran out since the last check (1, else 0) and clears the word.
 */
q8mv_status_t q8kv_attend_check(q8kv_attend_plan_t plan, int32_t *device_error);
/* For tests of the bounded waits only: the bound in nanoseconds (0 restores it). */
q8mv_status_t q8kv_attend_set_wait(q8kv_attend_plan_t plan, uint64_t wait_ns);
/* Synchronises the plan's device, then releases its workspace.  NULL is accepted. */
q8mv_status_t q8kv_attend_destroy(q8kv_attend_plan_t plan);

/*
 * Verification of drafted tokens.  Request b has T_b nodes; node 0 is its
 * newest token, node i >= 1 a drafted token tokens[i] after its node
 * parents[i] < i (numbers within the request).  Row r of logits is the
 * target's for the token after node r.  Per row, with t = temperature[b]
 * (1 if NULL):
 *     z = l * (1 / t)  (f32),  m = max z,  e = expf(z - m),  w = trunc(2^40 e)
 * w and all sums of it are whole numbers, so no order of summation changes a
 * result.  t <= 0 means greedy: z = l, and e = 1 for the first largest, else
 * 0.  NaN logits count as -inf; a row without finite or +inf logits has W = 0.
 *
 * The walk starts at node 0 and tests nodes in index order; only children of
 * the node it stands on are tested, each with its own uniforms[i] in [0, 1).
 * Without draft probabilities (drafted tokens not drawn at random), W the sum
 * of the node's w: child x is accepted if
 *     u * W < w[x]     (as doubles),
 * else w[x] becomes 0 and W loses it.  With draft probabilities (children of a
 * node drawn from row `node` of draft_probs, finite and >= 0), p = e * f32(2^40 / W),
 * a = 0, N = 1 at first, child x is accepted if
 *     (u * q[x]) * N < max(p[x] - a * q[x], 0)     (f32, each step rounded),
 * else a += N, w becomes trunc(2^40 max(p - a q, 0)) and N = sum w / 2^40; if
 * that sum is 0, w stays the target's own and no other child is tested.  An
 * accepted child becomes the node to stand on.  At the end the next token is
 * the first x whose prefix sum of w exceeds min(trunc(uniforms[node 0] * W),
 * W - 1), or -1 if W = 0.  The accepted tokens and the next one are then
 * distributed as the target's own.
 *
 * Outputs: path[starts[b] + k] is the k-th node of the walk (0 first), -1
 * after its end; count[b] the accepted drafts; next_token[b] (-1 for a request
 * without nodes).  Outputs must not overlap inputs or one another.
 */
typedef struct q8kv_verify_s *q8kv_verify_plan_t;

typedef struct {
    const void *logits;      /* [R, vocab] of `type`, row stride logits_row */
    const float *draft_probs;/* [R, vocab], row stride draft_row, or NULL */
    const int32_t *tokens;   /* [R] */
    const int32_t *parents;  /* [R] */
    const float *uniforms;   /* [R] */
    const float *temperature;/* [B] or NULL */
    const int32_t *starts;   /* [B + 1] or NULL: R / B nodes each */
    int32_t *path;           /* [R] */
    int32_t *count;          /* [B] */
    int32_t *next_token;     /* [B] */
    int64_t logits_row, draft_row;
    int64_t rows;
    int32_t requests;
    int32_t vocab;
    int32_t type;            /* Q8KV_* of logits */
    int32_t reserved;        /* 0 */
} q8kv_verify_args_t;

/* vocab 1 .. 2^22, max_requests <= 65535, max_rows <= 2^20 */
q8mv_status_t q8kv_verify_plan(q8kv_verify_plan_t *out, int32_t max_requests, int64_t max_rows, int32_t vocab,
                               int device);
q8mv_status_t q8kv_verify(q8kv_verify_plan_t plan, const q8kv_verify_args_t *args, cudaStream_t stream);
q8mv_status_t q8kv_verify_destroy(q8kv_verify_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* Q8KV_H */
