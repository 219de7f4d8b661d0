// The Q4_0 cache (../../include/q4kv.h) as the kernels take it.  Internal to the
// library.
#pragma once

#include "../../include/q4kv.h"
#include "kv.h"

namespace kv {

// A row's bytes as rows of kv::Cache: `rows.dim` bytes of codes (16 a block) and
// `rows.blocks` 4-byte words of scales (2 scales each).  What only carries rows
// about (moves, copies of pages) takes `rows` alone.
struct Cache4 {
    Cache rows;
    int dim;     // elements of a head
    int blocks;  // stored blocks NB
};

inline int blocks4(int dim) { return dim <= 64 ? 2 : dim <= 96 ? 3 : dim <= 128 ? 4 : dim <= 192 ? 6 : 8; }

inline bool make_cache4(const q4kv_cache_t *c, Cache4 *out) {
    if (c == nullptr || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0) return false;
    const int nb = blocks4(c->head_dim);
    const q8kv_cache_t d = {reinterpret_cast<int8_t *>(c->k_codes), reinterpret_cast<float *>(c->k_scales),
                            reinterpret_cast<int8_t *>(c->v_codes), reinterpret_cast<float *>(c->v_scales),
                            c->pages, c->page_size, c->heads, c->head_dim, c->reserved,
                            c->stride_page, c->stride_head, c->stride_token};
    if (!make_cache(&d, &out->rows)) return false;
    out->dim = c->head_dim;
    out->blocks = nb;
    out->rows.dim = 16 * nb;
    out->rows.blocks = nb == 2 ? 1 : nb <= 4 ? 2 : 4;
    return true;
}

// Moves rows (q8kv_cache_move) of a checked cache; kv_cache.cu.
q8mv_status_t cache_move(const Cache &c, int64_t batch, int64_t path, const int64_t *src, const int64_t *dst,
                         cudaStream_t stream);

// How a store kernel's threads are laid out: threads of one token along x (a
// multiple of 32, at most 256), tokens along y, `tokens` tokens a thread once that
// leaves several blocks an SM, else one; kv_cache.cu.
struct Shape {
    dim3 grid, block;
    bool many;
};
Shape shape(int lanes, int64_t n, int tokens);

bool valid_stride(int64_t s);

}  // namespace kv
