// Plan, checks and launch of the draft-tree attention over the Q4_0 cache (kv4_attend.cuh).
#include "kv4_attend.h"

#include <algorithm>
#include <new>

namespace kv {

namespace {

Attend4Variant variant4(int dim, int type, Attend4Shape shape) {
    const int nb = blocks4(dim);
    return type == Q8KV_F32   ? attend4_variant_f32(nb, shape)
           : type == Q8KV_F16 ? attend4_variant_f16(nb, shape)
                              : attend4_variant_bf16(nb, shape);
}

}  // namespace

}  // namespace kv

static constexpr uint64_t kDefaultWaitNs = 2000000000ull;

struct q4kv_attend_s {
    int device = 0;
    int heads_q = 0, heads_kv = 0, dim = 0;
    int max_requests = 0;
    int64_t max_rows = 0;
    kv::Attend4Variant variant[3][kv::kAttend4Shapes];  // per type
    int grid[3][kv::kAttend4Shapes] = {};               // and their CTAs: every SM full
    kv::AttendVariant tc;                               // bf16, 128 rows
    int tc_grid = 0;
    int64_t max_items = 0;
    float *partial = nullptr;
    unsigned *tickets = nullptr;
    int *err = nullptr;
    uint64_t wait_ns = kDefaultWaitNs;
};

extern "C" {

q8mv_status_t q4kv_attend_plan(q4kv_attend_plan_t *out, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                               int32_t max_requests, int64_t max_rows, int device) {
    if (out == nullptr) return Q8MV_ERR_INVALID_ARG;
    *out = nullptr;
    if (heads_kv < 1 || heads_kv > 65535 || heads_q < heads_kv || heads_q > 65535 || heads_q % heads_kv != 0)
        return Q8MV_ERR_INVALID_ARG;
    if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return Q8MV_ERR_INVALID_ARG;
    if (max_requests < 1 || max_requests > 65536 || max_rows < 1 || max_rows > (1 << 20)) return Q8MV_ERR_INVALID_ARG;
    const int64_t group = heads_q / heads_kv;
    // each request's rows round up to whole tiles
    const int64_t items = (max_rows * group / 8 + max_requests) * heads_kv;
    if (items > (1LL << 28)) return Q8MV_ERR_INVALID_ARG;

    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(device);
    if (st != Q8MV_OK) return st;
    q4kv_attend_s *p = new (std::nothrow) q4kv_attend_s();
    if (p == nullptr) return Q8MV_ERR_OUT_OF_MEMORY;
    p->device = scope.device();
    p->heads_q = heads_q;
    p->heads_kv = heads_kv;
    p->dim = head_dim;
    p->max_requests = max_requests;
    p->max_rows = max_rows;
    p->max_items = items;
    int sms = 0;
    int64_t floats = 0;  // of partial results: two per CTA
    int64_t tickets = items;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, p->device);
    for (int t = 0; t < 3; ++t)
        for (int v = 0; v < kv::kAttend4Shapes && e == cudaSuccess; ++v) {
            int ctas = 0;
            const kv::Attend4Variant k = p->variant[t][v] = kv::variant4(head_dim, t, static_cast<kv::Attend4Shape>(v));
            if (k.fn == nullptr) continue;
            e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, k.fn, kv::kWarps * 32, k.smem);
            p->grid[t][v] = sms * std::max(1, ctas);
            tickets = std::max(tickets, items + 2 * kv::ceil_div(p->grid[t][v], kv::kJoinGroup));
            floats = std::max<int64_t>(floats, 2LL * p->grid[t][v] * k.rows * (head_dim + kv::kPartExtra));
        }
    p->tc = kv::attend4_variant_tc(kv::blocks4(head_dim));
    if (e == cudaSuccess && p->tc.fn != nullptr) {
        int ctas = 0;
        e = cudaFuncSetAttribute(p->tc.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, p->tc.smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, p->tc.fn, p->tc.threads, p->tc.smem);
        p->tc_grid = sms * std::max(1, ctas);
        tickets = std::max(tickets, items + 2 * kv::ceil_div(p->tc_grid, kv::kJoinGroup));
        floats = std::max<int64_t>(floats, 2LL * p->tc_grid * p->tc.part);
    }
    if (e == cudaSuccess) e = cudaMalloc(&p->partial, sizeof(float) * static_cast<size_t>(floats));
    if (e == cudaSuccess) e = cudaMalloc(&p->tickets, sizeof(unsigned) * static_cast<size_t>(tickets));
    if (e == cudaSuccess) e = cudaMemset(p->tickets, 0, sizeof(unsigned) * static_cast<size_t>(tickets));
    if (e == cudaSuccess) e = cudaMalloc(&p->err, sizeof(int));
    if (e == cudaSuccess) e = cudaMemset(p->err, 0, sizeof(int));
    // the zeros, before any stream may use them
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (p->partial) cudaFree(p->partial);
        if (p->tickets) cudaFree(p->tickets);
        if (p->err) cudaFree(p->err);
        delete p;
        return q8i::cuda_status(e);
    }
    *out = p;
    return Q8MV_OK;
}

q8mv_status_t q4kv_attend(q4kv_attend_plan_t plan, const q4kv_cache_t *cache, const q8kv_attend_args_t *a,
                          cudaStream_t stream) {
    kv::Cache4 c = {};
    if (plan == nullptr || a == nullptr || !kv::make_cache4(cache, &c)) return Q8MV_ERR_INVALID_ARG;
    if (c.rows.heads != plan->heads_kv || c.dim != plan->dim || !kv::valid_type(a->type)) return Q8MV_ERR_INVALID_ARG;
    if (a->requests < 0 || a->requests > plan->max_requests || a->rows < 0 || a->rows > plan->max_rows)
        return Q8MV_ERR_INVALID_ARG;
    if (a->table_cols < 0 || a->table_row < 0 || a->mask_words < 0 || a->mask_row < 0) return Q8MV_ERR_INVALID_ARG;
    const int64_t most = 1LL << 40;
    for (int64_t s : {a->q_row, a->q_head, a->out_row, a->out_head})
        if (s < 0 || s > most) return Q8MV_ERR_INVALID_ARG;
    if (a->table_row > most || a->mask_row > most) return Q8MV_ERR_INVALID_ARG;
    // rows of the cache are numbered in 32 bits here
    const kv::Cache &r = c.rows;
    if (r.pages > 0 && (r.pages - 1) * r.stride_page + (r.heads - 1) * r.stride_head + (r.page_size - 1) * r.stride_token >=
                           0xFFFFFFFFLL)
        return Q8MV_ERR_INVALID_ARG;
    // and positions in 31
    if (static_cast<int64_t>(a->table_cols) * r.page_size > (1LL << 31) - 512) return Q8MV_ERR_INVALID_ARG;
    if (a->rows == 0 || a->requests == 0) return Q8MV_OK;
    if (a->starts == nullptr && a->rows % a->requests != 0) return Q8MV_ERR_INVALID_ARG;
    const int size = kv::type_size(a->type);
    if (!a->q || !a->out || !a->lengths || (!a->table && a->table_cols > 0)) return Q8MV_ERR_INVALID_ARG;
    if (!kv::aligned(a->q, size) || !kv::aligned(a->out, size) || !kv::aligned(a->lse, 4) ||
        !kv::aligned(a->lengths, 4) || !kv::aligned(a->table, 4) || !kv::aligned(a->mask, 4) ||
        !kv::aligned(a->starts, 4))
        return Q8MV_ERR_INVALID_ARG;
    kv::Attend4Params pp = {};
    kv::AttendParams &p = pp.a;
    pp.dim = c.dim;
    pp.stride_page = static_cast<uint32_t>(r.stride_page);
    pp.stride_head = static_cast<uint32_t>(r.stride_head);
    pp.stride_token = static_cast<uint32_t>(r.stride_token);
    p.c = c.rows;
    p.q = a->q;
    p.out = a->out;
    p.lse = a->lse;
    p.q_row = a->q_row;
    p.q_head = a->q_head;
    p.out_row = a->out_row;
    p.out_head = a->out_head;
    p.starts = a->starts;
    p.lengths = a->lengths;
    p.table = a->table;
    p.table_row = a->table_row;
    p.table_cols = a->table_cols;
    p.mask = a->mask;
    p.mask_row = a->mask_row;
    p.mask_words = a->mask_words;
    p.rows = a->rows;
    p.requests = a->requests;
    p.heads_q = plan->heads_q;
    p.group = plan->heads_q / plan->heads_kv;
    p.scale_log2 = a->scale * 1.44269504088896341f;
    while ((1u << p.page_shift) < static_cast<uint32_t>(r.page_size)) ++p.page_shift;
    p.page_mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << p.page_shift) - r.page_size)) / r.page_size + 1);
    p.partial = plan->partial;
    p.tickets = plan->tickets;
    p.tickets_n = static_cast<int>(plan->max_items);
    p.group_tickets = plan->tickets + plan->max_items;
    p.err = plan->err;
    p.wait_ns = plan->wait_ns;
    p.dim = c.dim;
    p.q_vec = kv::aligned(a->q, 16) && ((a->q_row | a->q_head) & 7) == 0;
    p.out_vec = kv::aligned(a->out, 16) && ((a->out_row | a->out_head) & 7) == 0;
    // 8 rows at a time or 16, by the mean rows of a request: the fewest that hold them (16 requests of 700 .. 4000 tokens, 8
    // heads of 128, bf16: 12 rows 29.1 us by 16; one token each of groups of 8 is 8 rows); heads above 128 by 8 alone, as 16 do
    // not fit the registers.
    const int64_t mean = (a->rows + a->requests - 1) / a->requests * p.group;
    const bool wide = mean > 8 && c.blocks <= 4;
    // 128 bf16 rows at a time where there are more than 48 and enough to do, in tiles of 16 rows x 128 keys of the tables'
    // reach (kv_attend.cu): the 16 requests above, 48 rows 61.0 us by 16 and 67.2 by 128, 52 rows 77.9 and 69.2, 64 rows 77.9
    // and 69.4.  One request of 124 rows over 8000 tokens (4032 tiles) 34.6 and 40.3, over 16000 (8064) 57.1 and 49.2; four
    // over 2000 (4096) 37.5 and 34.4, over 4000 (8192) 59.4 and 43.4; four of 64 rows over 4000 (4096) 35.7 and 42.6, over 8000
    // (8064) 57.1 and 55.6; 16 of 64 rows over 1000 (4096) 41.8 and 43.4, over 2000 (8192) 62.4 and 55.1.  The host knows the
    // tables' reach, not the lengths: under columns for 131072 tokens one request of 124 rows over 1000 takes 34.8 us and not
    // 16.2, four of them 32.2 and not 28.5.
    const int64_t reach = static_cast<int64_t>(a->table_cols) * r.page_size;
    const double tiles = static_cast<double>(kv::ceil_div(mean, 16) * kv::ceil_div(reach, 128)) * a->requests * r.heads;
    if (a->type == Q8KV_BF16 && plan->tc.fn != nullptr && mean > 48 && tiles >= 6144) {
        plan->tc.fn<<<plan->tc_grid, plan->tc.threads, plan->tc.smem, stream>>>(p);
        return q8i::cuda_status(cudaGetLastError());
    }
    // Sixteen keys are one stretch of memory where a head's tokens of a page are, and start on 16 bytes (64 requests of 180 ..
    // 8100 tokens: 82.7 us, key by key 85.8).
    const int scales = 4 * r.blocks;  // bytes of a row's
    const bool in_turn = r.stride_token == 1 && r.page_size % 16 == 0 && (r.stride_page * scales) % 16 == 0 &&
                         (r.stride_head * scales) % 16 == 0;
    // With 8 rows, and a token's heads side by side, each warp can take a head of its own, so that a CTA reads longer stretches
    // than one head's 64 bytes (kv_attend.cu).  But four heads' parts are to be joined instead of one's, so only where the
    // tables reach 150 MB: 69 MB of two requests 30 us by one head and 43 by four, 138 MB 57 and 58, 277 MB 102 and 87, 1.2 GB
    // 425 and 259; of 64 requests 297 MB 82 and 81, 598 MB 106 and 88; heads of 256 (595 MB) 153 and 147.  (Short sequences
    // under columns for 131072 tokens: one request of 511, 32 heads, 16.5 us and not 10.9, eight of 600 19.7 and not 17.6.)
    const double bytes = static_cast<double>(reach) * a->requests * r.heads * 2.0 * (r.dim + scales);
    const bool side_by_side = r.stride_head < r.stride_token && r.heads % kv::kWarps == 0 && bytes >= 1.5e8;
    const kv::Attend4Shape v = side_by_side && mean <= 8 ? kv::k4Heads4 : in_turn ? (wide ? kv::k4Rows16InTurn : kv::k4Rows8InTurn) : wide ? kv::k4Rows16 : kv::k4Rows8;
    const kv::Attend4Variant &k = plan->variant[a->type][v];
    k.fn<<<plan->grid[a->type][v], kv::kWarps * 32, k.smem, stream>>>(pp);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t q4kv_attend_check(q4kv_attend_plan_t p, int32_t *device_error) {
    if (p == nullptr || device_error == nullptr) return Q8MV_ERR_INVALID_ARG;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(p->device);
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceSynchronize());
    int word = 0;
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaMemcpy(&word, p->err, sizeof(int), cudaMemcpyDeviceToHost));
    if (st == Q8MV_OK && word != 0) {
        st = q8i::cuda_status(cudaMemset(p->err, 0, sizeof(int)));
        if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceSynchronize());
    }
    *device_error = word;
    return st;
}

q8mv_status_t q4kv_attend_set_wait(q4kv_attend_plan_t p, uint64_t wait_ns) {
    if (p == nullptr || wait_ns > 10000000000ull) return Q8MV_ERR_INVALID_ARG;
    p->wait_ns = wait_ns == 0 ? kDefaultWaitNs : wait_ns;
    return Q8MV_OK;
}

q8mv_status_t q4kv_attend_destroy(q4kv_attend_plan_t p) {
    if (p == nullptr) return Q8MV_OK;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(p->device);
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceSynchronize());
    if (p->partial) cudaFree(p->partial);
    if (p->tickets) cudaFree(p->tickets);
    if (p->err) cudaFree(p->err);
    delete p;
    return st;
}

}  // extern "C"
