// Plan, checks and launch of the draft-tree attention (kv_attend.cuh).
#include "kv_attend.h"

#include <algorithm>
#include <new>

namespace kv {

namespace {

AttendVariant variant(int dim, int type, AttendShape shape) {
    if (shape == kRows128) return type == Q8KV_BF16 ? attend_variant_tc(dim) : AttendVariant{};
    return type == Q8KV_F32   ? attend_variant_f32(dim, shape)
           : type == Q8KV_F16 ? attend_variant_f16(dim, shape)
                              : attend_variant_bf16(dim, shape);
}

}  // namespace

}  // namespace kv

static constexpr uint64_t kDefaultWaitNs = 2000000000ull;

struct q8kv_attend_s {
    int device = 0;
    int heads_q = 0, heads_kv = 0, dim = 0;
    int max_requests = 0;
    int64_t max_rows = 0;
    kv::AttendVariant variant[3][kv::kAttendShapes];  // per type
    int grid[3][kv::kAttendShapes] = {};              // and their CTAs: every SM full
    int64_t max_items = 0;
    float *partial = nullptr;
    unsigned *tickets = nullptr;
    int *err = nullptr;
    uint64_t wait_ns = kDefaultWaitNs;
};

extern "C" {

q8mv_status_t q8kv_attend_plan(q8kv_attend_plan_t *out, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
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
    q8kv_attend_s *p = new (std::nothrow) q8kv_attend_s();
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
        for (int v = 0; v < kv::kAttendShapes && e == cudaSuccess; ++v) {
            int ctas = 0;
            const kv::AttendVariant k = p->variant[t][v] = kv::variant(head_dim, t, static_cast<kv::AttendShape>(v));
            if (k.fn == nullptr) continue;
            e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, k.fn, k.threads, k.smem);
            p->grid[t][v] = sms * std::max(1, ctas);
            tickets = std::max(tickets, items + 2 * kv::ceil_div(p->grid[t][v], kv::kJoinGroup));
            floats = std::max<int64_t>(floats, 2LL * p->grid[t][v] * k.part);
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

q8mv_status_t q8kv_attend(q8kv_attend_plan_t plan, const q8kv_cache_t *cache, const q8kv_attend_args_t *a,
                          cudaStream_t stream) {
    kv::AttendParams p = {};
    if (plan == nullptr || a == nullptr || !kv::make_cache(cache, &p.c)) return Q8MV_ERR_INVALID_ARG;
    if (p.c.heads != plan->heads_kv || p.c.dim != plan->dim || !kv::valid_type(a->type)) return Q8MV_ERR_INVALID_ARG;
    if (a->requests < 0 || a->requests > plan->max_requests || a->rows < 0 || a->rows > plan->max_rows)
        return Q8MV_ERR_INVALID_ARG;
    if (a->table_cols < 0 || a->table_row < 0 || a->mask_words < 0 || a->mask_row < 0) return Q8MV_ERR_INVALID_ARG;
    const int64_t most = 1LL << 40;
    if (a->q_row < 0 || a->q_row > most || a->q_head < 0 || a->q_head > most || a->out_row < 0 || a->out_row > most ||
        a->out_head < 0 || a->out_head > most || a->table_row > most || a->mask_row > most)
        return Q8MV_ERR_INVALID_ARG;
    // rows of the cache are numbered in 32 bits here
    if (p.c.pages > 0 && (p.c.pages - 1) * p.c.stride_page + (p.c.heads - 1) * p.c.stride_head +
                                 (p.c.page_size - 1) * p.c.stride_token >= 0xFFFFFFFFLL)
        return Q8MV_ERR_INVALID_ARG;
    // and positions in 31
    if (static_cast<int64_t>(a->table_cols) * p.c.page_size > (1LL << 31) - 2 * kv::kWarps * kv::kStepKeys * kv::kStages)
        return Q8MV_ERR_INVALID_ARG;
    if (a->rows == 0 || a->requests == 0) return Q8MV_OK;
    if (a->starts == nullptr && a->rows % a->requests != 0) return Q8MV_ERR_INVALID_ARG;
    const int size = kv::type_size(a->type);
    if (!a->q || !a->out || !a->lengths || (!a->table && a->table_cols > 0)) return Q8MV_ERR_INVALID_ARG;
    if (!kv::aligned(a->q, size) || !kv::aligned(a->out, size) || !kv::aligned(a->lse, 4) ||
        !kv::aligned(a->lengths, 4) || !kv::aligned(a->table, 4) || !kv::aligned(a->mask, 4) ||
        !kv::aligned(a->starts, 4))
        return Q8MV_ERR_INVALID_ARG;
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
    while ((1u << p.page_shift) < static_cast<uint32_t>(p.c.page_size)) ++p.page_shift;
    p.page_mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << p.page_shift) - p.c.page_size)) / p.c.page_size + 1);
    p.partial = plan->partial;
    p.tickets = plan->tickets;
    p.tickets_n = static_cast<int>(plan->max_items);
    p.group_tickets = plan->tickets + plan->max_items;
    p.err = plan->err;
    p.wait_ns = plan->wait_ns;
    p.q_vec = kv::aligned(a->q, 16) && ((a->q_row | a->q_head) & 7) == 0;
    p.out_vec = kv::aligned(a->out, 16) && ((a->out_row | a->out_head) & 7) == 0;
    // By the mean rows of a request, the fewest at a time that hold them: 8 or 16 (16 requests of 700 .. 4000 tokens, 8
    // heads of 128, bf16: 12 rows 47.9 us by 8, 39.2 by 16; 8 rows 32.0 and 37.8).  32 at a time do not fit the
    // registers (32 rows 60 us by 16, 90 by 32), nor do 16 of a head_dim above 128 (as fast as by 8, with spills).
    const int64_t mean = (a->rows + a->requests - 1) / a->requests * p.group;
    // With 8, and a token's heads side by side, each warp can take a head of its own, so that a CTA reads longer
    // stretches: DRAM gives 128-byte pieces of 1 KB rows slowly (1.2 GB of cache, f32: 318 us with one head a CTA,
    // 240 us with four; 0.59 GB: 143 and 119 us).  But four heads' partial results are to be joined instead of one's
    // (0.28 GB of two requests: 68 and 81 us; 5 MB: 11.6 and 16.3 us), so only where the tables reach 0.5 GB.  The host
    // knows the tables' reach, not the lengths: short sequences under tables for long ones pay for it (columns for 131072
    // tokens: one request of 511, 32 heads, 16.1 us and 10.9 under a table of its own size; eight of 600 23.9 and 14.5).
    const int64_t reach = static_cast<int64_t>(a->table_cols) * p.c.page_size;
    const double bytes = static_cast<double>(reach) * a->requests * p.c.heads * (2.0 * p.c.dim + 8.0 * p.c.blocks);
    const bool side_by_side = p.c.stride_head < p.c.stride_token && p.c.heads % kv::kWarps == 0 && bytes >= 5e8;
    // 128 bf16 rows at a time where there are more than 32 (36 rows of the 16 requests above: 75 us, by 16 rows 83;
    // 128 rows: 86 and 189; but 32 rows: 75 and 60), and enough to do: its tiles of 128 keys take longer to fill and to
    // join.  In tiles of 16 rows x 128 keys of the tables' reach, one request of 124 rows: 2048 tiles 45 us, by 16
    // rows 31; four of 64 rows: 4096 tiles 50 and 49; four of 124 rows: 8192 tiles 53 and 82.  (Under columns for 131072
    // tokens one request of 124 rows over 1000 tokens takes 41 us and not 19.6, four of them 36.6 and not 33.7.)
    const double tiles = static_cast<double>(kv::ceil_div(mean, 16) * kv::ceil_div(reach, 128)) * a->requests * p.c.heads;
    const bool wide = a->type == Q8KV_BF16 && p.c.dim <= 128 && mean > 32 && tiles >= 4096;
    const kv::AttendShape v = wide                         ? kv::kRows128
                              : mean <= 8 && side_by_side  ? kv::kHeads4
                              : mean <= 8 || p.c.dim > 128 ? kv::kRows8
                                                           : kv::kRows16;
    const kv::AttendVariant &k = plan->variant[a->type][v];
    k.fn<<<plan->grid[a->type][v], k.threads, k.smem, stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t q8kv_attend_check(q8kv_attend_plan_t p, int32_t *device_error) {
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

q8mv_status_t q8kv_attend_set_wait(q8kv_attend_plan_t p, uint64_t wait_ns) {
    if (p == nullptr || wait_ns > 10000000000ull) return Q8MV_ERR_INVALID_ARG;
    p->wait_ns = wait_ns == 0 ? kDefaultWaitNs : wait_ns;
    return Q8MV_OK;
}

q8mv_status_t q8kv_attend_destroy(q8kv_attend_plan_t p) {
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
