// Rotary positions (../../include/kvrope.h): plan, checks and launch of the rotating
// variants of kv_store_kernel (kv_store.cuh).
#include "../../include/kvrope.h"
#include "kvrope.h"
#include "strided.h"

#include <cmath>
#include <new>

struct kvrope_s {
    int device = 0;
    int head_dim = 0, half = 0, interleaved = 0;
    float factor = 1.0f;
    float4 *circle = nullptr;   // 256 points
    uint64_t *turns = nullptr;  // behind them
};

namespace kv {

namespace {

// Shape and shared memory of `lanes` lanes a token; 32 KB of angles a block at most.
Shape shape_of(const StoreParams &p, int lanes, int tokens, bool vec, size_t *smem) {
    Shape s = shape(lanes, p.n, tokens);
    const auto bytes = [&](int each) { return static_cast<size_t>(s.block.y) * each * p.half * 2 * sizeof(float); };
    if (!vec || bytes(tokens) > 32768) s.many = false;
    s.grid.x = static_cast<unsigned>(ceil_div(p.n, static_cast<int64_t>(s.block.y) * (s.many ? tokens : 1)));
    *smem = bytes(s.many ? tokens : 1);
    return s;
}

template <typename T>
void launch_q(const StoreParams &p, bool vec, const Shape &s, size_t smem, cudaStream_t stream) {
    if (!vec)
        kv_rotate_kernel<T, false, 1><<<s.grid, s.block, smem, stream>>>(p);
    else if (!s.many)
        kv_rotate_kernel<T, true, 1><<<s.grid, s.block, smem, stream>>>(p);
    else
        kv_rotate_kernel<T, true, kStoreTokens><<<s.grid, s.block, smem, stream>>>(p);
}

// q_lanes comes as q's heads.  One launch, whose blocks along y rotate q behind those that store, a token a lane: with k's
// other halves and the angles two or four take more registers than they are worth, and q in a launch of its own, four
// tokens a lane, gains less than the launch costs (8192 tokens of 8 heads x 128 and 32 of q, bf16, with five blocks an SM and
// cosines to 2^-35: 43.4 us; with two 46.4, four 48.5; two launches 45.0.  As it is now 43.2).
q8mv_status_t launch(StoreParams p, int bits, int type, bool vec, cudaStream_t stream) {
    const int e = vec ? 16 / type_size(type) : 1;
    p.q_items = p.q == nullptr ? 0 : !vec || !p.interleaved ? (p.dim - p.half) / e : p.dim / e;
    const int64_t q_lanes = static_cast<int64_t>(p.q_items) * p.q_lanes;
    if (q_lanes >= (1LL << 31)) return Q8MV_ERR_INVALID_ARG;
    p.q_lanes = static_cast<int>(q_lanes);
    size_t smem;
    Shape s = shape_of(p, p.lanes > 0 ? p.lanes : p.q_lanes, p.lanes > 0 ? 1 : kStoreTokens, vec, &smem);
    if (p.lanes > 0) {
        p.kv_y = static_cast<int>(s.grid.y);
        const int64_t y = p.kv_y + ceil_div(p.q_lanes, s.block.x);
        if (y > 65535) return Q8MV_ERR_INVALID_ARG;
        s.grid.y = static_cast<unsigned>(y);
        if (bits == 4)
            launch_rotate_4(p, type, vec, s, smem, stream);
        else
            launch_rotate_8(p, type, vec, s, smem, stream);
    } else {
        if (s.grid.y > 65535u) return Q8MV_ERR_INVALID_ARG;
        if (type == Q8KV_F32)
            launch_q<float>(p, vec, s, smem, stream);
        else if (type == Q8KV_F16)
            launch_q<__half>(p, vec, s, smem, stream);
        else
            launch_q<__nv_bfloat16>(p, vec, s, smem, stream);
    }
    return q8i::cuda_status(cudaGetLastError());
}

void take(const kvrope_s *plan, StoreParams *p) {
    p->turns = plan->turns;
    p->circle = plan->circle;
    p->factor = plan->factor;
    p->half = plan->half;
    p->interleaved = plan->interleaved;
}

// Whole 16-byte pieces of e elements hold whole pairs, or whole halves of them.
bool whole_pieces(const StoreParams &p, int64_t e) {
    return p.dim % e == 0 && (p.interleaved ? 2 * p.half % e == 0 : p.half % e == 0 && (p.dim - 2 * p.half) % e == 0);
}

// Memory of [n, heads, dim] elements, and of n whole numbers.
Strided tensor(const void *at, int64_t n, int64_t row, int64_t heads, int64_t head, int64_t dim, int size) {
    return {at, n, row * size, heads, head * size, dim * size};
}
Strided numbers(const int64_t *at, int64_t n) { return {at, 1, 0, 1, 0, 8 * n}; }

// Whether `out` is `in` itself, to be rotated in place.
bool same(const Strided &out, const Strided &in) {
    return out.at == in.at && (out.rows == 1 || out.row == in.row) && (out.heads == 1 || out.head == in.head);
}

q8mv_status_t write(kvrope_s *plan, StoreParams &p, int bits, const kvrope_write_args_t *a, cudaStream_t stream) {
    if (p.dim != plan->head_dim) return Q8MV_ERR_INVALID_ARG;
    if (a->n < 0 || a->n >= (1LL << 31) || !valid_type(a->type) || a->heads_q < 0 || a->heads_q > 65535)
        return Q8MV_ERR_INVALID_ARG;
    for (int64_t s : {a->q_row, a->q_head, a->k_row, a->k_head, a->v_row, a->v_head, a->out_row, a->out_head})
        if (!valid_stride(s)) return Q8MV_ERR_INVALID_ARG;
    if (a->n == 0) return Q8MV_OK;
    const int size = type_size(a->type);
    if (!a->k || !a->v || !a->positions || !a->slots || !aligned(a->k, size) || !aligned(a->v, size) ||
        !aligned(a->positions, 8) || !aligned(a->slots, 8))
        return Q8MV_ERR_INVALID_ARG;
    if (a->heads_q > 0) {
        if (!a->q || !a->out || !aligned(a->q, size) || !aligned(a->out, size)) return Q8MV_ERR_INVALID_ARG;
        const Strided out = tensor(a->out, a->n, a->out_row, a->heads_q, a->out_head, p.dim, size);
        const Strided q = tensor(a->q, a->n, a->q_row, a->heads_q, a->q_head, p.dim, size);
        if (folds(out) || (!same(out, q) && meet(out, q)) ||
            meet(out, tensor(a->k, a->n, a->k_row, p.c.heads, a->k_head, p.dim, size)) ||
            meet(out, tensor(a->v, a->n, a->v_row, p.c.heads, a->v_head, p.dim, size)) ||
            meet(out, numbers(a->positions, a->n)) || meet(out, numbers(a->slots, a->n)))
            return Q8MV_ERR_INVALID_ARG;
    }
    take(plan, &p);
    p.in[0] = a->k;
    p.in[1] = a->v;
    p.row[0] = a->k_row;
    p.row[1] = a->v_row;
    p.head[0] = a->k_head;
    p.head[1] = a->v_head;
    p.slots = a->slots;
    p.n = a->n;
    p.lanes = p.c.heads * p.blocks * (size == 4 ? 8 : 4);
    p.positions = a->positions;
    const int64_t e = 16 / size;
    int64_t strides = a->k_row | a->k_head | a->v_row | a->v_head;
    bool vec = aligned(a->k, 16) && aligned(a->v, 16);
    if (a->heads_q > 0) {
        p.q = a->q;
        p.out = a->out;
        p.q_row = a->q_row;
        p.q_head = a->q_head;
        p.out_row = a->out_row;
        p.out_head = a->out_head;
        p.q_lanes = a->heads_q;
        strides |= a->q_row | a->q_head | a->out_row | a->out_head;
        vec = vec && aligned(a->q, 16) && aligned(a->out, 16);
    }
    return launch(p, bits, a->type, vec && (strides & (e - 1)) == 0 && whole_pieces(p, e), stream);
}

}  // namespace

}  // namespace kv

extern "C" {

q8mv_status_t kvrope_plan(kvrope_plan_t *out, int32_t head_dim, int32_t rotary_dim, int32_t interleaved,
                          const uint64_t *turns, float factor, int device) {
    if (out == nullptr) return Q8MV_ERR_INVALID_ARG;
    *out = nullptr;
    if (head_dim < 2 || head_dim > 65536 || rotary_dim < 2 || rotary_dim > head_dim || rotary_dim > 512 || rotary_dim % 2 != 0)
        return Q8MV_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || turns == nullptr || !std::isfinite(factor)) return Q8MV_ERR_INVALID_ARG;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(device);
    if (st != Q8MV_OK) return st;
    kvrope_s *p = new (std::nothrow) kvrope_s();
    if (p == nullptr) return Q8MV_ERR_OUT_OF_MEMORY;
    p->device = scope.device();
    p->head_dim = head_dim;
    p->half = rotary_dim / 2;
    p->interleaved = interleaved;
    p->factor = factor;
    float4 circle[256];
    for (int k = 0; k < 256; ++k) {
        // from the first eighth, so that the axes' points are exact
        const int q = k & 63, quarter = k >> 6;
        const double pi = 3.14159265358979323846;
        double c = q <= 32 ? std::cos(pi * q / 128) : std::sin(pi * (64 - q) / 128);
        double s = q <= 32 ? std::sin(pi * q / 128) : std::cos(pi * (64 - q) / 128);
        for (int i = 0; i < quarter; ++i) {
            const double t = c;
            c = -s;
            s = t;
        }
        const float ch = static_cast<float>(c), sh = static_cast<float>(s);
        circle[k] = make_float4(ch, sh, static_cast<float>(c - ch), static_cast<float>(s - sh));
    }
    const size_t bytes = sizeof(uint64_t) * static_cast<size_t>(p->half);
    cudaError_t e = cudaMalloc(&p->circle, sizeof circle + bytes);
    if (e == cudaSuccess) {
        p->turns = reinterpret_cast<uint64_t *>(p->circle + 256);
        e = cudaMemcpy(p->circle, circle, sizeof circle, cudaMemcpyHostToDevice);
    }
    if (e == cudaSuccess) e = cudaMemcpy(p->turns, turns, bytes, cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (p->circle) cudaFree(p->circle);
        delete p;
        return q8i::cuda_status(e);
    }
    *out = p;
    return Q8MV_OK;
}

q8mv_status_t kvrope_apply(kvrope_plan_t plan, int64_t n, int32_t heads, int32_t type, const void *x, int64_t x_row,
                           int64_t x_head, const int64_t *positions, void *out, int64_t out_row, int64_t out_head,
                           int32_t inverse, cudaStream_t stream) {
    if (plan == nullptr || n < 0 || n >= (1LL << 31) || heads < 0 || heads > 65535 || !kv::valid_type(type))
        return Q8MV_ERR_INVALID_ARG;
    if (!kv::valid_stride(x_row) || !kv::valid_stride(x_head) || !kv::valid_stride(out_row) || !kv::valid_stride(out_head))
        return Q8MV_ERR_INVALID_ARG;
    if (n == 0 || heads == 0) return Q8MV_OK;
    const int size = kv::type_size(type);
    if (!x || !out || !positions || !kv::aligned(x, size) || !kv::aligned(out, size) || !kv::aligned(positions, 8))
        return Q8MV_ERR_INVALID_ARG;
    const kv::Strided to = kv::tensor(out, n, out_row, heads, out_head, plan->head_dim, size);
    const kv::Strided from = kv::tensor(x, n, x_row, heads, x_head, plan->head_dim, size);
    if (kv::folds(to) || (!kv::same(to, from) && kv::meet(to, from)) || kv::meet(to, kv::numbers(positions, n)))
        return Q8MV_ERR_INVALID_ARG;
    kv::StoreParams p = {};
    kv::take(plan, &p);
    p.dim = plan->head_dim;
    p.n = n;
    p.q = x;
    p.out = out;
    p.q_row = x_row;
    p.q_head = x_head;
    p.out_row = out_row;
    p.out_head = out_head;
    p.q_lanes = heads;
    p.positions = positions;
    p.back = inverse != 0;
    const int64_t e = 16 / size;
    const bool vec = kv::aligned(x, 16) && kv::aligned(out, 16) && ((x_row | x_head | out_row | out_head) & (e - 1)) == 0 &&
                     kv::whole_pieces(p, e);
    return kv::launch(p, 8, type, vec, stream);
}

q8mv_status_t kvrope_write_q8(kvrope_plan_t plan, const q8kv_cache_t *cache, const kvrope_write_args_t *args,
                              cudaStream_t stream) {
    kv::StoreParams p = {};
    if (plan == nullptr || args == nullptr || !kv::make_cache(cache, &p.c)) return Q8MV_ERR_INVALID_ARG;
    p.dim = p.c.dim;
    p.blocks = p.c.blocks;
    return kv::write(plan, p, 8, args, stream);
}

q8mv_status_t kvrope_write_q4(kvrope_plan_t plan, const q4kv_cache_t *cache, const kvrope_write_args_t *args,
                              cudaStream_t stream) {
    kv::StoreParams p = {};
    kv::Cache4 c = {};
    if (plan == nullptr || args == nullptr || !kv::make_cache4(cache, &c)) return Q8MV_ERR_INVALID_ARG;
    p.c = c.rows;
    p.dim = c.dim;
    p.blocks = c.blocks;
    return kv::write(plan, p, 4, args, stream);
}

q8mv_status_t kvrope_destroy(kvrope_plan_t p) {
    if (p == nullptr) return Q8MV_OK;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(p->device);
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceSynchronize());
    if (p->circle) cudaFree(p->circle);
    delete p;
    return st;
}

}  // extern "C"
