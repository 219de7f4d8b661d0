// Host side shared by the q8kv translation units: status conversion, argument
// checks and the device guard.  Internal to the library.
#pragma once

#include "../../include/q8kv.h"

#include <cstddef>
#include <cstdint>
#include <cuda_runtime_api.h>

namespace q8i {
// q8mv_status_t of a CUDA error, remembered for q8mv_last_cuda_error (q8mv.cu).
q8mv_status_t cuda_status(cudaError_t e);
}  // namespace q8i

namespace kv {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Memory of one argument, for the checks that outputs meet no input.
struct Range {
    const void *at;
    int64_t bytes;
};

inline bool overlap(const Range &a, const Range &b) {
    if (a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

inline int type_size(int type) { return type == Q8KV_F32 ? 4 : 2; }

inline bool valid_type(int type) { return type == Q8KV_F32 || type == Q8KV_F16 || type == Q8KV_BF16; }

// The cache as the kernels take it: codes of row r at r * dim, scales at r * blocks.
struct Cache {
    int8_t *k_codes;
    float *k_scales;
    int8_t *v_codes;
    float *v_scales;
    int64_t slots;  // pages * page_size
    int64_t stride_page, stride_head, stride_token;
    int pages, page_size, heads, dim, blocks;
};

// Checks a cache description.  Pages are numbered in 32 bits; a cache without
// pages may have null pointers.
inline bool make_cache(const q8kv_cache_t *c, Cache *out) {
    if (c == nullptr || c->reserved != 0) return false;
    if (c->pages < 0 || c->pages >= (1LL << 31) || c->page_size < 1 || c->page_size > 65536) return false;
    if (c->pages * c->page_size >= (1LL << 40)) return false;
    if (c->heads < 1 || c->heads > 65535 || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0)
        return false;
    if (c->stride_page < 1 || c->stride_head < 1 || c->stride_token < 1) return false;
    if (c->pages > 0) {
        // each axis reaches 2^52 rows at most, so that the last row's offset in bytes (256 a row) fits 63 bits
        const int64_t most = 1LL << 52;
        if (c->stride_page > most / c->pages || c->stride_head > most / c->heads || c->stride_token > most / c->page_size)
            return false;
        if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return false;
        if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
            !aligned(c->v_scales, 16))
            return false;
    }
    out->k_codes = c->k_codes;
    out->k_scales = c->k_scales;
    out->v_codes = c->v_codes;
    out->v_scales = c->v_scales;
    out->slots = c->pages * c->page_size;
    out->stride_page = c->stride_page;
    out->stride_head = c->stride_head;
    out->stride_token = c->stride_token;
    out->pages = static_cast<int>(c->pages);
    out->page_size = c->page_size;
    out->heads = c->heads;
    out->dim = c->head_dim;
    out->blocks = (c->head_dim + 31) / 32;
    return true;
}

// Makes `device` (-1 = the current one) current for the scope and checks that
// it is an sm_103 GPU.
class DeviceScope {
   public:
    DeviceScope() = default;
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;
    q8mv_status_t enter(int device);
    ~DeviceScope() {
        if (prev_ >= 0 && prev_ != device_) cudaSetDevice(prev_);
    }
    int device() const { return device_; }

   private:
    int prev_ = -1, device_ = -1;
};

}  // namespace kv
