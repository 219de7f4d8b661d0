// The rotating variants of kv_store_kernel, a translation unit for each cache.
// Internal to the library.
#pragma once

#include "kv_store.cuh"

namespace kv {

void launch_rotate_4(const StoreParams &p, int type, bool vec, const Shape &s, size_t smem, cudaStream_t stream);
void launch_rotate_8(const StoreParams &p, int type, bool vec, const Shape &s, size_t smem, cudaStream_t stream);

template <int BITS>
void launch_rotate(const StoreParams &p, int type, bool vec, const Shape &s, size_t smem, cudaStream_t stream) {
    if (type == Q8KV_F32)
        launch_store<float, BITS, true>(p, vec, s, smem, stream);
    else if (type == Q8KV_F16)
        launch_store<__half, BITS, true>(p, vec, s, smem, stream);
    else
        launch_store<__nv_bfloat16, BITS, true>(p, vec, s, smem, stream);
}

}  // namespace kv
