// The kernels that rotate and write to the Q4_0 cache.
#include "kvrope.h"

namespace kv {

void launch_rotate_4(const StoreParams &p, int type, bool vec, const Shape &s, size_t smem, cudaStream_t stream) {
    launch_rotate<4>(p, type, vec, s, smem, stream);
}

}  // namespace kv
