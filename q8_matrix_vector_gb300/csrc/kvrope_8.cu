// The kernels that rotate and write to the Q8_0 cache, and that only rotate.
#include "kvrope.h"

namespace kv {

void launch_rotate_8(const StoreParams &p, int type, bool vec, const Shape &s, size_t smem, cudaStream_t stream) {
    launch_rotate<8>(p, type, vec, s, smem, stream);
}

}  // namespace kv
