// The Q4_0 attention kernels of f16 queries and outputs.
#include "kv4_attend.cuh"

namespace kv {

Attend4Variant attend4_variant_f16(int blocks, Attend4Shape shape) { return attend4_variant_of<__half, 1, 2>(blocks, shape); }

}  // namespace kv
