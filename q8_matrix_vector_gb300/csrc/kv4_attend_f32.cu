// The Q4_0 attention kernels of f32 queries and outputs.
#include "kv4_attend.cuh"

namespace kv {

Attend4Variant attend4_variant_f32(int blocks, Attend4Shape shape) { return attend4_variant_of<float, 2, 2>(blocks, shape); }

}  // namespace kv
