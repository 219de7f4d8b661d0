// The Q4_0 attention kernels of bf16 queries and outputs.
#include "kv4_attend.cuh"

namespace kv {

Attend4Variant attend4_variant_bf16(int blocks, Attend4Shape shape) { return attend4_variant_of<__nv_bfloat16, 1, 1>(blocks, shape); }

}  // namespace kv
