// The draft-tree attention kernels of bf16 queries and outputs.
#include "kv_attend.cuh"

namespace kv {

AttendVariant attend_variant_bf16(int dim, AttendShape shape) { return attend_variant_of<__nv_bfloat16, 1, 1>(dim, shape); }

}  // namespace kv
