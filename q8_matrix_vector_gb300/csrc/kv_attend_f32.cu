// The draft-tree attention kernels of f32 queries and outputs.
#include "kv_attend.cuh"

namespace kv {

AttendVariant attend_variant_f32(int dim, AttendShape shape) { return attend_variant_of<float, 2, 2>(dim, shape); }

}  // namespace kv
