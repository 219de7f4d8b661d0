// The draft-tree attention kernels of f16 queries and outputs.
#include "kv_attend.cuh"

namespace kv {

AttendVariant attend_variant_f16(int dim, AttendShape shape) { return attend_variant_of<__half, 1, 2>(dim, shape); }

}  // namespace kv
