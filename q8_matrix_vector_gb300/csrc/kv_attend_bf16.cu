// The draft-tree attention kernels of bf16 queries and outputs: weights times scales in one f16 part.  Two parts bring
// the outputs nearer to a plain program's in 32 bits (8.6e-4 of their norm to 0.6e-4, where the rounding to bf16 is
// 1.7e-3; the error against 64 bits falls by less than 2 %) and cost 32 requests of 180 .. 8100 tokens 71.0 us in
// place of 67.1, 12 rows a request 42.7 in place of 37.2, 32 rows 67.1 in place of 57.9.
#include "kv_attend.cuh"

namespace kv {

AttendVariant attend_variant_bf16(int dim, AttendShape shape) { return attend_variant_of<__nv_bfloat16, 1, 1>(dim, shape); }

}  // namespace kv
