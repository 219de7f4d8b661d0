// The tensor-memory variants of the draft-tree attention (bf16, dim up to 128).
#include "kv_attend_tc.cuh"

namespace kv {

AttendVariant attend_variant_tc(int dim) {
    if (dim <= 64) return {q8kv_attend_tc_kernel<64, 0>, TcSmem<64, 0>::kTotal, kTcThreads, TcSmem<64, 0>::kPart};
    if (dim <= 128) return {q8kv_attend_tc_kernel<128, 0>, TcSmem<128, 0>::kTotal, kTcThreads, TcSmem<128, 0>::kPart};
    return {};
}

}  // namespace kv
