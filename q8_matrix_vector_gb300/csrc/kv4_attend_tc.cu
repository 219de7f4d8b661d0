// The tensor-memory variants of the Q4_0 attention (bf16, up to four stored blocks).
#include "kv_attend_tc.cuh"

namespace kv {

namespace {

template <int DP, int NB4>
AttendVariant variant_tc() {
    return {q8kv_attend_tc_kernel<DP, NB4>, TcSmem<DP, NB4>::kTotal, kTcThreads, TcSmem<DP, NB4>::kPart};
}

}  // namespace

AttendVariant attend4_variant_tc(int blocks) {
    return blocks == 2 ? variant_tc<64, 2>() : blocks == 3 ? variant_tc<128, 3>() : blocks == 4 ? variant_tc<128, 4>() : AttendVariant{};
}

}  // namespace kv
