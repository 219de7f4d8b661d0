// Parameters and variants of the draft-tree attention over the Q4_0 cache
// (kv4_attend.cuh).  Internal to the library; the C ABI reaches it through q4kv_attend.
#pragma once

#include "kv4.h"
#include "kv_attend.h"

namespace kv {

// As AttendParams, whose cache is Cache4::rows here.
struct Attend4Params {
    AttendParams a;
    int dim;  // elements of a head
    uint32_t stride_page, stride_head, stride_token;  // of the cache, modulo 2^32
};

struct Attend4Variant {
    void (*fn)(Attend4Params) = nullptr;
    int smem = 0;
    int rows = 0;  // of an item
};

// 8 or 16 query rows of one kv head at a time, for NB = 2, 3, 4, 6 or 8 stored blocks (16: up to 4); a warp's keys one
// by one, or 16 at a time that follow one another in memory; or 8 rows of four kv heads, one for each warp.
enum Attend4Shape { k4Rows8 = 0, k4Rows16, k4Rows8InTurn, k4Rows16InTurn, k4Heads4, kAttend4Shapes };

Attend4Variant attend4_variant_f32(int blocks, Attend4Shape shape);
Attend4Variant attend4_variant_f16(int blocks, Attend4Shape shape);
Attend4Variant attend4_variant_bf16(int blocks, Attend4Shape shape);
// 128 bf16 query rows at a time (kv_attend_tc.cuh), up to four blocks
AttendVariant attend4_variant_tc(int blocks);

}  // namespace kv
