// Parameters and launch of the draft-tree attention kernel (kv_attend.cuh).
// Internal to the library; the C ABI reaches it through q8kv_attend.
#pragma once

#include "kv.h"

namespace kv {

constexpr int kWarps = 4;        // warps of a CTA, each with its own keys
constexpr int kStepKeys = 32;    // keys a warp takes at a time
constexpr int kStages = 2;       // steps in flight per warp
constexpr int kPartExtra = 4;    // of a partial row: its maximum and sum, and 16-byte alignment
constexpr int kJoinGroup = 8;    // parts of a cut item that one CTA joins at once
constexpr int kItemUnits = 3;    // an item's fixed cost (start of its keys, q, join) in tiles: of 0, 1, 2, 3, 4, 6 the best
                                 // for 32 requests of 180 .. 8100 tokens (84.4, 72.4, 67.5, 67.3, 67.6, 70.3 us)

struct AttendParams {
    Cache c;
    const void *q;
    void *out;
    float *lse;
    int64_t q_row, q_head, out_row, out_head;
    const int32_t *starts;
    const int32_t *lengths;
    const int32_t *table;
    int64_t table_row;
    const uint32_t *mask;
    int64_t mask_row;
    int64_t rows;
    int table_cols, mask_words;
    int requests, heads_q, group;
    float scale_log2;   // scale * log2(e)
    uint32_t page_mul, page_shift;  // position / page_size = (umulhi(position, mul) + position) >> shift
    float *partial;     // 2 per CTA: [rows of an item][dim + kPartExtra]
    unsigned *tickets;  // one per item
    int tickets_n;
    unsigned *group_tickets;  // two per kJoinGroup CTAs
    int *err;           // the plan's error word, and the bound on waits (kRows128)
    uint64_t wait_ns;
    int dim;            // elements of a head (kRows128; the Q4_0 cache's rows are shorter)
    int q_vec, out_vec; // 16-byte loads of eight queries, stores of eight outputs are aligned (kRows128)
};

// What an item is: 8 or 16 query rows (node, head of the group) of one kv head
// whose keys the warps share, 8 rows of four kv heads, one for each warp, or 128
// rows of one kv head on the tensor-memory path (kv_attend_tc.cuh).
enum AttendShape { kRows8 = 0, kRows16, kHeads4, kRows128, kAttendShapes };

// One variant of the kernel: dim up to 64, 128 or 256, and a shape (kRows16 and
// kRows128: dim up to 128; kRows128: bf16).  The parts of q and of the weights go
// by the type (see q8kv.h), a translation unit each.
struct AttendVariant {
    void (*fn)(AttendParams) = nullptr;
    int smem = 0;
    int threads = kWarps * 32;
    int part = 0;  // floats of a partial result
};
AttendVariant attend_variant_f32(int dim, AttendShape shape);
AttendVariant attend_variant_f16(int dim, AttendShape shape);
AttendVariant attend_variant_bf16(int dim, AttendShape shape);
AttendVariant attend_variant_tc(int dim);

}  // namespace kv
