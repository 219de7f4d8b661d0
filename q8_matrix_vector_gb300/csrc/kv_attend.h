// Parameters and launch of the draft-tree attention kernel (kv_attend.cuh).
// Internal to the library; the C ABI reaches it through q8kv_attend.
#pragma once

#include "kv.h"

namespace kv {

constexpr int kRowTiles[] = {1, 2, 4};  // variants: an item has 8, 16 or 32 query rows (node, head of the group)
constexpr int kWarps = 4;        // warps of a CTA, each with its own keys
constexpr int kStepKeys = 32;    // keys a warp takes at a time
constexpr int kTileKeys = kWarps * kStepKeys;
constexpr int kStages = 2;       // steps in flight per warp
constexpr int kPartExtra = 4;    // of a partial row: its maximum and sum, and 16-byte alignment
constexpr int kItemUnits = 2;    // an item's fixed cost (start of its keys, q, join) in tiles

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
};

// One variant of the kernel: dim up to 64, 128 or 256, and row tiles.  The parts
// of q and of the weights go by the type (see q8kv.h), a translation unit each.
struct AttendVariant {
    void (*fn)(AttendParams) = nullptr;
    int smem = 0;
};
AttendVariant attend_variant_f32(int dim, int row_tiles);
AttendVariant attend_variant_f16(int dim, int row_tiles);
AttendVariant attend_variant_bf16(int dim, int row_tiles);

}  // namespace kv
