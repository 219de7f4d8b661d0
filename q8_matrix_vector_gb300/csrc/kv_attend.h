// Parameters and launch of the draft-tree attention kernel (kv_attend.cuh).
// Internal to the library; the C ABI reaches it through q8kv_attend.
#pragma once

#include "kv.h"

namespace kv {

constexpr int kTileRows = 16;    // query rows (node, head of the group) of one item
constexpr int kWarps = 4;        // warps of a CTA, each with its own keys
constexpr int kStepKeys = 32;    // keys a warp takes at a time
constexpr int kTileKeys = kWarps * kStepKeys;
constexpr int kStages = 2;       // steps in flight per warp

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
    float *partial;     // 2 per CTA: [16 rows][dim + 2]
    unsigned *tickets;  // one per item
    int tickets_n;
};

// Launches the kernel for `type`; grid = the CTAs that the plan sized its workspace for.
cudaError_t attend_launch(const AttendParams &p, int type, int grid, cudaStream_t stream);
// Resident CTAs per SM of the variant for (dim, type).
cudaError_t attend_occupancy(int dim, int type, int *ctas);

}  // namespace kv
