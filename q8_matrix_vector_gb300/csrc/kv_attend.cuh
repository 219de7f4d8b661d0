// Attention of draft trees over a paged Q8_0 cache (../../include/q8kv.h).
//
//     s[r, j] = scale * sum_b dK[j, b] * ( sum_{e in b} q[r, e] * cK[j, e] )
//     out[r, e] = sum_j P[r, j] * dV[j, b(e)] * cV[j, e] / sum_j P[r, j],   P = exp(s - max)
//
// Work.  An item is (request, kv head, 8 or 16 query rows); its query rows are
// the (node, head of the group) pairs that share the kv head, so a grouped head's
// cache is read once for all of them.  Items times tiles of 128 keys form one
// line of units, and CTA c takes units [c U / G, (c+1) U / G): every CTA has the
// same share whatever the lengths are, an item is cut only where a share ends,
// and a CTA leaves at most two partial results.  The last CTA of a cut item (an
// atomic ticket, nobody waits) joins its parts in order.
//
// A warp.  The warps of a CTA take 32 keys of a tile each and keep their own
// running maximum, sum and dim x rows accumulator, so there is no barrier in the
// loop; each warp fills its own two-step ring with cp.async.  Both products are
// mma.sync m16n8k16 with f16 operands and f32 accumulators, the cache on the side
// of 16 and 8 query rows on the other: few rows waste little, and with more of
// them (NT tiles of 8) a code is converted once for all.
//   * S^T = K Q^T, one 32-element block at a time.  A lane's 8 bytes of a key are
//     its operands of the block's two mma (the order of e within a block is free
//     as long as q has the same).  A byte with its sign bit flipped is, as the bits
//     of an f16, (code + 128) 2^-24: exact without arithmetic.  The 128 sum q is
//     taken off by the accumulator's initial value, 2^-24 by the row's factor, and
//     the block's scale is folded in f32.
//   * O^T = V^T P^T.  The value's scale multiplies P; an 8 x 8 transpose
//     (movmatrix) turns the f16 weights into the second operand.  A lane's words
//     of four keys are re-paired by byte permutes into operands of two keys; here
//     the 128 is subtracted, as a sum of thousands of keys would drown in it.  A
//     lane ends up with 4 neighbouring e of the output per block.
//   * P dV would leave f16's range with the scales.  With 2^(E + 14) just above the
//     scales of a step's keys and the running maximum taken over s + E (log2),
//     P dV stays below 2^14 and is exact enough down to 2^-28 of that; the factor
//     cancels in the quotient.
//
// One token a request, groups of 8, 8 kv heads of 128.  bf16: 32 requests of 180 ..
// 8100 tokens 66.7 us (288 MB, 4.3 TB/s, 64 % of the copy rate), of 8000 tokens each
// 108 us (82 %).  f32, two of 200001 .. 262143: 242 us (1.2 GB, 5.0 TB/s, 73 %; heads
// apart in memory 80 %).  32 heads of one request of 511 tokens: 11.3 us.  Where the
// cache is long, HBM and the latencies of 940 instructions for a warp's 32 keys bound
// it together: shared memory for two steps of keys leaves two CTAs, 8 warps, an SM,
// which issue in 0.44 of the cycles, and the tensor cores, that make the products, are
// idle most of the time.  16 rows at a time are the same: 12 rows of 16 requests of 700
// .. 4000 tokens 37 us (0.40, the tensor cores 13 %), 128 f32 rows 221 us (0.54, 32 %).
// Where the cache is short, the chain lengths -> page -> keys -> join does, 8 us with no
// key at all, and shares of one unit: the 511 tokens' 32 items are cut into 224 of them.
#pragma once

#include "kv_attend.h"
#include "kv_common.cuh"

namespace kv {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d = a b + c
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// f16 pair minus 1152 each: (1024 + byte with flipped sign bit) -> the signed byte
__device__ __forceinline__ uint32_t unbias(uint32_t x) {
    uint32_t y;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x64806480u));
    return y;
}

// transpose of an 8 x 8 matrix of 16-bit elements, lane l holding elements 2 (l % 4) and + 1 of row l / 4
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory of one variant: dim up to DP, NT tiles of 8 query rows, QP parts of
// q, HW kv heads (the warps' own, or one for all warps).
// Row pitches are chosen so that the fragment loads hit 32 banks: keys (8 bytes
// per lane, rows 0..3 per half warp) need a pitch of 32 mod 64 bytes, values (4
// bytes, every second row) 16 mod 64, q (16 bytes, 2 rows a phase) 64 mod 128.
template <int DP, int NT, int QP, int HW>
struct Smem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kTileKeys = kStepKeys * kWarps / HW;
    static constexpr int kBlocks = DP / 32;
    static constexpr int kKPitch = (DP / 32) % 2 ? DP : DP + 32;
    static constexpr int kVPitch = DP + 16;
    static constexpr int kScaleBytes = kStepKeys * kBlocks * 4;
    static constexpr int kStage = kStepKeys * (kKPitch + kVPitch) + 2 * kScaleBytes;
    static constexpr int kRing = kStage * kStages * kWarps;
    // the join of the warps, 8 rows at a time: O, then m and l
    static constexpr int kJoinPitch = DP + 4;
    static constexpr int kJoin = HW == 1 ? kWarps * 8 * kJoinPitch * 4 : 0;
    static constexpr int kQPitch = 2 * DP + ((2 * DP) % 128 == 64 ? 0 : 64);
    static constexpr int kQHead = QP * kRows * kQPitch;
    static constexpr int kQ = HW * kQHead;
    static constexpr int kBiasHead = kRows * kBlocks * 4;
    static constexpr int kBias = HW * kBiasHead;  // -128 * 2^-24 * the block's sum of q
    static constexpr int kTotal = kRing + kJoin + kQ + kBias;
};

// Where a CTA is on the line of units.  An item is kItemUnits units of its fixed
// cost, then its tiles.
struct Place {
    int b;            // request
    int nodes;        // T_b
    int prefix;       // P_b
    int row0;         // first row of the request
    int tiles_r;      // row tiles
    int64_t tiles_k;  // key tiles
    int h, rt;        // head (of the first warp), row tile
    int64_t item;     // number of the item over all requests
    int64_t first;    // the unit of its first tile
};

template <int ROWS, int KEYS>
__device__ __forceinline__ void load_request(const AttendParams &p, int b, Place &w) {
    w.b = b;
    int64_t s, e;
    if (p.starts) {
        s = p.starts[b];
        e = p.starts[b + 1];
        s = s < 0 ? 0 : s > p.rows ? p.rows : s;
        e = e < s ? s : e > p.rows ? p.rows : e;
    } else {
        const int64_t t = p.rows / p.requests;
        s = t * b;
        e = s + t;
    }
    w.row0 = static_cast<int>(s);
    w.nodes = static_cast<int>(e - s);
    w.prefix = max(p.lengths[b], 0);
    // no more than the page table reaches
    const int64_t reach = static_cast<int64_t>(p.table_cols) * p.c.page_size;
    const int64_t keys = min(static_cast<int64_t>(w.prefix) + w.nodes, reach);
    w.tiles_r = static_cast<int>((static_cast<int64_t>(w.nodes) * p.group + ROWS - 1) / ROWS);
    w.tiles_k = max(static_cast<int64_t>(1), (keys + KEYS - 1) / KEYS);
}

template <int HW>
__device__ __forceinline__ int64_t units_of(const AttendParams &p, const Place &w) {
    return static_cast<int64_t>(p.c.heads / HW) * w.tiles_r * (w.tiles_k + kItemUnits);
}

// What joining needs of an item's parts.
struct Split {
    int64_t units, ctas;
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * units / ctas; }
    __device__ __forceinline__ int64_t owner(int64_t u) const { return ((u + 1) * ctas - 1) / units; }
};

constexpr uint32_t kNoRow = 0xFFFFFFFFu;  // of a key that is not there

// NB scales of one key
template <int NB>
__device__ __forceinline__ void load_scales(const float *p, float (&d)[NB]) {
    if constexpr (NB % 4 == 0) {
#pragma unroll
        for (int b = 0; b < NB; b += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + b);
            d[b] = x.x;
            d[b + 1] = x.y;
            d[b + 2] = x.z;
            d[b + 3] = x.w;
        }
    } else {
        static_assert(NB == 2, "dim up to 64, 128 or 256");
        const float2 x = *reinterpret_cast<const float2 *>(p);
        d[0] = x.x;
        d[1] = x.y;
    }
}

// Which of 32 keys query row idx (node * group + head) of a request sees, some of
// them drafted; the first key is drafted node j0 (below 0: so far before the first).
static __device__ __noinline__ uint32_t sees(const uint32_t *mask, int64_t mask_row, int mask_words, int group, int nodes,
                                      int row0, int j0, int idx) {
    const int node = idx / group;
    if (node >= nodes) return 0;  // a row past the request's last
    if (mask == nullptr) {
        const int n = node + 1 - j0;  // keys seen
        return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
    }
    const uint32_t *mw = mask + (static_cast<int64_t>(row0) + node) * mask_row;
    auto word = [&](int k) -> uint32_t { return k < mask_words ? __ldg(mw + k) : 0u; };
    if (j0 >= 0) return __funnelshift_r(word(j0 >> 5), word((j0 >> 5) + 1), j0 & 31);
    return (word(0) << -j0) | ((1u << -j0) - 1u);  // keys below -j0 are prefix
}

// LIVE of the DP / 32 blocks are computed with: the rest lies past the head.
template <typename T, int DP, int NT, int QP, int PP, int HW, int LIVE>
__global__ void __launch_bounds__(kWarps * 32, DP == 64 && NT == 1 ? 3 : 2) q8kv_attend_kernel(const AttendParams p) {
    using S = Smem<DP, NT, QP, HW>;
    static_assert(HW == 1 || (HW == kWarps && NT == 1), "one head for all warps, or one each with 8 rows");
    constexpr int NB = S::kBlocks, ROWS = S::kRows, KEYS = S::kTileKeys;
    constexpr int TILES = HW == 1 ? NT : HW;  // of 8 rows in a partial result
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scan_units[kWarps], scan_items[kWarps];
    __shared__ int64_t start_b, start_item, start_unit;
    __shared__ float row_mul[HW * ROWS];
    __shared__ int is_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    float *jo = reinterpret_cast<float *>(smem + S::kRing);  // [warp][8 rows][kJoinPitch]
    unsigned char *q_sm = smem + S::kRing + S::kJoin;
    float *bias_sm = reinterpret_cast<float *>(q_sm + S::kQ);  // [row / 2][block][row % 2]

    // ---- the CTA's share of the line of units
    Split split;
    int64_t u, u_end;
    Place w;
    {
        const int per = (p.requests + kWarps * 32 - 1) / (kWarps * 32);
        const int b0 = min(tid * per, p.requests), b1 = min(b0 + per, p.requests);
        int64_t units = 0, items = 0;
        for (int b = b0; b < b1; ++b) {
            load_request<ROWS, KEYS>(p, b, w);
            units += units_of<HW>(p, w);
            items += static_cast<int64_t>(p.c.heads / HW) * w.tiles_r;
        }
        int64_t iu = units, ii = items;  // inclusive over the warp
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t a = __shfl_up_sync(~0u, iu, d), b = __shfl_up_sync(~0u, ii, d);
            if (lane >= d) {
                iu += a;
                ii += b;
            }
        }
        if (lane == 31) {
            scan_units[warp] = iu;
            scan_items[warp] = ii;
        }
        __syncthreads();
        int64_t total = 0, before_u = 0, before_i = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) {
                before_u += scan_units[i];
                before_i += scan_items[i];
            }
            total += scan_units[i];
        }
        if (total == 0) return;
        split.units = total;
        split.ctas = min(static_cast<int64_t>(gridDim.x), total);
        if (blockIdx.x >= split.ctas) return;
        u = split.begin(blockIdx.x);
        u_end = split.begin(blockIdx.x + 1);
        before_u += iu - units;
        before_i += ii - items;
        if (u >= before_u && u < before_u + units) {  // exactly one thread
            int b = b0;
            for (; b < b1; ++b) {
                load_request<ROWS, KEYS>(p, b, w);
                const int64_t n = units_of<HW>(p, w);
                if (u < before_u + n) break;
                before_u += n;
                before_i += static_cast<int64_t>(p.c.heads / HW) * w.tiles_r;
            }
            start_b = b;
            start_unit = before_u;
            start_item = before_i;
        }
        __syncthreads();
        load_request<ROWS, KEYS>(p, static_cast<int>(start_b), w);
        const int64_t k = (u - start_unit) / (w.tiles_k + kItemUnits);  // item within the request
        w.h = static_cast<int>(k / w.tiles_r);
        w.rt = static_cast<int>(k - static_cast<int64_t>(w.h) * w.tiles_r);
        w.h *= HW;
        w.item = start_item + k;
        w.first = start_unit + k * (w.tiles_k + kItemUnits) + kItemUnits;
    }
    // the item after w
    auto advance = [&](Place &x) {
        x.first += x.tiles_k + kItemUnits;
        ++x.item;
        if (++x.rt == x.tiles_r) {
            x.rt = 0;
            if ((x.h += HW) == p.c.heads) {
                x.h = 0;
                do load_request<ROWS, KEYS>(p, x.b + 1, x);
                while (x.tiles_r == 0);
            }
        }
    };
    const bool wide_scales = (p.c.blocks & 3) == 0;

    // ---- the warp's ring: stage `slot` takes 32 keys, of which the lane's is row `row`
    unsigned char *ring = smem + warp * (S::kStage * kStages);
    // scales past the cache's blocks are never copied: they stay 0
    for (int i = lane; i < S::kStage * kStages / 16; i += 32) reinterpret_cast<uint4 *>(ring)[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
    auto issue = [&](bool any, int slot, uint32_t row) {
        if (any) {
            unsigned char *st = ring + slot * S::kStage;
            const uint32_t sk = static_cast<uint32_t>(__cvta_generic_to_shared(st));
            const uint32_t sv = sk + kStepKeys * S::kKPitch;
            const uint32_t ss = sv + kStepKeys * S::kVPitch;
            constexpr int CPR = DP / 16;         // 16-byte pieces of a row
            constexpr int KPI = 32 / CPR;        // keys of one load of the warp
            const int part = lane % CPR, k0 = lane / CPR;
            const bool live = part * 16 < p.c.dim;
            const int8_t *kc = p.c.k_codes + part * 16, *vc = p.c.v_codes + part * 16;
            const uint32_t dk0 = sk + k0 * S::kKPitch + part * 16, dv0 = sv + k0 * S::kVPitch + part * 16;
#pragma unroll
            for (int j = 0; j < CPR; ++j) {
                const uint32_t r = __shfl_sync(~0u, row, k0 + j * KPI);
                if (r != kNoRow && live) {
                    cp_async16(dk0 + j * KPI * S::kKPitch, kc + static_cast<uint64_t>(r) * static_cast<uint32_t>(p.c.dim));
                    cp_async16(dv0 + j * KPI * S::kVPitch, vc + static_cast<uint64_t>(r) * static_cast<uint32_t>(p.c.dim));
                }
            }
            const uint32_t dk = ss + lane * (NB * 4), dv = dk + S::kScaleBytes;
            if (row != kNoRow) {
                const float *ks = p.c.k_scales + static_cast<uint64_t>(row) * static_cast<uint32_t>(p.c.blocks);
                const float *vs = p.c.v_scales + static_cast<uint64_t>(row) * static_cast<uint32_t>(p.c.blocks);
                if (wide_scales) {
#pragma unroll
                    for (int b = 0; b < (NB + 3) / 4; ++b) {
                        if (b * 4 < p.c.blocks) {
                            cp_async16(dk + b * 16, ks + b * 4);
                            cp_async16(dv + b * 16, vs + b * 4);
                        }
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        if (b < p.c.blocks) {
                            cp_async4(dk + b * 4, ks + b);
                            cp_async4(dv + b * 4, vs + b);
                        }
                    }
                }
            } else {
                // an absent key has scales of 0: whatever codes the ring holds, it adds nothing
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    *reinterpret_cast<float *>(st + (dk - sk) + 4 * b) = 0.0f;
                    *reinterpret_cast<float *>(st + (dv - sk) + 4 * b) = 0.0f;
                }
            }
        }
        cp_commit();
    };

    // What a CTA does of one item: key tiles kt0 .. kt1 - 1, one step of the warp in each.
    struct Work {
        int64_t kt0, kt1;
        int base0, n_steps, keys, h;
        const int32_t *table;
    };
    auto work_of = [&](const Place &x) -> Work {
        Work k;
        k.kt0 = max(u, x.first) - x.first;
        k.kt1 = max(min(u_end, x.first + x.tiles_k) - x.first, k.kt0);
        k.base0 = static_cast<int>(k.kt0) * KEYS + (HW == 1 ? warp * kStepKeys : 0);
        k.n_steps = static_cast<int>(k.kt1 - k.kt0);
        k.keys = static_cast<int>(min(static_cast<int64_t>(x.prefix) + x.nodes,
                                      static_cast<int64_t>(p.table_cols) * p.c.page_size));
        k.h = x.h + (HW == 1 ? 0 : warp);
        k.table = p.table + static_cast<int64_t>(x.b) * p.table_row;
        return k;
    };
    // row number of the lane's key of step i, or kNoRow
    auto find = [&](const Work &k, int i) -> uint32_t {
        const int pos = k.base0 + i * KEYS + lane;
        if (i >= k.n_steps || pos >= k.keys) return kNoRow;
        const uint32_t col = (__umulhi(pos, p.page_mul) + pos) >> p.page_shift;  // pos / page_size
        const int page = __ldg(k.table + col);
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.pages)) return kNoRow;
        return static_cast<uint32_t>(row_of(p.c, page, k.h, pos - static_cast<int>(col) * p.c.page_size));
    };
    uint32_t row_cur[kStages];  // rows of the steps in the ring: their lanes' keys are there
    uint32_t row_next;
    int slot0 = 0;              // stage of the item's first step
    auto begin = [&](const Work &k) {
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            row_cur[i] = find(k, i);
            issue(i < k.n_steps, (slot0 + i) % kStages, row_cur[i]);
        }
        row_next = find(k, kStages - 1);
    };

    Work k = work_of(w);
    begin(k);
    bool first_item = true;  // that has tiles here
    for (;;) {
        const int rows = min(ROWS, w.nodes * p.group - w.rt * ROWS);
        if (k.n_steps > 0) {
            // ---- q rows to shared memory: a power of two per row, then f16 parts
            for (int rr = tid >> 3; rr < HW * ROWS; rr += kWarps * 4) {
                const int l8 = tid & 7, hw = rr / ROWS, r = rr % ROWS;
                const int idx = w.rt * ROWS + r, node = idx / p.group, hq = (w.h + hw) * p.group + idx - node * p.group;
                const T *src = static_cast<const T *>(p.q) + (static_cast<int64_t>(w.row0) + node) * p.q_row + hq * p.q_head;
                float x[DP / 8];
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    const int e = l8 + 8 * i;
                    x[i] = r < rows && e < p.c.dim ? to_f32(src[e]) : 0.0f;
                    top = fmaxf(top, fabsf(x[i]));
                }
#pragma unroll
                for (int d = 1; d < 8; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 13, -100), 100);
                // 2^-ex, and the sign of the scale, so that the rows' factors are positive
                const float down = copysignf(__uint_as_float(static_cast<uint32_t>(127 - ex) << 23), p.scale_log2);
                float sum[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) sum[b] = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    const float y = x[i] * down;
                    const __half hi = __float2half_rn(y);
                    __half *dst = reinterpret_cast<__half *>(q_sm + hw * S::kQHead + r * S::kQPitch) + l8 + 8 * i;
                    *dst = hi;
                    float used = __half2float(hi);
                    if constexpr (QP == 2) {
                        const __half lo = __float2half_rn(y - used);
                        dst[ROWS * S::kQPitch / 2] = lo;
                        used += __half2float(lo);
                    }
                    sum[i / 4] += used;
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int d = 1; d < 8; d *= 2) sum[b] += __shfl_xor_sync(~0u, sum[b], d);
                    if (l8 == 0) bias_sm[hw * (ROWS * NB) + ((r >> 1) * NB + b) * 2 + (r & 1)] = -128.0f / 16777216.0f * sum[b];
                }
                // not 0: a score of -inf has to stay that
                if (l8 == 0)
                    row_mul[rr] = fmaxf(__uint_as_float(static_cast<uint32_t>(127 + ex + 24) << 23) * fabsf(p.scale_log2), 1e-37f);
            }
            __syncthreads();

            float o[NT][NB * 2][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NB * 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[t][i][j] = 0.0f;
            // of rows 8 t + 2c and 8 t + 2c + 1; m: running maximum (log2) plus E
            float m[NT][2], l[NT][2], mul[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    m[t][r] = -INFINITY;
                    l[t][r] = 0.0f;
                    mul[t][r] = row_mul[(HW == 1 ? 0 : warp * ROWS) + 8 * t + 2 * c + r];
                }

            const unsigned char *my_q = q_sm + (HW == 1 ? 0 : warp * S::kQHead);
            const float *my_bias = bias_sm + (HW == 1 ? 0 : warp * (ROWS * NB));
            int slot = slot0;
            for (int i = 0; i < k.n_steps; ++i) {
                // row_cur[0] is step i's; the next free stage takes step i + kStages - 1
                row_cur[kStages - 1] = row_next;
                issue(i + kStages - 1 < k.n_steps, slot == 0 ? kStages - 1 : slot - 1, row_next);
                row_next = find(k, i + kStages);
                cp_wait<kStages - 1>();
                __syncwarp();
                const unsigned char *sk = ring + slot * S::kStage, *sv = sk + kStepKeys * S::kKPitch;
                const float *ks = reinterpret_cast<const float *>(sv + kStepKeys * S::kVPitch);
                const float *vs = ks + kStepKeys * NB;
                const uint32_t there = __ballot_sync(~0u, row_cur[0] != kNoRow);
                const int base = k.base0 + i * KEYS;
                if (there != 0) {
                    // 2^(E + 14) is above the scales of the lane's key, and of all keys
                    uint32_t top_bits = 0;
#pragma unroll
                    for (int b = 0; b < NB; ++b) top_bits = max(top_bits, __float_as_uint(vs[lane * NB + b]) & 0x7FFFFFFFu);
                    const float e_key = static_cast<float>(max(min(static_cast<int>(top_bits >> 23) - 127 + 1 - 14, 114), -100));
                    const float e_all = static_cast<float>(
                        max(min(static_cast<int>(__reduce_max_sync(~0u, top_bits) >> 23) - 127 + 1 - 14, 114), -100));

                    // ---- scores: s[t][2 j + k][r] of key 16 j + 8 k + g and row 8 t + 2c + r
                    float s[NT][4][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float d0[NB], d1[NB];  // scales of keys 16 j + g and 16 j + 8 + g
                        load_scales<NB>(ks + (16 * j + g) * NB, d0);
                        load_scales<NB>(ks + (16 * j + 8 + g) * NB, d1);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 2; ++r) s[t][2 * j][r] = s[t][2 * j + 1][r] = 0.0f;
#pragma unroll
                        for (int b = 0; b < LIVE; ++b) {
                            const uint2 x = *reinterpret_cast<const uint2 *>(sk + (16 * j + g) * S::kKPitch + b * 32 + c * 8);
                            const uint2 y = *reinterpret_cast<const uint2 *>(sk + (16 * j + 8 + g) * S::kKPitch + b * 32 + c * 8);
                            const uint32_t x0 = x.x ^ 0x80808080u, x1 = x.y ^ 0x80808080u;
                            const uint32_t y0 = y.x ^ 0x80808080u, y1 = y.y ^ 0x80808080u;
                            const uint32_t a0[4] = {__byte_perm(x0, 0, 0x4140u), __byte_perm(y0, 0, 0x4140u),
                                                    __byte_perm(x0, 0, 0x4342u), __byte_perm(y0, 0, 0x4342u)};
                            const uint32_t a1[4] = {__byte_perm(x1, 0, 0x4140u), __byte_perm(y1, 0, 0x4140u),
                                                    __byte_perm(x1, 0, 0x4342u), __byte_perm(y1, 0, 0x4342u)};
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const float2 z = *reinterpret_cast<const float2 *>(my_bias + ((4 * t + c) * NB + b) * 2);
                                float part[4] = {z.x, z.y, z.x, z.y};
#pragma unroll
                                for (int q = 0; q < QP; ++q) {
                                    const uint4 qq = *reinterpret_cast<const uint4 *>(
                                        my_q + (q * ROWS + 8 * t + g) * S::kQPitch + b * 64 + c * 16);
                                    mma_f16(part, a0, qq.x, qq.y, part);
                                    mma_f16(part, a1, qq.z, qq.w, part);
                                }
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    s[t][2 * j][r] = fmaf(part[r], d0[b], s[t][2 * j][r]);
                                    s[t][2 * j + 1][r] = fmaf(part[2 + r], d1[b], s[t][2 * j + 1][r]);
                                }
                            }
                        }
                    }
                    // ---- softmax
                    const bool drafts = base + kStepKeys > w.prefix;
                    const bool partial = drafts || there != ~0u;
                    bool moved = false;
                    float z[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float top[2];
                        if (partial) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                uint32_t see = there;
                                if (drafts)
                                    see &= sees(p.mask, p.mask_row, p.mask_words, p.group, w.nodes, w.row0, base - w.prefix,
                                                w.rt * ROWS + 8 * t + 2 * c + r);
                                top[r] = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int key = 8 * k + g;
                                    if (((see >> key) & 1u) == 0) s[t][k][r] = -INFINITY;
                                    // a row's E comes from keys that it sees, so that no other's scale matters
                                    top[r] = fmaxf(top[r], fmaf(s[t][k][r], mul[t][r], __shfl_sync(~0u, e_key, key)));
                                }
                            }
                        } else {
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                top[r] = fmaf(fmaxf(fmaxf(s[t][0][r], s[t][1][r]), fmaxf(s[t][2][r], s[t][3][r])), mul[t][r], e_all);
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
#pragma unroll
                            for (int d = 4; d < 32; d *= 2) top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], d));
                            const float n = fmaxf(m[t][r], top[r]);
                            moved |= n != m[t][r];
                            z[t][r] = n;
                        }
                    }
                    if (__any_sync(~0u, moved)) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float f[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                f[r] = ex2(m[t][r] - (z[t][r] == -INFINITY ? 0.0f : z[t][r]));
                                m[t][r] = z[t][r];
                                l[t][r] *= f[r];
                            }
#pragma unroll
                            for (int k = 0; k < LIVE * 2; ++k) {
                                o[t][k][0] *= f[0];
                                o[t][k][1] *= f[1];
                                o[t][k][2] *= f[0];
                                o[t][k][3] *= f[1];
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float n = z[t][r] == -INFINITY ? 0.0f : -z[t][r];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                s[t][k][r] = ex2(fmaf(s[t][k][r], mul[t][r], n));
                                l[t][r] += s[t][k][r];
                            }
                        }
                    // ---- O^T += V^T (P dV)^T, block by block, 16 keys at a time
                    float dv[4][NB];  // scales of keys 8 k + g
#pragma unroll
                    for (int k = 0; k < 4; ++k) load_scales<NB>(vs + (8 * k + g) * NB, dv[k]);
#pragma unroll
                    for (int b = 0; b < LIVE; ++b) {
                        // The tensor cores cut their f32 sums toward zero.  Over thousands of keys that bias is
                        // 1e-5 of the sum: with f32 or f16 outputs a step's 32 keys are summed apart, and added
                        // with rounding.
                        float acc[NT][2][4];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            // the lane's keys 16 j + {2c, 2c + 1, 2c + 8, 2c + 9}, e = 32 b + 4 g + {0 .. 3}
                            const unsigned char *at = sv + (16 * j + 2 * c) * S::kVPitch + b * 32 + g * 4;
                            const uint32_t v0 = *reinterpret_cast<const uint32_t *>(at);
                            const uint32_t v1 = *reinterpret_cast<const uint32_t *>(at + S::kVPitch);
                            const uint32_t v2 = *reinterpret_cast<const uint32_t *>(at + 8 * S::kVPitch);
                            const uint32_t v3 = *reinterpret_cast<const uint32_t *>(at + 9 * S::kVPitch);
                            uint32_t a[2][4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // byte e of both keys' words into bytes 0 and 2
                                const uint32_t sel = static_cast<uint32_t>(e | ((4 + e) << 8));
                                a[e >> 1][e & 1] = unbias((__byte_perm(v0, v1, sel) & 0x00FF00FFu) ^ 0x64806480u);
                                a[e >> 1][2 + (e & 1)] = unbias((__byte_perm(v2, v3, sel) & 0x00FF00FFu) ^ 0x64806480u);
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                uint32_t wgt[PP][2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float(&pr)[2] = s[t][2 * j + k];
                                    float x0 = pr[0] * dv[2 * j + k][b], x1 = pr[1] * dv[2 * j + k][b];
                                    if (partial) {
                                        // a key that the row does not see keeps weight 0 whatever its scale is
                                        x0 = pr[0] == 0.0f ? 0.0f : x0;
                                        x1 = pr[1] == 0.0f ? 0.0f : x1;
                                    }
                                    const uint32_t h = pack_half2(x0, x1);
                                    wgt[0][k] = transpose8(h);
                                    if constexpr (PP == 2) {
                                        const float2 back = unpack_half2(h);
                                        wgt[1][k] = transpose8(pack_half2(x0 - back.x, x1 - back.y));
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    if constexpr (PP == 2) {
                                        if (j == 0) {
#pragma unroll
                                            for (int k = 0; k < 4; ++k) acc[t][e][k] = 0.0f;
                                        }
                                        mma_f16(acc[t][e], a[e], wgt[0][0], wgt[0][1], acc[t][e]);
                                        mma_f16(acc[t][e], a[e], wgt[1][0], wgt[1][1], acc[t][e]);
                                    } else {
                                        mma_f16(o[t][2 * b + e], a[e], wgt[0][0], wgt[0][1], o[t][2 * b + e]);
                                    }
                                }
                            }
                        }
                        if constexpr (PP == 2) {
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
#pragma unroll
                                    for (int k = 0; k < 4; ++k) o[t][2 * b + e][k] += acc[t][e][k];
                        }
                    }
                }
                __syncwarp();
                slot = slot + 1 == kStages ? 0 : slot + 1;
#pragma unroll
                for (int j = 0; j + 1 < kStages; ++j) row_cur[j] = row_cur[j + 1];
            }
            slot0 = slot;
            // ---- the next item's first keys are on their way while the warps of this one are joined
            const Place done = w;
            const Work did = k;
            const bool more = w.first + w.tiles_k < u_end;
            if (more) {
                advance(w);
                k = work_of(w);
                begin(k);
            }
            const bool whole = did.kt0 == 0 && did.kt1 == done.tiles_k;
            const int pitch = p.c.dim + kPartExtra;
            const int64_t slot_p = 2 * static_cast<int64_t>(blockIdx.x) + (first_item ? 0 : 1);
            first_item = false;
            // tile t, row r8 of the item's results: its output row and query head
            auto place_row = [&](int t, int r8, int64_t *row, int *hq) -> bool {
                const int r = HW == 1 ? 8 * t + r8 : r8;
                const int idx = done.rt * ROWS + r, node = idx / p.group;
                *row = static_cast<int64_t>(done.row0) + node;
                *hq = (done.h + (HW == 1 ? 0 : t)) * p.group + idx - node * p.group;
                return r < rows;
            };
            if constexpr (HW > 1) {
                // each warp has whole results of its head
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int r8 = 2 * c + r;
                    int64_t row;
                    int hq;
                    const bool live = place_row(warp, r8, &row, &hq);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) l[0][r] += __shfl_xor_sync(~0u, l[0][r], d);
                    if (live) {
                        T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
                        float *part = p.partial + (slot_p * (8 * TILES) + warp * 8 + r8) * pitch;
                        const float sum = l[0][r], inv = sum > 0.0f ? __frcp_rn(sum) : sum == 0.0f ? 0.0f : sum;
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const int e = 32 * b + 4 * g;
                            const float4 x = make_float4(o[0][2 * b][r], o[0][2 * b][2 + r], o[0][2 * b + 1][r], o[0][2 * b + 1][2 + r]);
                            if (e < p.c.dim) {
                                if (whole) {
                                    out[e] = from_f32<T>(x.x * inv);
                                    out[e + 1] = from_f32<T>(x.y * inv);
                                    out[e + 2] = from_f32<T>(x.z * inv);
                                    out[e + 3] = from_f32<T>(x.w * inv);
                                } else {
                                    *reinterpret_cast<float4 *>(part + e) = x;
                                }
                            }
                        }
                        if (g == 0) {
                            if (!whole) {
                                part[p.c.dim] = m[0][r];
                                part[p.c.dim + 1] = sum;
                            } else if (p.lse) {
                                p.lse[row * p.heads_q + hq] = ((m[0][r] == -INFINITY ? 0.0f : m[0][r]) + log2f(sum)) * 0.693147180559945f;
                            }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t > 0) __syncthreads();
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float *at = jo + (warp * 8 + 2 * c + r) * S::kJoinPitch;
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            *reinterpret_cast<float4 *>(at + 32 * b + 4 * g) =
                                make_float4(o[t][2 * b][r], o[t][2 * b][2 + r], o[t][2 * b + 1][r], o[t][2 * b + 1][2 + r]);
#pragma unroll
                        for (int d = 4; d < 32; d *= 2) l[t][r] += __shfl_xor_sync(~0u, l[t][r], d);
                        if (g == 0) {
                            at[DP] = m[t][r];
                            at[DP + 1] = l[t][r];
                        }
                    }
                    __syncthreads();
                    // kWarps * 4 threads a row
                    constexpr int TPR = kWarps * 4;
                    const int r8 = tid / TPR, lr = tid % TPR;
                    float f[kWarps], top = -INFINITY, sum = 0.0f;
#pragma unroll
                    for (int q = 0; q < kWarps; ++q) top = fmaxf(top, jo[(q * 8 + r8) * S::kJoinPitch + DP]);
                    const float z = top == -INFINITY ? 0.0f : top;
#pragma unroll
                    for (int q = 0; q < kWarps; ++q) {
                        const float *x = jo + (q * 8 + r8) * S::kJoinPitch;
                        f[q] = ex2(x[DP] - z);
                        sum = fmaf(f[q], x[DP + 1], sum);
                    }
                    int64_t row;
                    int hq;
                    if (place_row(t, r8, &row, &hq)) {
                        T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
                        float *part = p.partial + (slot_p * (8 * TILES) + 8 * t + r8) * pitch;
                        const float inv = sum > 0.0f ? __frcp_rn(sum) : sum == 0.0f ? 0.0f : sum;  // NaN stays
#pragma unroll
                        for (int q = 0; q < DP / TPR; ++q) {
                            const int e = lr + TPR * q;
                            if (e < p.c.dim) {
                                float x = 0.0f;
#pragma unroll
                                for (int v = 0; v < kWarps; ++v) x = fmaf(f[v], jo[(v * 8 + r8) * S::kJoinPitch + e], x);
                                if (whole)
                                    out[e] = from_f32<T>(x * inv);
                                else
                                    part[e] = x;
                            }
                        }
                        if (lr == 0) {
                            if (!whole) {
                                part[p.c.dim] = top;
                                part[p.c.dim + 1] = sum;
                            } else if (p.lse) {
                                p.lse[row * p.heads_q + hq] = (z + log2f(sum)) * 0.693147180559945f;
                            }
                        }
                    }
                }
            }
            // (an item past the tickets exists only if `starts` is not ascending: it has no output)
            if (!whole && done.item < p.tickets_n) {
                constexpr int PR = 8 * TILES, TPR = kWarps * 32 / PR, V = DP / 4 / TPR;  // rows, threads a row, float4 a thread
                const int pr = tid / TPR, lr = tid % TPR;
                int64_t row;
                int hq;
                const bool live = place_row(pr / 8, pr % 8, &row, &hq);
                // Adds n parts, the first at slot `head`, the i-th at slot `at + i * step`: to the output, or to the
                // first part's place.
                auto join = [&](int n, int64_t head, int64_t at, int64_t step, bool last) {
                    const float *from = p.partial + (at * PR + pr) * pitch, *from0 = p.partial + (head * PR + pr) * pitch;
                    step *= PR * pitch;
                    float top = -INFINITY, sum = 0.0f, x[V][4];
#pragma unroll
                    for (int q = 0; q < V; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[q][e] = 0.0f;
                    if (live) {
                        for (int i = 0; i < n; ++i) top = fmaxf(top, __ldcg((i == 0 ? from0 : from + i * step) + p.c.dim));
                        const float z = top == -INFINITY ? 0.0f : top;
#pragma unroll (V <= 2 ? 8 : 4)
                        for (int i = 0; i < n; ++i) {
                            const float *part = i == 0 ? from0 : from + i * step;
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part + p.c.dim));
                            const float f = ex2(ml.x - z);
                            sum = fmaf(f, ml.y, sum);
#pragma unroll
                            for (int q = 0; q < V; ++q) {
                                const int e0 = 4 * (lr + TPR * q);
                                if (e0 < p.c.dim) {
                                    const float4 y = __ldcg(reinterpret_cast<const float4 *>(part + e0));
                                    x[q][0] = fmaf(f, y.x, x[q][0]);
                                    x[q][1] = fmaf(f, y.y, x[q][1]);
                                    x[q][2] = fmaf(f, y.z, x[q][2]);
                                    x[q][3] = fmaf(f, y.w, x[q][3]);
                                }
                            }
                        }
                    }
                    __syncwarp();  // a row's threads have read the first part
                    if (live && last) {
                        const float inv = sum > 0.0f ? __frcp_rn(sum) : sum == 0.0f ? 0.0f : sum;
                        T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
#pragma unroll
                        for (int q = 0; q < V; ++q)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (4 * (lr + TPR * q) < p.c.dim) out[4 * (lr + TPR * q) + e] = from_f32<T>(x[q][e] * inv);
                        if (lr == 0 && p.lse)
                            p.lse[row * p.heads_q + hq] = ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * 0.693147180559945f;
                    } else if (live) {
                        float *to = p.partial + (head * PR + pr) * pitch;
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            if (4 * (lr + TPR * q) < p.c.dim)
                                *reinterpret_cast<float4 *>(to + 4 * (lr + TPR * q)) = make_float4(x[q][0], x[q][1], x[q][2], x[q][3]);
                        if (lr == 0) {
                            to[p.c.dim] = top;
                            to[p.c.dim + 1] = sum;
                        }
                    }
                };
                // true in the CTA that is the last of n to come
                auto arrive = [&](unsigned *ticket, unsigned n) -> bool {
                    __threadfence();
                    __syncthreads();
                    if (tid == 0) {
                        const unsigned t = atomicAdd(ticket, 1u);
                        is_last = t == n - 1;
                        if (is_last) *ticket = 0;
                    }
                    __syncthreads();
                    const bool yes = is_last;
                    if (yes) __threadfence();
                    return yes;
                };
                // Parts c0 .. c1.  Up to kJoinGroup of them are joined at once; more are joined in groups of CTAs
                // whose numbers agree but for the last bits, by each group's last, and then the groups.
                const int c0 = static_cast<int>(split.owner(done.first)), c1 = static_cast<int>(split.owner(done.first + done.tiles_k - 1));
                const int slot_c0 = split.begin(c0) >= done.first - kItemUnits ? 2 * c0 : 2 * c0 + 1;
                if (c1 - c0 < kJoinGroup) {
                    if (arrive(p.tickets + done.item, c1 - c0 + 1)) join(c1 - c0 + 1, slot_c0, 2 * c0, 2, true);
                } else {
                    const int grp = blockIdx.x / kJoinGroup, g0 = c0 / kJoinGroup, g1 = c1 / kJoinGroup;
                    const int lo = max(c0, grp * kJoinGroup), hi = min(c1, grp * kJoinGroup + kJoinGroup - 1);
                    // one item may come into a group from its left, and one may begin in it and leave it
                    if (arrive(p.group_tickets + 2 * grp + (c0 < grp * kJoinGroup ? 0 : 1), hi - lo + 1)) {
                        join(hi - lo + 1, lo == c0 ? slot_c0 : 2 * lo, 2 * lo, 2, false);
                        if (arrive(p.tickets + done.item, g1 - g0 + 1))
                            join(g1 - g0 + 1, slot_c0, 2 * kJoinGroup * g0, 2 * kJoinGroup, true);
                    }
                }
            }
            if (!more) break;
        } else {
            // only units of the item's fixed cost are here
            if (w.first + w.tiles_k >= u_end) break;
            advance(w);
            k = work_of(w);
            begin(k);
        }
        __syncthreads();  // the join's reads, before the next item's q
    }
}

// The variants of one type: dim up to 64, 96, 128, 192 or 256, the second and fourth in the layout of the next with
// fewer blocks (4 requests of 67756 tokens, dim 80, f32: 126 us with all of
// them, 111 so; one of 58636, dim 192, f16: 87 and 70).  A test of each block at run time cost full heads 2 to 6 %.
template <typename T, int DP, int QP, int PP, int NT, int HW, int LIVE = DP / 32>
AttendVariant attend_variant_of(int dim) {
    return {q8kv_attend_kernel<T, DP, NT, QP, PP, HW, LIVE>, Smem<DP, NT, QP, HW>::kTotal, kWarps * 32,
            8 * (HW == 1 ? NT : HW) * (dim + kPartExtra)};
}

template <typename T, int QP, int PP, int NT, int HW>
AttendVariant attend_variant_of(int dim) {
    if (dim <= 64) return attend_variant_of<T, 64, QP, PP, NT, HW>(dim);
    if (dim <= 96) return attend_variant_of<T, 128, QP, PP, NT, HW, 3>(dim);
    if (dim <= 128) return attend_variant_of<T, 128, QP, PP, NT, HW>(dim);
    if constexpr (NT == 1) {
        if (dim <= 192) return attend_variant_of<T, 256, QP, PP, NT, HW, 6>(dim);
        return attend_variant_of<T, 256, QP, PP, NT, HW>(dim);
    }
    return {};
}

template <typename T, int QP, int PP>
AttendVariant attend_variant_of(int dim, AttendShape shape) {
    switch (shape) {
        case kRows8: return attend_variant_of<T, QP, PP, 1, 1>(dim);
        case kRows16: return attend_variant_of<T, QP, PP, 2, 1>(dim);
        case kHeads4: return attend_variant_of<T, QP, PP, 1, kWarps>(dim);
        default: return {};
    }
}

}  // namespace kv
