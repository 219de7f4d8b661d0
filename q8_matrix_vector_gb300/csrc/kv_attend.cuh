// Attention of draft trees over a paged Q8_0 cache (../../include/q8kv.h).
//
//     s[r, j] = scale * sum_b dK[j, b] * ( sum_{e in b} q[r, e] * cK[j, e] )
//     out[r, e] = sum_j P[r, j] * dV[j, b(e)] * cV[j, e] / sum_j P[r, j],   P = exp(s - max)
//
// Work.  An item is (request, kv head, 16 query rows); its query rows are the
// (node, head of the group) pairs that share the kv head, so a grouped head's
// cache is read once for all of them.  Items times tiles of 128 keys form one
// line of units, and CTA c takes units [c U / G, (c+1) U / G): every CTA has the
// same share whatever the lengths are, an item is cut only where a share ends,
// and a CTA leaves at most two partial results.  The last CTA of a cut item (an
// atomic ticket, nobody waits) joins its parts in order.
//
// A warp.  The four warps of a CTA take 32 keys of a tile each and keep their own
// running maximum, sum and 16 x dim accumulator, so there is no barrier in the
// loop; each warp fills its own two-step ring with cp.async.  Both products are
// mma.sync m16n8k16 with f16 operands and f32 accumulators:
//   * int8 codes are exact in f16: the byte with its sign bit flipped, in the low
//     mantissa bits of 1024, minus 1152.
//   * Q K^T: one 32-element block at a time; a lane's 8 bytes of a key are its B
//     operand of the block's two mma (the order of e within a block is free as
//     long as q has the same), and the block's scale is folded into f32.
//   * P V: the value's scale multiplies P, which is the A operand; a lane's words
//     of four keys are re-paired by byte permutes into B operands whose column is
//     every fourth e, which leaves a lane with 8 neighbouring e of the output.
//   * P dV would leave f16's range with the scales.  With 2^(E + 14) just above the
//     scales of a step's keys and the running maximum taken over s + E (log2),
//     P dV stays below 2^14 and is exact enough down to 2^-28 of that; the factor
//     cancels in the quotient.
#pragma once

#include "kv_attend.h"
#include "kv_common.cuh"

namespace kv {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// f16 pair minus 1152 each: (1024 + byte with flipped sign bit) -> the signed byte
__device__ __forceinline__ uint32_t unbias(uint32_t x) {
    uint32_t y;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x64806480u));
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

// Shared memory of one variant.  Row pitches are chosen so that the fragment
// loads hit 32 banks: keys (8 bytes per lane, rows 0..3 per half warp) need a
// pitch of 32 mod 64 bytes, values (4 bytes, every second row) 16 mod 64.
template <int DP>
struct Smem {
    static constexpr int kBlocks = DP / 32;
    static constexpr int kKPitch = (DP / 32) % 2 ? DP : DP + 32;
    static constexpr int kVPitch = DP + 16;
    static constexpr int kScaleBytes = kStepKeys * kBlocks * 4;
    static constexpr int kStage = kStepKeys * (kKPitch + kVPitch) + 2 * kScaleBytes;
    static constexpr int kRing = kStage * kStages * kWarps;
    // the ring is reused by the join of the four warps: O, then m and l
    static constexpr int kJoin = kWarps * kTileRows * (DP + 4) * 4;
    static constexpr int kMain = kRing > kJoin ? kRing : kJoin;
    // q as f16 parts; a row's pitch is 64 mod 128 bytes (16-byte fragment loads)
    static constexpr int kQPitch = 2 * DP + ((2 * DP) % 128 == 64 ? 0 : 64);
    static constexpr int q_bytes(int parts) { return parts * kTileRows * kQPitch; }
    static constexpr int total(int parts) { return kMain + q_bytes(parts); }
};

// Where a CTA is on the line of units.
struct Place {
    int b;            // request
    int nodes;        // T_b
    int prefix;       // P_b
    int row0;         // first row of the request
    int tiles_r;      // row tiles
    int64_t tiles_k;  // key tiles
    int h, rt;
    int64_t item;     // number of the item over all requests
    int64_t first;    // its first unit
};

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
    w.tiles_r = static_cast<int>((static_cast<int64_t>(w.nodes) * p.group + kTileRows - 1) / kTileRows);
    w.tiles_k = max(static_cast<int64_t>(1), (keys + kTileKeys - 1) / kTileKeys);
}

__device__ __forceinline__ int64_t units_of(const AttendParams &p, const Place &w) {
    return static_cast<int64_t>(p.c.heads) * w.tiles_r * w.tiles_k;
}

// What joining needs of an item's parts.
struct Split {
    int64_t units, ctas;
    __device__ __forceinline__ int64_t begin(int64_t c) const { return c * units / ctas; }
    __device__ __forceinline__ int64_t owner(int64_t u) const { return ((u + 1) * ctas - 1) / units; }
};

template <typename T, int DP, int QP, int PP>
__global__ void __launch_bounds__(kWarps * 32, 2) q8kv_attend_kernel(const AttendParams p) {
    using S = Smem<DP>;
    constexpr int NB = S::kBlocks;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scan_units[kWarps], scan_items[kWarps];
    __shared__ int64_t start_b, start_item, start_unit;
    __shared__ float row_mul[kTileRows];
    __shared__ int is_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    unsigned char *q_sm = smem + S::kMain;

    // ---- the CTA's share of the line of units
    Split split;
    int64_t u, u_end;
    Place w;
    {
        const int per = (p.requests + kWarps * 32 - 1) / (kWarps * 32);
        const int b0 = min(tid * per, p.requests), b1 = min(b0 + per, p.requests);
        int64_t units = 0, items = 0;
        for (int b = b0; b < b1; ++b) {
            load_request(p, b, w);
            units += units_of(p, w);
            items += static_cast<int64_t>(p.c.heads) * w.tiles_r;
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
                load_request(p, b, w);
                const int64_t n = units_of(p, w);
                if (u < before_u + n) break;
                before_u += n;
                before_i += static_cast<int64_t>(p.c.heads) * w.tiles_r;
            }
            start_b = b;
            start_unit = before_u;
            start_item = before_i;
        }
        __syncthreads();
        load_request(p, static_cast<int>(start_b), w);
        const int64_t k = (u - start_unit) / w.tiles_k;  // item within the request
        w.h = static_cast<int>(k / w.tiles_r);
        w.rt = static_cast<int>(k - static_cast<int64_t>(w.h) * w.tiles_r);
        w.item = start_item + k;
        w.first = start_unit + k * w.tiles_k;
    }
    const bool wide_scales = (p.c.blocks & 3) == 0;

    for (bool first_item = true; u < u_end; first_item = false) {
        const int64_t item_end = w.first + w.tiles_k;
        const int64_t kt0 = u - w.first, kt1 = min(u_end, item_end) - w.first;
        const int rows = min(kTileRows, w.nodes * p.group - w.rt * kTileRows);
        const int keys = static_cast<int>(min(static_cast<int64_t>(w.prefix) + w.nodes,
                                              static_cast<int64_t>(p.table_cols) * p.c.page_size));

        // ---- q rows to shared memory: a power of two per row, then f16 parts
        {
            const int r = tid >> 3, l8 = tid & 7;
            const int idx = w.rt * kTileRows + r, node = idx / p.group, hq = w.h * p.group + idx - node * p.group;
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
            const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 13, -100), 114);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);  // 2^-ex
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                const float y = x[i] * down;
                const __half hi = __float2half_rn(y);
                __half *dst = reinterpret_cast<__half *>(q_sm + r * S::kQPitch) + l8 + 8 * i;
                *dst = hi;
                if constexpr (QP == 2)
                    dst[kTileRows * S::kQPitch / 2] = __float2half_rn(y - __half2float(hi));
            }
            if (l8 == 0) row_mul[r] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * p.scale_log2;
        }
        __syncthreads();
        const float mul0 = row_mul[g], mul1 = row_mul[g + 8];

        // ---- the warp's keys: steps of 32 from tile to tile
        const int base0 = static_cast<int>(kt0) * kTileKeys + warp * kStepKeys;
        const int n_steps = static_cast<int>(kt1 - kt0);
        unsigned char *ring = smem + warp * (S::kStage * kStages);
        const int32_t *table = p.table + static_cast<int64_t>(w.b) * p.table_row;

        // row number of the lane's key of step i, or -1
        auto find = [&](int i) -> int64_t {
            const int pos = base0 + i * kTileKeys + lane;
            if (i >= n_steps || pos >= keys) return -1;
            const int col = static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.c.page_size));
            const int page = __ldg(table + col);
            if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.pages)) return -1;
            return row_of(p.c, page, w.h, pos - col * p.c.page_size);
        };
        auto issue = [&](int i, int64_t row) {
            if (i < n_steps) {
                unsigned char *st = ring + (i % kStages) * S::kStage;
                const uint32_t sk = static_cast<uint32_t>(__cvta_generic_to_shared(st));
                const uint32_t sv = sk + kStepKeys * S::kKPitch;
                const uint32_t ss = sv + kStepKeys * S::kVPitch;
                constexpr int CPR = DP / 16;         // 16-byte pieces of a row
#pragma unroll
                for (int j = 0; j < CPR; ++j) {
                    const int piece = lane + 32 * j, key = piece / CPR, part = piece % CPR;
                    const int64_t r = __shfl_sync(~0u, row, key);
                    if (r >= 0 && part * 16 < p.c.dim) {
                        cp_async16(sk + key * S::kKPitch + part * 16, p.c.k_codes + r * p.c.dim + part * 16);
                        cp_async16(sv + key * S::kVPitch + part * 16, p.c.v_codes + r * p.c.dim + part * 16);
                    }
                }
                if (row >= 0) {
                    const float *ks = p.c.k_scales + row * p.c.blocks, *vs = p.c.v_scales + row * p.c.blocks;
                    const uint32_t dk = ss + lane * (NB * 4), dv = dk + S::kScaleBytes;
                    if (wide_scales) {
                        for (int b = 0; b < NB / 4; ++b) {
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
                }
            }
            cp_commit();
        };

        float o[NB * 4][4];
#pragma unroll
        for (int i = 0; i < NB * 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // m: running maximum (log2) plus E

        // the lane's two rows' nodes, for the mask
        const int idx0 = w.rt * kTileRows + g, idx1 = idx0 + 8;
        const int node0 = idx0 / p.group, node1 = idx1 / p.group;

        int64_t row_cur[kStages];  // rows of the steps in the ring: their lanes' keys are there
        int64_t row_next;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            row_cur[i] = find(i);
            issue(i, row_cur[i]);
        }
        row_next = find(kStages - 1);
        for (int i = 0; i < n_steps; ++i) {
            // row_cur[0] is step i's; the next free stage takes step i + kStages - 1
            row_cur[kStages - 1] = row_next;
            issue(i + kStages - 1, row_next);
            row_next = find(i + kStages);
            cp_wait<kStages - 1>();
            __syncwarp();
            const unsigned char *st = ring + (i % kStages) * S::kStage;
            const unsigned char *sk = st, *sv = st + kStepKeys * S::kKPitch;
            const float *ks = reinterpret_cast<const float *>(sv + kStepKeys * S::kVPitch);
            const float *vs = ks + kStepKeys * NB;
            const uint32_t there = __ballot_sync(~0u, row_cur[0] >= 0);
            if (there != 0) {
                // largest value scale of the step's keys
                uint32_t top_bits = 0;
                if (row_cur[0] >= 0) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (b < p.c.blocks) top_bits = max(top_bits, __float_as_uint(vs[lane * NB + b]) & 0x7FFFFFFFu);
                }
                // E of the lane's key: 2^(E + 14) is above its scales
                const float e_key = static_cast<float>(max(min(static_cast<int>(top_bits >> 23) - 127 + 1 - 14, 114), -100));
                const float e_f = static_cast<float>(
                    max(min(static_cast<int>(__reduce_max_sync(~0u, top_bits) >> 23) - 127 + 1 - 14, 114), -100));

                // ---- scores: s[j][.] of keys 8 j + {2c, 2c+1}, rows g and g + 8
                float s[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[j][k] = 0.0f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (b < p.c.blocks) {
                        uint32_t a[QP][2][4];  // [part][mma of the block]
#pragma unroll
                        for (int q = 0; q < QP; ++q) {
                            const unsigned char *qb = q_sm + q * (kTileRows * S::kQPitch) + b * 64 + c * 16;
                            const uint4 x0 = *reinterpret_cast<const uint4 *>(qb + g * S::kQPitch);
                            const uint4 x1 = *reinterpret_cast<const uint4 *>(qb + (g + 8) * S::kQPitch);
                            a[q][0][0] = x0.x; a[q][0][1] = x1.x; a[q][0][2] = x0.y; a[q][0][3] = x1.y;
                            a[q][1][0] = x0.z; a[q][1][1] = x1.z; a[q][1][2] = x0.w; a[q][1][3] = x1.w;
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint2 kw = *reinterpret_cast<const uint2 *>(sk + (8 * j + g) * S::kKPitch + b * 32 + c * 8);
                            const uint32_t w0 = kw.x ^ 0x80808080u, w1 = kw.y ^ 0x80808080u;
                            const uint32_t b00 = unbias(__byte_perm(w0, 0x64646464u, 0x4140u));
                            const uint32_t b01 = unbias(__byte_perm(w0, 0x64646464u, 0x4342u));
                            const uint32_t b10 = unbias(__byte_perm(w1, 0x64646464u, 0x4140u));
                            const uint32_t b11 = unbias(__byte_perm(w1, 0x64646464u, 0x4342u));
                            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int q = 0; q < QP; ++q) {
                                mma_f16(part, a[q][0], b00, b01);
                                mma_f16(part, a[q][1], b10, b11);
                            }
                            const float d0 = ks[(8 * j + 2 * c) * NB + b], d1 = ks[(8 * j + 2 * c + 1) * NB + b];
                            s[j][0] = fmaf(part[0], d0, s[j][0]);
                            s[j][1] = fmaf(part[1], d1, s[j][1]);
                            s[j][2] = fmaf(part[2], d0, s[j][2]);
                            s[j][3] = fmaf(part[3], d1, s[j][3]);
                        }
                    }
                }
                // ---- what each row sees of these keys
                const int base = base0 + i * kTileKeys;
                uint32_t see0 = there, see1 = there;
                const bool drafts = base + kStepKeys > w.prefix;
                if (drafts) {
                    auto drafted = [&](int node) -> uint32_t {
                        uint32_t bits = 0;  // bit k: key base + k
                        if (p.mask == nullptr) {
                            const int64_t n = static_cast<int64_t>(w.prefix) + node + 1 - base;  // keys seen
                            bits = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
                        } else {
                            const int j0 = base - w.prefix;  // drafted number of the first key, maybe negative
                            const uint32_t *mw = p.mask + (static_cast<int64_t>(w.row0) + node) * p.mask_row;
                            auto word = [&](int k) -> uint32_t { return k >= 0 && k < p.mask_words ? __ldg(mw + k) : 0u; };
                            if (j0 >= 0) {
                                bits = __funnelshift_r(word(j0 >> 5), word((j0 >> 5) + 1), j0 & 31);
                            } else {  // keys below -j0 are prefix
                                bits = (word(0) << -j0) | ((1u << -j0) - 1u);
                            }
                        }
                        return bits;
                    };
                    see0 &= node0 < w.nodes ? drafted(node0) : 0u;
                    see1 &= node1 < w.nodes ? drafted(node1) : 0u;
                }
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 8 * j + 2 * c;
                    s[j][0] = (see0 >> k) & 1u ? s[j][0] * mul0 : -INFINITY;
                    s[j][1] = (see0 >> (k + 1)) & 1u ? s[j][1] * mul0 : -INFINITY;
                    s[j][2] = (see1 >> k) & 1u ? s[j][2] * mul1 : -INFINITY;
                    s[j][3] = (see1 >> (k + 1)) & 1u ? s[j][3] * mul1 : -INFINITY;
                    if (drafts) {
                        // a row's E comes from keys that it sees, so that no other's scale matters
                        const float ea = __shfl_sync(~0u, e_key, k), eb = __shfl_sync(~0u, e_key, k + 1);
                        t0 = fmaxf(t0, fmaxf(s[j][0] + ea, s[j][1] + eb));
                        t1 = fmaxf(t1, fmaxf(s[j][2] + ea, s[j][3] + eb));
                    } else {
                        t0 = fmaxf(t0, fmaxf(s[j][0], s[j][1]) + e_f);
                        t1 = fmaxf(t1, fmaxf(s[j][2], s[j][3]) + e_f);
                    }
                }
#pragma unroll
                for (int d = 1; d < 4; d *= 2) {
                    t0 = fmaxf(t0, __shfl_xor_sync(~0u, t0, d));
                    t1 = fmaxf(t1, __shfl_xor_sync(~0u, t1, d));
                }
                const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
                const bool moved = n0 != m0 || n1 != m1;
                const float z0 = n0 == -INFINITY ? 0.0f : n0, z1 = n1 == -INFINITY ? 0.0f : n1;
                if (__any_sync(~0u, moved)) {
                    const float f0 = ex2(m0 - z0), f1 = ex2(m1 - z1);
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int k = 0; k < NB * 4; ++k) {
                        o[k][0] *= f0;
                        o[k][1] *= f0;
                        o[k][2] *= f1;
                        o[k][3] *= f1;
                    }
                    m0 = n0;
                    m1 = n1;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j][0] = ex2(s[j][0] - z0);
                    s[j][1] = ex2(s[j][1] - z0);
                    s[j][2] = ex2(s[j][2] - z1);
                    s[j][3] = ex2(s[j][3] - z1);
                    l0 += s[j][0] + s[j][1];
                    l1 += s[j][2] + s[j][3];
                }
                // ---- O += (P dV) V, block by block, 16 keys at a time
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if (b < p.c.blocks) {
                        // The tensor cores cut their f32 sums toward zero.  Over thousands of keys that bias is
                        // 1e-5 of the sum: with f32 or f16 outputs a step's 32 keys are summed apart, and added
                        // with rounding.
                        float acc[4][4];
                        float(&d)[4][4] = PP == 2 ? acc : *reinterpret_cast<float(*)[4][4]>(&o[4 * b]);
                        if constexpr (PP == 2) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int k = 0; k < 4; ++k) acc[e][k] = 0.0f;
                        }
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int k0 = 16 * hh + 2 * c;  // the lane's keys: k0, k0 + 1, k0 + 8, k0 + 9
                            float dv[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int key = k0 + (k & 1) + 8 * (k >> 1);
                                // what the ring holds for an absent key may be anything
                                dv[k] = (there >> key) & 1u ? vs[key * NB + b] : 0.0f;
                            }
                            const float(&pa)[4] = s[2 * hh], (&pb)[4] = s[2 * hh + 1];
                            float x[8] = {pa[0] * dv[0], pa[1] * dv[1], pa[2] * dv[0], pa[3] * dv[1],
                                          pb[0] * dv[2], pb[1] * dv[3], pb[2] * dv[2], pb[3] * dv[3]};
                            if (drafts) {
                                // a key that the row does not see keeps weight 0 whatever its scale is
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    x[k] = pa[k] == 0.0f ? 0.0f : x[k];
                                    x[4 + k] = pb[k] == 0.0f ? 0.0f : x[4 + k];
                                }
                            }
                            uint32_t a[PP][4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                a[0][k] = pack_half2(x[2 * k], x[2 * k + 1]);
                                if constexpr (PP == 2) {
                                    const float2 back = unpack_half2(a[0][k]);
                                    a[1][k] = pack_half2(x[2 * k] - back.x, x[2 * k + 1] - back.y);
                                }
                            }
                            uint32_t v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = *reinterpret_cast<const uint32_t *>(
                                    sv + (k0 + (k & 1) + 8 * (k >> 1)) * S::kVPitch + b * 32 + g * 4);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                // byte e of both keys' words into bytes 0 and 2
                                const uint32_t sel = static_cast<uint32_t>(e | ((4 + e) << 8));
                                const uint32_t b0 =
                                    unbias((__byte_perm(v[0], v[1], sel) & 0x00FF00FFu) ^ 0x64806480u);
                                const uint32_t b1 =
                                    unbias((__byte_perm(v[2], v[3], sel) & 0x00FF00FFu) ^ 0x64806480u);
#pragma unroll
                                for (int q = 0; q < PP; ++q) mma_f16(d[e], a[q], b0, b1);
                            }
                        }
                        if constexpr (PP == 2) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int k = 0; k < 4; ++k) o[4 * b + e][k] += acc[e][k];
                        }
                    }
                }
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k + 1 < kStages; ++k) row_cur[k] = row_cur[k + 1];
        }
        cp_wait<0>();
        // ---- join the four warps
        l0 += __shfl_xor_sync(~0u, l0, 1);
        l1 += __shfl_xor_sync(~0u, l1, 1);
        l0 += __shfl_xor_sync(~0u, l0, 2);
        l1 += __shfl_xor_sync(~0u, l1, 2);
        __syncthreads();  // every warp is done with its ring
        float *jo = reinterpret_cast<float *>(smem);                    // [warp][row][DP + 4]
        {
            float *w0 = jo + (warp * kTileRows + g) * (DP + 4), *w1 = w0 + 8 * (DP + 4);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                // columns 2c and 2c+1 of mma column tile e are e' = 8c + e and 8c + 4 + e
                *reinterpret_cast<float4 *>(w0 + 32 * b + 8 * c) = make_float4(o[4 * b][0], o[4 * b + 1][0], o[4 * b + 2][0], o[4 * b + 3][0]);
                *reinterpret_cast<float4 *>(w0 + 32 * b + 8 * c + 4) = make_float4(o[4 * b][1], o[4 * b + 1][1], o[4 * b + 2][1], o[4 * b + 3][1]);
                *reinterpret_cast<float4 *>(w1 + 32 * b + 8 * c) = make_float4(o[4 * b][2], o[4 * b + 1][2], o[4 * b + 2][2], o[4 * b + 3][2]);
                *reinterpret_cast<float4 *>(w1 + 32 * b + 8 * c + 4) = make_float4(o[4 * b][3], o[4 * b + 1][3], o[4 * b + 2][3], o[4 * b + 3][3]);
            }
            if (c == 0) {
                w0[DP] = m0;
                w0[DP + 1] = l0;
                w1[DP] = m1;
                w1[DP + 1] = l1;
            }
        }
        __syncthreads();
        const bool whole = kt0 == 0 && kt1 == w.tiles_k;
        const int pitch = p.c.dim + 2;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (first_item ? 0 : 1);
        {
            const int r = tid >> 3, l8 = tid & 7;  // 8 threads a row
            float f[kWarps], m = -INFINITY, l = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) m = fmaxf(m, jo[(k * kTileRows + r) * (DP + 4) + DP]);
            const float z = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float *x = jo + (k * kTileRows + r) * (DP + 4);
                f[k] = ex2(x[DP] - z);
                l = fmaf(f[k], x[DP + 1], l);
            }
            if (r < rows) {
                const int idx = w.rt * kTileRows + r, node = idx / p.group, hq = w.h * p.group + idx - node * p.group;
                const int64_t row = static_cast<int64_t>(w.row0) + node;
                T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
                float *part = p.partial + (slot * kTileRows + r) * pitch;
                const float inv = l > 0.0f ? __frcp_rn(l) : l == 0.0f ? 0.0f : l;  // NaN stays
#pragma unroll
                for (int k = 0; k < DP / 8; ++k) {
                    const int e = l8 + 8 * k;
                    if (e < p.c.dim) {
                        float x = 0.0f;
#pragma unroll
                        for (int q = 0; q < kWarps; ++q) x = fmaf(f[q], jo[(q * kTileRows + r) * (DP + 4) + e], x);
                        if (whole)
                            out[e] = from_f32<T>(x * inv);
                        else
                            part[e] = x;
                    }
                }
                if (l8 == 0) {
                    if (!whole) {
                        part[p.c.dim] = m;
                        part[p.c.dim + 1] = l;
                    } else if (p.lse) {
                        p.lse[row * p.heads_q + hq] = (z + log2f(l)) * 0.693147180559945f;
                    }
                }
            }
        }
        // (an item past the tickets exists only if `starts` is not ascending: it has no output)
        if (!whole && w.item < p.tickets_n) {
            const int64_t c0 = split.owner(w.first), c1 = split.owner(item_end - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned t = atomicAdd(p.tickets + w.item, 1u);
                is_last = t == static_cast<unsigned>(c1 - c0);
                if (is_last) p.tickets[w.item] = 0;
            }
            __syncthreads();
            if (is_last) {
                __threadfence();
                const int r = tid >> 3, l8 = tid & 7;
                if (r < rows) {
                    auto part_of = [&](int64_t k) {
                        const int64_t sl = k > c0 || split.begin(k) == w.first ? 2 * k : 2 * k + 1;
                        return p.partial + (sl * kTileRows + r) * pitch;
                    };
                    float m = -INFINITY, l = 0.0f;
                    for (int64_t k = c0; k <= c1; ++k) m = fmaxf(m, __ldcg(part_of(k) + p.c.dim));
                    const float z = m == -INFINITY ? 0.0f : m;
                    float x[DP / 8];
#pragma unroll
                    for (int k = 0; k < DP / 8; ++k) x[k] = 0.0f;
                    for (int64_t k = c0; k <= c1; ++k) {
                        const float *part = part_of(k);
                        const float f = ex2(__ldcg(part + p.c.dim) - z);
                        l = fmaf(f, __ldcg(part + p.c.dim + 1), l);
#pragma unroll
                        for (int q = 0; q < DP / 8; ++q)
                            if (l8 + 8 * q < p.c.dim) x[q] = fmaf(f, __ldcg(part + l8 + 8 * q), x[q]);
                    }
                    const float inv = l > 0.0f ? __frcp_rn(l) : l == 0.0f ? 0.0f : l;
                    const int idx = w.rt * kTileRows + r, node = idx / p.group, hq = w.h * p.group + idx - node * p.group;
                    const int64_t row = static_cast<int64_t>(w.row0) + node;
                    T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
#pragma unroll
                    for (int q = 0; q < DP / 8; ++q)
                        if (l8 + 8 * q < p.c.dim) out[l8 + 8 * q] = from_f32<T>(x[q] * inv);
                    if (l8 == 0 && p.lse) p.lse[row * p.heads_q + hq] = (z + log2f(l)) * 0.693147180559945f;
                }
            }
        }
        // ---- the next item
        u = w.first + kt1;
        if (u < u_end) {
            w.first = item_end;
            ++w.item;
            if (++w.rt == w.tiles_r) {
                w.rt = 0;
                if (++w.h == p.c.heads) {
                    w.h = 0;
                    do load_request(p, w.b + 1, w);
                    while (w.tiles_r == 0);
                }
            }
        }
        __syncthreads();  // the join's reads, before the next item fills the ring and q
    }
}

}  // namespace kv
