// Attention of draft trees over a paged Q4_0 cache (../../include/q4kv.h).
//
//     s[r, j] = scale * sum_b dK[j, b] * ( sum_{e in b} q[r, e] * (cK[j, e] - 8) )
//     out[r, e] = sum_j P[r, j] * dV[j, b(e)] * (cV[j, e] - 8) / sum_j P[r, j],   P = exp(s - max)
//
// Work is cut and joined as in kv_attend.cuh: (request, kv head, 8 or 16 query rows)
// items, or 8 rows of four heads, on one line of units, equal shares of it a CTA, parts
// joined by the last to come.  A warp takes 32 keys of a tile of 128, keeps its own maximum, sum and
// accumulators, and fills its own ring with cp.async.  The cache is the first operand
// of mma.sync m16n8k16, 8 rows the second.  What four bits change:
//   * A nibble where it lies in a half word is, as an f16's bits, c 2^-24 or 16 c 2^-24,
//     exactly: `and` alone makes operands of two.  Nibbles 0 and 4, 1 and 5 of a word
//     are pairs, and 2 and 6, 3 and 7 after one shift by 8: five instructions for eight
//     elements.  The 16 of every second pair is taken off q's f16 beforehand, or in the
//     output at the end; 2^-24 with the rows' factors.
//   * The order of a row's bytes (q4kv.h) puts what a lane needs of all blocks in one
//     load: of a key 4 NB bytes (8 elements of each block), of a value 2 NB (4 of each).
//     Values of two keys are paired by one byte permute a word.
//   * The 8 is not subtracted from codes.  Of the scores it is one more product for all
//     blocks, the keys' scales times -8 times the blocks' sums of q (two f16 parts), from
//     which the scores start.  Of the values it is a product of its own, a matrix of -8
//     (-128 where the codes carry 16) with the same weights, whose result is the accumulator
//     that the codes' products start from: one more mma a block in place of eight
//     subtractions.  A step's 32 keys are summed in it and added to the output in f32 with
//     rounding, so that neither the 8s nor the tensor cores' cut sums pile up.  Sums that
//     start from 8s keep 5 bits less of small results, which an f32 output would show (its
//     error was 5e-6 of its norm): for f32 the 8 is subtracted from f16 codes.
//   * bf16: the weights go to f16 once and are transposed once for all blocks, and then
//     multiplied by the values' scales in f16, two at a time: two roundings to 11 bits where
//     the output's own has 8.  f16: the same with the weights in two f16 parts, whose products
//     are again two, to 2^-22.  f32: products in f32, then two parts.
// The weights' scale 2^E (kv_attend.cuh) is taken from the f16 scales' exponents; with 16-bit
// weights small scales are brought up by a power of two first, for all keys of a step.  The
// running maximum moves only when a score is 2^kSlack above it, so that most steps need no
// maximum over the lanes; f16 has the room.
//
// Measured on GB300, groups of 4 or 8 heads of 128, bf16 (copy rate 6792 GB/s): two requests
// of 300k .. 524k tokens 231 us, 4.9 TB/s of the cache; f16 286, f32 343.  64 requests of
// 180 .. 8100 tokens 82 us, 3.7 TB/s; 64 of 8000 141 us, 4.2 TB/s.  What bounds the loop is
// issue: 589 instructions a warp's 32 keys, a third of them masks, shifts and permutes on the
// half-rate pipe, with three warps a scheduler; in the mixed batch an item's start, end and
// join take a quarter of the time.
#pragma once

#include "kv4_attend.h"
#include "kv_attend.cuh"

#include <type_traits>

namespace kv {

// Steps in flight a warp, and CTAs an SM.  8 rows of up to 128: three CTAs (168 registers a thread); with four the registers
// spill in the loop (two requests of 300k .. 524k tokens, bf16: 231 and 242 us; 64 of 180 .. 8100: 82 and 85), and
// three steps with three CTAs gained nothing (an earlier loop: 233.0 and 233.0; 64 requests of 8000: 143.4 and 144.3).  Heads
// of 64: four (64 of 180 .. 8100: 57.6 us with three, 54.7 with four).
constexpr int kStages4 = 2;
constexpr float kSlack = 5.0f;

// Shared memory of one variant: NB stored blocks, NT tiles of 8 query rows, QP parts of q, HW kv heads (the warps' own,
// or one for all warps).
template <int NB, int NT, int QP, int HW>
struct Smem4 {
    static constexpr int kRows = 8 * NT;
    static constexpr int kTileKeys = kStepKeys * kWarps / HW;
    static constexpr int kCodes = 16 * NB;                       // of a row
    static constexpr int kKPitch = NB == 8 ? kCodes + 16 : kCodes;  // 8: rows two apart would share banks
    static constexpr int kScales = NB == 2 ? 4 : NB <= 4 ? 8 : 16;  // bytes of a row's scales
    static constexpr int kStage = kStepKeys * (kKPitch + kCodes + 2 * kScales);
    static constexpr int kRing = kStage * kStages4 * kWarps;
    static constexpr int kJoinPitch = 32 * NB + 4;
    // 8 rows of a warp's results, f32, in the stage that is free when an item ends
    static_assert(8 * kJoinPitch * 4 <= kStage, "a stage holds them");
    static constexpr int kQPitch = 64 * NB + ((64 * NB) % 128 == 64 ? 0 : 64);
    static constexpr int kQHead = QP * kRows * kQPitch;
    static constexpr int kQ = HW * kQHead;
    static constexpr int kBiasHead = kRows * 32;  // 8 pairs of f16 a row
    static constexpr int kBias = HW * kBiasHead;
    static constexpr int kTotal = kRing + kQ + kBias;
    // where the 16-byte piece `c` of value row r is: spread so that the lanes of a load meet no bank twice
    static __host__ __device__ constexpr int v_piece(int r, int c) {
        return NB == 4 ? c ^ (r & 2) : NB == 8 ? c ^ ((r & 3) << 1) : c;
    }
};

// 4 NB bytes of a key, or 2 NB of a value, of this lane
template <int NB>
__device__ __forceinline__ void load_key(const unsigned char *at, uint32_t (&w)[NB]) {
    if constexpr (NB % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NB; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(at + 4 * i);
            w[i] = x.x;
            w[i + 1] = x.y;
            w[i + 2] = x.z;
            w[i + 3] = x.w;
        }
    } else if constexpr (NB % 2 == 0) {
#pragma unroll
        for (int i = 0; i < NB; i += 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(at + 4 * i);
            w[i] = x.x;
            w[i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) w[i] = *reinterpret_cast<const uint32_t *>(at + 4 * i);
    }
}
template <int NB>
__device__ __forceinline__ void load_value(const unsigned char *at, uint32_t (&w)[(NB + 1) / 2]) {
    if constexpr (NB == 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(at);
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
    } else if constexpr (NB == 4) {
        const uint2 x = *reinterpret_cast<const uint2 *>(at);
        w[0] = x.x;
        w[1] = x.y;
    } else if constexpr (NB % 2 == 0) {
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) w[i] = *reinterpret_cast<const uint32_t *>(at + 4 * i);
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(at);
#pragma unroll
        for (int i = 0; i < (NB + 1) / 2; ++i)
            w[i] = h[2 * i] | (2 * i + 1 < NB ? static_cast<uint32_t>(h[2 * i + 1]) << 16 : 0u);
    }
}

// scales of one key, two a word
template <int NB>
__device__ __forceinline__ void load_scales4(const unsigned char *at, uint32_t (&w)[(NB + 1) / 2]) {
    if constexpr (NB > 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(at);
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        if constexpr (NB == 8) w[3] = x.w;
    } else if constexpr (NB > 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(at);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(at);
    }
}
__device__ __forceinline__ float scale_of(uint32_t w, int b) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return b & 1 ? __high2float(h) : __low2float(h);
}

// with constant offsets of both
template <int D, int S>
__device__ __forceinline__ void cp_async16_at(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;" ::"r"(dst), "l"(src), "n"(D), "n"(S) : "memory");
}

// two f32 at a time
__device__ __forceinline__ void add2(float &a, float &b, float x, float y) {
    asm("{.reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
__device__ __forceinline__ void fma2(float &a, float &b, float x, float y, float u, float v) {  // a = a x + u
    asm("{.reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n mov.b64 r, {%4, %5};\n"
        " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y), "f"(u), "f"(v));
}

// Scales whose greatest has the f16 exponent field f (0 counts as 1) are below 2^(E + 9), E = f - 23, so that weights of at
// most 2^(kSlack - E) times scales stay below 2^14.
__device__ __forceinline__ int field_of(uint32_t bits) { return max(static_cast<int>(bits >> 10), 1); }
__device__ __forceinline__ float exponent_of(int field) { return static_cast<float>(field - 23); }
// PACKED: weights, and their products with scales, are f16 themselves.  The field counts as 15 at least, which keeps
// weights at 2^(kSlack + 8) at most; but where it is more than kFine below, the scales are brought up to 15 instead, exactly,
// by 2^-G, and the weights are taken times 2^G, so that small values' products do not end in f16's last bits.  Bringing them up
// takes 3 in a hundred of the time (two requests of 300k .. 524k: 231.5 and 239 us), so it is left out where the largest
// weight times the step's largest scale is 2 or more without it: then a product's own 2^-25 is 2^-24 of the largest or less.
constexpr int kFine = 7;
__device__ __forceinline__ int counted(int field) { return field >= 15 - kFine ? max(field, 15) : field; }
__device__ __forceinline__ int shift_of(int counted_field) { return min(counted_field - 15, 0); }
// Operands of 8 nibbles of the same place in the two halves of a word's nibbles: pairs 0 and 2 as c, 1 and 3 as 16 c, in
// units of 2^-24, or (EXACT) c - 8 and 16 (c - 8) themselves.
template <bool EXACT>
__device__ __forceinline__ uint32_t codes1(uint32_t w) {
    if constexpr (EXACT) {
        uint32_t y;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"((w & 0x000F000Fu) | 0x64006400u), "r"(0x64086408u));
        return y;
    }
    return w & 0x000F000Fu;
}
template <bool EXACT>
__device__ __forceinline__ uint32_t codes16(uint32_t w) {
    if constexpr (EXACT) {
        uint32_t y;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"((w & 0x00F000F0u) | 0x64006400u), "r"(0x64806480u));
        return y;
    }
    return w & 0x00F000F0u;
}

__device__ __forceinline__ uint32_t fma_half2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t y;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
    return y;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

template <typename T, int NB, int NT, int QP, int PP, bool SEG, int HW>
__global__ void __launch_bounds__(kWarps * 32, NB == 2 && NT == 1 ? 4 : NB <= 4 && NT == 1 ? 3 : 2)
    q4kv_attend_kernel(const Attend4Params pp) {
    using S = Smem4<NB, NT, QP, HW>;
    static_assert(HW == 1 || (HW == kWarps && NT == 1), "one head for all warps, or one each with 8 rows");
    constexpr int ROWS = S::kRows, KEYS = S::kTileKeys, W = (NB + 1) / 2;
    constexpr int TILES = HW == 1 ? NT : HW;  // of 8 rows in a partial result
    constexpr bool EXACT = QP == 2, PACKED = !EXACT;
    constexpr float kUnit = EXACT ? 1.0f : 16777216.0f;  // codes stand for so many
    const AttendParams &p = pp.a;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t scan_units[kWarps], scan_items[kWarps];
    __shared__ int64_t start_b, start_item, start_unit;
    __shared__ float row_mul[HW * ROWS];
    __shared__ int ahead[kWarps][2][32];  // pages of the next item's first two steps
    __shared__ int is_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    unsigned char *q_sm = smem + S::kRing;
    unsigned char *bias_sm = q_sm + S::kQ;  // [row][slot][2]: slot part * W + block / 2

    // ---- the CTA's share of the line of units (kv_attend.cuh)
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

    // ---- the warp's ring: a stage takes 32 keys, K codes, V codes, K scales, V scales
    unsigned char *ring = smem + warp * (S::kStage * kStages4);
    // row: of the lane's key, or (SEG) of the first key of the lane's half of the step.  What is not there is not copied:
    // whatever the ring holds in its place is finite as codes, and its scores and weights are replaced (`partial`).
    // 32 pieces of 16 bytes at a time, NB a key: the lane's i-th is piece (lane + 32 i) % NB of key (lane + 32 i) / NB.
    constexpr int kKJump = NB == 8 ? 4 * S::kKPitch : 512;  // from a lane's piece of K to its next, in the ring
    const uint32_t ring_k = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + lane / NB * S::kKPitch + lane % NB * 16;
    const uint32_t ring_v = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + kStepKeys * S::kKPitch +
                            lane / NB * S::kCodes + S::v_piece(lane / NB, lane % NB) * 16;
    const int8_t *const lane_k = p.c.k_codes + lane * 16, *const lane_v = p.c.v_codes + lane * 16;
    auto issue = [&](bool any, int slot, uint32_t row) {
        if (any) {
            const uint32_t at = slot * S::kStage, ss = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + at +
                                                       kStepKeys * (S::kKPitch + S::kCodes);
            const uint32_t sk = ring_k + at, sv = ring_v + at;
            if constexpr (SEG) {
                // 16 keys in a row: 16 NB pieces
                const uint32_t half[2] = {__shfl_sync(~0u, row, 0), __shfl_sync(~0u, row, 16)};
                const int8_t *fk[2], *fv[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    fk[h] = lane_k + static_cast<uint64_t>(half[h]) * S::kCodes;
                    fv[h] = lane_v + static_cast<uint64_t>(half[h]) * S::kCodes;
                }
                auto both = [&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    if constexpr (j < NB) {
                        constexpr bool split = 32 * j < 16 * NB && 32 * j + 32 > 16 * NB;  // NB = 3: half of it each
                        constexpr int h = 32 * j >= 16 * NB ? 1 : 0, from = 512 * j - h * 256 * NB;
                        if constexpr (split) {
                            const bool second = lane >= 16;
                            if (half[second] != kNoRow) {
                                cp_async16_at<j * kKJump, 0>(sk, fk[second] + (second ? 512 * j - 256 * NB : 512 * j));
                                cp_async16_at<j * 512, 0>(sv, fv[second] + (second ? 512 * j - 256 * NB : 512 * j));
                            }
                        } else if (half[h] != kNoRow) {
                            cp_async16_at<j * kKJump, from>(sk, fk[h]);
                            cp_async16_at<j * 512, from>(sv, fv[h]);
                        }
                    }
                };
                both(std::integral_constant<int, 0>());
                both(std::integral_constant<int, 1>());
                both(std::integral_constant<int, 2>());
                both(std::integral_constant<int, 3>());
                both(std::integral_constant<int, 4>());
                both(std::integral_constant<int, 5>());
                both(std::integral_constant<int, 6>());
                both(std::integral_constant<int, 7>());
            } else {
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const int i = lane + 32 * j;
                    const uint32_t r = __shfl_sync(~0u, row, i / NB);
                    if (r != kNoRow) {
                        const uint64_t from = static_cast<uint64_t>(r) * S::kCodes + i % NB * 16;
                        cp_async16(sk + j * kKJump, p.c.k_codes + from);
                        cp_async16(sv + j * 512, p.c.v_codes + from);
                    }
                }
            }
            if (row != kNoRow) {
                const uint32_t dk = ss + lane * S::kScales, dv = dk + kStepKeys * S::kScales;
                const uint64_t from = static_cast<uint64_t>(row) * S::kScales + (SEG ? (lane & 15) * S::kScales : 0);
                const char *ks = reinterpret_cast<const char *>(p.c.k_scales) + from;
                const char *vs = reinterpret_cast<const char *>(p.c.v_scales) + from;
                if constexpr (S::kScales == 16) {
                    cp_async16(dk, ks);
                    cp_async16(dv, vs);
                } else if constexpr (S::kScales == 8) {
                    cp_async8(dk, ks);
                    cp_async8(dv, vs);
                } else {
                    cp_async4(dk, ks);
                    cp_async4(dv, vs);
                }
            }
        }
        cp_commit();
    };

    // What a CTA does of one item: key tiles kt0 .. kt1 - 1, one step of the warp in each.
    struct Work {
        int64_t kt0, kt1;
        int base0, n_steps, keys;
        uint32_t head;  // rows before the head's in a page
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
        k.head = static_cast<uint32_t>(x.h + (HW == 1 ? 0 : warp)) * pp.stride_head;
        k.table = p.table + static_cast<int64_t>(x.b) * p.table_row;
        return k;
    };
    // position of the lane's key of step i (SEG: of its half's first key) and its column of the table; false if there is none
    auto seek = [&](const Work &k, int i, int *pos, uint32_t *col) -> bool {
        *pos = k.base0 + i * KEYS + (SEG ? lane & 16 : lane);
        *col = (__umulhi(*pos, p.page_mul) + *pos) >> p.page_shift;  // pos / page_size
        return i < k.n_steps && *pos < k.keys;
    };
    // its row number, or kNoRow
    auto row_at = [&](const Work &k, int pos, uint32_t col, int page) -> uint32_t {
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.pages)) return kNoRow;
        // (rows are numbered in 32 bits: products may be taken modulo 2^32)
        return static_cast<uint32_t>(page) * pp.stride_page + (pos - col * p.c.page_size) * pp.stride_token + k.head;
    };
    auto find = [&](const Work &k, int i) -> uint32_t {
        int pos;
        uint32_t col;
        return seek(k, i, &pos, &col) ? row_at(k, pos, col, __ldg(k.table + col)) : kNoRow;
    };
    uint32_t row_cur[kStages4];  // rows of the steps in the ring: their lanes' keys are there
    uint32_t row_next;
    int slot0 = 0;  // stage of the item's first step
    auto begin = [&](const Work &k) {
#pragma unroll
        for (int i = 0; i < kStages4 - 1; ++i) {
            row_cur[i] = find(k, i);
            issue(i < k.n_steps, (slot0 + i) % kStages4, row_cur[i]);
        }
        row_next = find(k, kStages4 - 1);
    };
    // The same for an item whose pages are on their way to `ahead` since `look`, so that its first keys wait for no table.
    auto look = [&](const Work &k) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int pos;
            uint32_t col;
            if (seek(k, i, &pos, &col)) cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(&ahead[warp][i][lane])), k.table + col);
        }
    };
    auto begin_ahead = [&](const Work &k) {
        uint32_t row[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int pos;
            uint32_t col;
            row[i] = seek(k, i, &pos, &col) ? row_at(k, pos, col, ahead[warp][i][lane]) : kNoRow;
        }
        row_cur[0] = row[0];
        issue(k.n_steps > 0, slot0, row[0]);
        row_next = row[1];
    };
    // The thread's elements of an item's q: l8 + 8 i of rows tid / 8 and, with four heads, 16 behind it
    constexpr int PASSES = (HW * ROWS + kWarps * 4 - 1) / (kWarps * 4);
    const int q_row = tid >> 3, l8 = tid & 7;
    T q_raw[PASSES][4 * NB];
    auto load_q = [&](const Place &x) {
#pragma unroll
        for (int s = 0; s < PASSES; ++s) {
            const int rr = q_row + s * (kWarps * 4), hw = rr / ROWS, r = rr % ROWS;
            const int idx = x.rt * ROWS + r, node = idx / p.group, hq = (x.h + hw) * p.group + idx - node * p.group;
            const T *src = static_cast<const T *>(p.q) + (static_cast<int64_t>(x.row0) + node) * p.q_row + hq * p.q_head;
            const bool live = rr < HW * ROWS && r < min(ROWS, x.nodes * p.group - x.rt * ROWS);
#pragma unroll
            for (int i = 0; i < 4 * NB; ++i) {
                const int e = l8 + 8 * i;
                q_raw[s][i] = live && e < pp.dim ? src[e] : from_f32<T>(0.0f);
            }
        }
    };
    // Row g of an octet of the operands is place (g & 1) * 4 + g / 2 of eight keys, so that the four keys 2c, 2c + 1 of a
    // lane's values, over c, are neighbours in shared memory.
    const int place = (g & 1) * 4 + (g >> 1);

    Work k = work_of(w);
    begin(k);
    bool first_item = true;  // that has tiles here
    load_q(w);
    for (;;) {
        const int rows = min(ROWS, w.nodes * p.group - w.rt * ROWS);
        if (k.n_steps > 0) {
            // ---- q rows to shared memory: a power of two per row, then f16 parts
#pragma unroll
            for (int pass = 0; pass < PASSES; ++pass) {
                const int rr = q_row + pass * (kWarps * 4);
                if (rr >= HW * ROWS) break;  // whole warps
                float x[4 * NB];
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i) {
                    x[i] = to_f32(q_raw[pass][i]);
                    top = fmaxf(top, fabsf(x[i]));
                }
#pragma unroll
                for (int d = 1; d < 8; d *= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
                const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 13, -100), 100);
                // 2^-ex, and the sign of the scale, so that the rows' factors are positive
                const float down = copysignf(__uint_as_float(static_cast<uint32_t>(127 - ex) << 23), p.scale_log2);
                // element l8 of each word of 8: its nibble is pair l8 % 4, half l8 / 4; odd pairs carry 16
                const float part16 = l8 & 1 ? 0.0625f : 1.0f, times16 = l8 & 1 ? 16.0f : 1.0f;
                float sum[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) sum[b] = 0.0f;
#pragma unroll
                for (int i = 0; i < 4 * NB; ++i) {
                    const float y = x[i] * down * part16;
                    const __half hi = __float2half_rn(y);
                    __half *dst = reinterpret_cast<__half *>(q_sm + rr / ROWS * S::kQHead + rr % ROWS * S::kQPitch) + 8 * i + 2 * (l8 & 3) + (l8 >> 2);
                    *dst = hi;
                    float used = __half2float(hi);
                    if constexpr (QP == 2) {
                        const __half lo = __float2half_rn(y - used);
                        dst[ROWS * S::kQPitch / 2] = lo;
                        used += __half2float(lo);
                    }
                    sum[i / 4] += used * times16;
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int d = 1; d < 8; d *= 2) sum[b] += __shfl_xor_sync(~0u, sum[b], d);
                }
                if constexpr (!EXACT) {
                    if (l8 == 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x0 = i < 2 * W ? -8.0f / 16777216.0f * sum[i % W * 2] : 0.0f;
                            const float x1 = i < 2 * W && i % W * 2 + 1 < NB ? -8.0f / 16777216.0f * sum[i % W * 2 + 1 < NB ? i % W * 2 + 1 : 0] : 0.0f;
                            const uint32_t hi = pack_half2(x0, x1);
                            const float2 back = unpack_half2(hi);
                            reinterpret_cast<uint32_t *>(bias_sm)[rr * 8 + i] = i < W ? hi : pack_half2(x0 - back.x, x1 - back.y);
                        }
                    }
                }
                // not 0: a score of -inf has to stay that
                if (l8 == 0)
                    row_mul[rr] = fmaxf(__uint_as_float(static_cast<uint32_t>(127 + ex) << 23) * kUnit * fabsf(p.scale_log2), 1e-37f);
            }
            __syncthreads();
            const bool more = w.first + w.tiles_k < u_end;
            if (more) {
                Place next = w;
                advance(next);
                look(work_of(next));
            }

            float o[NT][NB * 2][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NB * 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[t][i][j] = 0.0f;
            // of rows 8 t + 2c and 8 t + 2c + 1; m: running maximum (log2) plus E
            // minus: -m, or 0 while there is none
            float m[NT][2], minus[NT][2], l[NT][2], mul[NT][2];
            uint32_t bias[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    m[t][r] = -INFINITY;
                    minus[t][r] = l[t][r] = 0.0f;
                    mul[t][r] = row_mul[(HW == 1 ? 0 : warp * ROWS) + 8 * t + 2 * c + r];
                    if constexpr (!EXACT)
                        bias[t][r] = reinterpret_cast<const uint32_t *>(bias_sm)[((HW == 1 ? 0 : warp * ROWS) + 8 * t + g) * 8 + 4 * r + c];
                }

            const unsigned char *my_q = q_sm + (HW == 1 ? 0 : warp * S::kQHead);
            int slot = slot0;
            for (int i = 0; i < k.n_steps; ++i) {
                // row_cur[0] is step i's; the next free stage takes step i + kStages4 - 1
                row_cur[kStages4 - 1] = row_next;
                issue(i + kStages4 - 1 < k.n_steps, slot == 0 ? kStages4 - 1 : slot - 1, row_next);
                row_next = find(k, i + kStages4);
                cp_wait<kStages4 - 1>();
                __syncwarp();
                const unsigned char *sk = ring + slot * S::kStage, *sv = sk + kStepKeys * S::kKPitch;
                const unsigned char *ks = sv + kStepKeys * S::kCodes, *vs = ks + kStepKeys * S::kScales;
                const int base = k.base0 + i * KEYS;
                const uint32_t there = __ballot_sync(~0u, row_cur[0] != kNoRow && (!SEG || base + lane < k.keys));
                if (there != 0) {
                    // ---- scores: s[t][2 j + k][r] of key 16 j + 8 k + place and row 8 t + 2c + r
                    float s[NT][4][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t d0[W], d1[W];
                        load_scales4<NB>(ks + (16 * j + place) * S::kScales, d0);
                        load_scales4<NB>(ks + (16 * j + 8 + place) * S::kScales, d1);
                        uint32_t x[NB], y[NB];
                        load_key<NB>(sk + (16 * j + place) * S::kKPitch + c * (4 * NB), x);
                        load_key<NB>(sk + (16 * j + 8 + place) * S::kKPitch + c * (4 * NB), y);
                        // the 8s of all blocks: scales times the rows' sums
                        float sum[NT][4];
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r) sum[t][r] = 0.0f;
                        if constexpr (!EXACT) {
                            const unsigned char *k0 = ks + (16 * j + place) * S::kScales, *k1 = k0 + 8 * S::kScales;
                            uint32_t a[4] = {0u, 0u, 0u, 0u};
                            a[0] = *reinterpret_cast<const uint32_t *>(k0 + 4 * (c % W));
                            a[1] = *reinterpret_cast<const uint32_t *>(k1 + 4 * (c % W));
                            if constexpr (W == 4) {
                                a[2] = a[0];
                                a[3] = a[1];
                            } else if constexpr (W == 3) {
                                a[2] = *reinterpret_cast<const uint32_t *>(k0 + 4 * ((c + 4) % W));
                                a[3] = *reinterpret_cast<const uint32_t *>(k1 + 4 * ((c + 4) % W));
                            }
                            if constexpr (NB == 3) {  // there is no fourth scale
                                a[0] &= c & 1 ? 0xFFFFu : ~0u;
                                a[1] &= c & 1 ? 0xFFFFu : ~0u;
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma_f16(sum[t], a, bias[t][0], bias[t][1], sum[t]);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                s[t][2 * j][r] = sum[t][r];
                                s[t][2 * j + 1][r] = sum[t][2 + r];
                            }
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const uint32_t xs = x[b] >> 8, ys = y[b] >> 8;
                            const uint32_t a0[4] = {codes1<EXACT>(x[b]), codes1<EXACT>(y[b]), codes16<EXACT>(x[b]), codes16<EXACT>(y[b])};
                            const uint32_t a1[4] = {codes1<EXACT>(xs), codes1<EXACT>(ys), codes16<EXACT>(xs), codes16<EXACT>(ys)};
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                                for (int q = 0; q < QP; ++q) {
                                    const uint4 qq = *reinterpret_cast<const uint4 *>(
                                        my_q + (q * ROWS + 8 * t + g) * S::kQPitch + b * 64 + c * 16);
                                    mma_f16(part, a0, qq.x, qq.y, part);
                                    mma_f16(part, a1, qq.z, qq.w, part);
                                }
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    s[t][2 * j][r] = fmaf(part[r], scale_of(d0[b / 2], b), s[t][2 * j][r]);
                                    s[t][2 * j + 1][r] = fmaf(part[2 + r], scale_of(d1[b / 2], b), s[t][2 * j + 1][r]);
                                }
                            }
                        }
                    }
                    // ---- which keys each row sees
                    const bool drafts = base + kStepKeys > w.prefix;
                    const bool partial = drafts || there != ~0u;
                    uint32_t see[NT][2];
                    if (partial) {
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                see[t][r] = there;
                                if (drafts)
                                    see[t][r] &= sees(p.mask, p.mask_row, p.mask_words, p.group, w.nodes, w.row0, base - w.prefix,
                                                      w.rt * ROWS + 8 * t + 2 * c + r);
                            }
                    }
                    // ---- the values' scales
                    int f_all = 15, f_key = 1;  // exponent fields: that all keys count with, the lane's key's own
                    uint32_t odd = 0;  // keys with a scale, of K or V, that is not finite (or whatever the ring holds for an absent one)
                    {
                        uint32_t d[W], dk[W], any = 0, any_k = 0;
                        load_scales4<NB>(vs + lane * S::kScales, d);
                        load_scales4<NB>(ks + lane * S::kScales, dk);
                        if constexpr (NB % 2 == 1) {
                            d[W - 1] &= 0xFFFFu;
                            dk[W - 1] &= 0xFFFFu;
                        }
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            any |= d[i];
                            any_k |= dk[i];
                        }
                        // Most steps: every row sees every key, and every key has scales of V below 2 and one of 2^-7 or more (a
                        // bit each of the field).  Of K, 0x7C00 and 0x0400 are 0x8000.
                        const bool plain = (any & 0x40004000u) == 0 && (any & 0x20002000u) != 0 &&
                                           (((any_k & 0x7FFF7FFFu) + 0x04000400u) & 0x80008000u) == 0;
                        if (EXACT || partial || !__all_sync(~0u, plain)) {
                            uint32_t most = 0, most_k = 0;
#pragma unroll
                            for (int i = 0; i < W; ++i) {
                                most = __vmaxu2(most, d[i] & 0x7FFF7FFFu);
                                most_k = __vmaxu2(most_k, dk[i] & 0x7FFF7FFFu);
                            }
                            const uint32_t top_bits = max(most & 0xFFFFu, most >> 16);
                            odd = __ballot_sync(~0u, max(top_bits, max(most_k & 0xFFFFu, most_k >> 16)) >= 0x7C00u);
                            uint32_t counting = ~odd;
                            if (partial) {  // what no row sees does not count
                                uint32_t by_any = 0;
#pragma unroll
                                for (int t = 0; t < NT; ++t) by_any |= see[t][0] | see[t][1];
                                counting &= __reduce_or_sync(~0u, by_any);
                            }
                            const bool counts = (counting >> lane & 1u) != 0;
                            f_key = field_of(top_bits);
                            f_all = __reduce_max_sync(~0u, counts ? f_key : 1);
                            if (PACKED) f_all = counted(f_all);
                            if (odd != 0 || (PACKED && f_all < 15)) {
                                // (rows that see an odd key are NaN; for the others its values' scales are 0, as their weights are)
                                const uint32_t up = static_cast<uint32_t>(15 - (PACKED ? shift_of(f_all) : 0)) * 0x04000400u;
#pragma unroll
                                for (int i = 0; i < W; ++i)
                                    reinterpret_cast<uint32_t *>(const_cast<unsigned char *>(vs) + lane * S::kScales)[i] =
                                        counts ? mul_half2(d[i], up) : 0u;
                                __syncwarp();
                            }
                        }
                    }
                    // ---- softmax
                    bool above = false;
                    float top[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (partial) {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                // whoever sees a scale that is not finite is NaN, however little its key weighs
                                if ((see[t][r] & odd) != 0) l[t][r] = NAN;
                                top[t][r] = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int key = 8 * k + place;
                                    if (((see[t][r] >> key) & 1u) == 0) s[t][k][r] = -INFINITY;
                                    // f32: a row's E comes from keys that it sees, so that no other's scale matters
                                    top[t][r] = fmaxf(top[t][r], fmaf(s[t][k][r], mul[t][r], exponent_of(EXACT ? __shfl_sync(~0u, f_key, key) : f_all)));
                                }
                            }
                        } else {
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                if (odd != 0) l[t][r] = NAN;
                                top[t][r] = fmaf(fmaxf(fmaxf(s[t][0][r], s[t][1][r]), fmaxf(s[t][2][r], s[t][3][r])), mul[t][r], exponent_of(f_all));
                            }
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) above |= top[t][r] > m[t][r] + kSlack;
                    }
                    if (__any_sync(~0u, above)) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float f[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
#pragma unroll
                                for (int d = 4; d < 32; d *= 2) top[t][r] = fmaxf(top[t][r], __shfl_xor_sync(~0u, top[t][r], d));
                                const float n = fmaxf(m[t][r], top[t][r]);
                                minus[t][r] = n == -INFINITY ? 0.0f : -n;
                                f[r] = ex2(m[t][r] + minus[t][r]);
                                m[t][r] = n;
                                l[t][r] *= f[r];
                            }
#pragma unroll
                            for (int k = 0; k < NB * 2; ++k) {
                                o[t][k][0] *= f[0];
                                o[t][k][1] *= f[1];
                                o[t][k][2] *= f[0];
                                o[t][k][3] *= f[1];
                            }
                        }
                    }
                    {
                        // weights, times 2^G if the scales were brought up by as much; their sum without
                        const int g = PACKED ? shift_of(f_all) : 0;
                        const float add = static_cast<float>(g), up = __uint_as_float(static_cast<uint32_t>(127 - g) << 23);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float sum[2] = {0.0f, 0.0f};
                            const float from[2] = {minus[t][0] + add, minus[t][1] + add};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                fma2(s[t][k][0], s[t][k][1], mul[t][0], mul[t][1], from[0], from[1]);
                                s[t][k][0] = ex2(s[t][k][0]);
                                s[t][k][1] = ex2(s[t][k][1]);
                                add2(sum[0], sum[1], s[t][k][0], s[t][k][1]);
                            }
                            fma2(sum[0], sum[1], up, up, l[t][0], l[t][1]);
                            l[t][0] = sum[0];
                            l[t][1] = sum[1];
                        }
                    }
                   // ---- O^T += V^T (P dV)^T, two blocks at a time (a word's halves), 16 keys at a time
                    uint32_t dv[4][W], p2[NT][PP][4];
                    if constexpr (PACKED) {
                        // (the scales of the lane's keys of the second operand are read where they are paired)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t h = pack_half2(s[t][k][0], s[t][k][1]);
                                p2[t][0][k] = transpose8(h);
                                if constexpr (PP == 2) {
                                    const float2 back = unpack_half2(h);
                                    p2[t][PP - 1][k] = transpose8(pack_half2(s[t][k][0] - back.x, s[t][k][1] - back.y));
                                }
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) load_scales4<NB>(vs + (8 * k + place) * S::kScales, dv[k]);
                    }
                    // the lane's keys 16 j + {2c, 2c + 1, 8 + 2c, 8 + 2c + 1}: places c, 4 + c, 8 + c, 12 + c
                    uint32_t v[2][4][W];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const int r = 16 * j + 4 * n + c;
                            load_value<NB>(sv + r * S::kCodes + S::v_piece(r, g * NB / 8) * 16 + g * (2 * NB) % 16, v[j][n]);
                        }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t wgt[2][NT][PP][2];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if constexpr (PACKED) {
                                // scales of keys 8 k + c and 8 k + 4 + c
                                const unsigned char *at = vs + (8 * k + c) * S::kScales + b / 2 * 4;
                                const uint32_t d = __byte_perm(*reinterpret_cast<const uint32_t *>(at),
                                                               *reinterpret_cast<const uint32_t *>(at + 4 * S::kScales),
                                                               b & 1 ? 0x7632u : 0x5410u);
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
                                    const uint32_t h = mul_half2(p2[t][0][k], d);
                                    wgt[k >> 1][t][0][k & 1] = h;
                                    // what that rounded off, and the lower part's product
                                    if constexpr (PP == 2)
                                        wgt[k >> 1][t][PP - 1][k & 1] = fma_half2(p2[t][PP - 1][k], d, fma_half2(p2[t][0][k], d, h ^ 0x80008000u));
                                }
                                continue;
                            }
                            const float d = PACKED ? 0.0f : scale_of(dv[k][b / 2], b);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const float(&pr)[2] = s[t][k];
                                const float x0 = pr[0] * d, x1 = pr[1] * d;
                                const uint32_t h = pack_half2(x0, x1);
                                wgt[k >> 1][t][0][k & 1] = transpose8(h);
                                if constexpr (PP == 2) {
                                    const float2 back = unpack_half2(h);
                                    wgt[k >> 1][t][PP - 1][k & 1] = transpose8(pack_half2(x0 - back.x, x1 - back.y));
                                }
                            }
                        }
                        // -8 2^-24 and -128 2^-24 times the weights, then the codes
                        float acc[NT][2][4];
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint32_t eight[4] = {0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u};
                            float off[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int j = 0; j < (EXACT ? 0 : 2); ++j)
#pragma unroll
                                for (int q = 0; q < PP; ++q) mma_f16(off, eight, wgt[j][t][q][0], wgt[j][t][q][1], off);
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[t][0][k] = acc[t][1][k] = off[k];
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t sel = b & 1 ? 0x7632u : 0x5410u;
                            const uint32_t x = __byte_perm(v[j][0][b / 2], v[j][1][b / 2], sel);
                            const uint32_t y = __byte_perm(v[j][2][b / 2], v[j][3][b / 2], sel);
                            const uint32_t xs = x >> 8, ys = y >> 8;
                            const uint32_t a0[4] = {codes1<EXACT>(x), codes16<EXACT>(x), codes1<EXACT>(y), codes16<EXACT>(y)};
                            const uint32_t a1[4] = {codes1<EXACT>(xs), codes16<EXACT>(xs), codes1<EXACT>(ys), codes16<EXACT>(ys)};
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int q = 0; q < PP; ++q) {
                                    mma_f16(acc[t][0], a0, wgt[j][t][q][0], wgt[j][t][q][1], acc[t][0]);
                                    mma_f16(acc[t][1], a1, wgt[j][t][q][0], wgt[j][t][q][1], acc[t][1]);
                                }
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int k = 0; k < 4; k += 2)
                                    add2(o[t][2 * b + e][k], o[t][2 * b + e][k + 1], acc[t][e][k], acc[t][e][k + 1]);
                    }
                }
                __syncwarp();
                slot = slot + 1 == kStages4 ? 0 : slot + 1;
#pragma unroll
                for (int j = 0; j + 1 < kStages4; ++j) row_cur[j] = row_cur[j + 1];
            }
            slot0 = slot;
            // ---- the next item's first keys and q are on their way while the warps of this one are joined
            const Place done = w;
            const Work did = k;
            if (more) {
                advance(w);
                k = work_of(w);
                cp_wait<0>();
                begin_ahead(k);
                load_q(w);
            }
            const bool whole = did.kt0 == 0 && did.kt1 == done.tiles_k;
            const int pitch = pp.dim + kPartExtra;
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
            // elements 4 g + {0 .. 3} of each block, in the codes' units, 16 in the odd ones
            constexpr float one = kUnit, sixteen = kUnit / 16.0f;
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
                            const float4 x = make_float4(o[0][2 * b][r] * one, o[0][2 * b][2 + r] * sixteen, o[0][2 * b + 1][r] * one,
                                                         o[0][2 * b + 1][2 + r] * sixteen);
                            if (e < pp.dim) {
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
                                part[pp.dim] = m[0][r];
                                part[pp.dim + 1] = sum;
                            } else if (p.lse) {
                                p.lse[row * p.heads_q + hq] = (-minus[0][r] + log2f(sum)) * 0.693147180559945f;
                            }
                        }
                    }
                }
            } else {
            // row r8 of warp q: [kJoinPitch], its maximum and sum behind its elements
            auto joined = [&](int q, int r8) {
                return reinterpret_cast<float *>(smem + q * (S::kStage * kStages4) + (slot0 ^ 1) * S::kStage) + r8 * S::kJoinPitch;
            };
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t > 0) __syncthreads();
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float *at = joined(warp, 2 * c + r);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        *reinterpret_cast<float4 *>(at + 32 * b + 4 * g) =
                            make_float4(o[t][2 * b][r] * one, o[t][2 * b][2 + r] * sixteen, o[t][2 * b + 1][r] * one,
                                        o[t][2 * b + 1][2 + r] * sixteen);
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) l[t][r] += __shfl_xor_sync(~0u, l[t][r], d);
                    if (g == 0) {
                        at[32 * NB] = m[t][r];
                        at[32 * NB + 1] = l[t][r];
                    }
                }
                __syncthreads();
                // kWarps * 4 threads a row
                constexpr int TPR = kWarps * 4;
                const int r8 = tid / TPR, lr = tid % TPR;
                float f[kWarps], top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) top = fmaxf(top, joined(q, r8)[32 * NB]);
                const float z = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) {
                    const float *x = joined(q, r8);
                    f[q] = ex2(x[32 * NB] - z);
                    sum = fmaf(f[q], x[32 * NB + 1], sum);
                }
                int64_t row;
                int hq;
                if (place_row(t, r8, &row, &hq)) {
                    T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
                    float *part = p.partial + (slot_p * (8 * TILES) + 8 * t + r8) * pitch;
                    const float inv = sum > 0.0f ? __frcp_rn(sum) : sum == 0.0f ? 0.0f : sum;  // NaN stays
#pragma unroll
                    for (int q = 0; q < 32 * NB / TPR; ++q) {
                        const int e = lr + TPR * q;
                        if (e < pp.dim) {
                            float x = 0.0f;
#pragma unroll
                            for (int v = 0; v < kWarps; ++v) x = fmaf(f[v], joined(v, r8)[e], x);
                            if (whole)
                                out[e] = from_f32<T>(x * inv);
                            else
                                part[e] = x;
                        }
                    }
                    if (lr == 0) {
                        if (!whole) {
                            part[pp.dim] = top;
                            part[pp.dim + 1] = sum;
                        } else if (p.lse) {
                            p.lse[row * p.heads_q + hq] = (z + log2f(sum)) * 0.693147180559945f;
                        }
                    }
                }
            }
            }
            // (an item past the tickets exists only if `starts` is not ascending: it has no output)
            if (!whole && done.item < p.tickets_n) {
                constexpr int PR = 8 * TILES, TPR = kWarps * 32 / PR, V = (8 * NB + TPR - 1) / TPR;  // rows, threads a row, float4 a thread
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
                        for (int i = 0; i < n; ++i) top = fmaxf(top, __ldcg((i == 0 ? from0 : from + i * step) + pp.dim));
                        const float z = top == -INFINITY ? 0.0f : top;
#pragma unroll (V <= 2 ? 8 : 4)
                        for (int i = 0; i < n; ++i) {
                            const float *part = i == 0 ? from0 : from + i * step;
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part + pp.dim));
                            const float f = ex2(ml.x - z);
                            sum = fmaf(f, ml.y, sum);
#pragma unroll
                            for (int q = 0; q < V; ++q) {
                                const int e0 = 4 * (lr + TPR * q);
                                if (e0 < pp.dim) {
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
                                if (4 * (lr + TPR * q) < pp.dim) out[4 * (lr + TPR * q) + e] = from_f32<T>(x[q][e] * inv);
                        if (lr == 0 && p.lse)
                            p.lse[row * p.heads_q + hq] = ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * 0.693147180559945f;
                    } else if (live) {
                        float *to = p.partial + (head * PR + pr) * pitch;
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            if (4 * (lr + TPR * q) < pp.dim)
                                *reinterpret_cast<float4 *>(to + 4 * (lr + TPR * q)) = make_float4(x[q][0], x[q][1], x[q][2], x[q][3]);
                        if (lr == 0) {
                            to[pp.dim] = top;
                            to[pp.dim + 1] = sum;
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
                // Parts c0 .. c1, up to kJoinGroup at once, more in two levels (kv_attend.cuh)
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
            load_q(w);
        }
        __syncthreads();  // the join's reads, before the next item's q
    }
}

template <typename T, int NB, int NT, int QP, int PP, int HW>
Attend4Variant attend4_variant_of(bool rows_in_turn) {
    constexpr int smem = Smem4<NB, NT, QP, HW>::kTotal, rows = 8 * (HW == 1 ? NT : HW);
    if constexpr (HW == 1)
        if (rows_in_turn) return {q4kv_attend_kernel<T, NB, NT, QP, PP, true, HW>, smem, rows};
    return {q4kv_attend_kernel<T, NB, NT, QP, PP, false, HW>, smem, rows};
}

template <typename T, int NB, int QP, int PP>
Attend4Variant attend4_variant_of(Attend4Shape shape) {
    switch (shape) {
        case k4Rows8: return attend4_variant_of<T, NB, 1, QP, PP, 1>(false);
        case k4Rows8InTurn: return attend4_variant_of<T, NB, 1, QP, PP, 1>(true);
        case k4Heads4: return attend4_variant_of<T, NB, 1, QP, PP, kWarps>(false);
        default: break;
    }
    if constexpr (NB <= 4) return attend4_variant_of<T, NB, 2, QP, PP, 1>(shape == k4Rows16InTurn);
    return {};
}

template <typename T, int QP, int PP>
Attend4Variant attend4_variant_of(int blocks, Attend4Shape shape) {
    switch (blocks) {
        case 2: return attend4_variant_of<T, 2, QP, PP>(shape);
        case 3: return attend4_variant_of<T, 3, QP, PP>(shape);
        case 4: return attend4_variant_of<T, 4, QP, PP>(shape);
        case 6: return attend4_variant_of<T, 6, QP, PP>(shape);
        case 8: return attend4_variant_of<T, 8, QP, PP>(shape);
        default: return {};
    }
}

}  // namespace kv
