// Storing keys and values in the Q4_0 cache, and rotating q and k with it: one
// kernel for q4kv_cache_write, kvrope_apply and kvrope_write_q8 / _q4
// (../../include/q4kv.h, kvrope.h).
//
// As q8kv_write_kernel (kv_cache.cu): a lane takes 16 bytes of the wide side, a
// 32-element block is 4 or 8 neighbouring lanes, keys and values of the same place
// are the same lane's, and a block's maximum takes 2 or 3 shuffles.  HBM bounds a
// prompt, next to the issue slots; one round trip a few rows.
//   * 4 bits.  The largest of x and of -x, the signed extreme is the greater one;
//     16-bit types are compared in pairs.  x / d + 8 is left, rounded to even, in the
//     low bits of its sum with 1.5 * 2^23 + 8; eight codes are put together by
//     multiply-adds of those words, whose exponents' sum is a constant to take off.
//   * Rotation.  The cosines and sines of a block's tokens are worked out once, by all
//     its threads, into shared memory, for all heads.  p * turns modulo 2^64 is the
//     angle to the last bit at any position.  Its top 8 bits pick one of 256 points of
//     the circle, kept as two f32 each; the rest, below pi / 256, is a two-term f32 number,
//     and sin r = r - r^3/6 + r^5/120, cos r = 1 - r^2/2 + r^4/24 have small terms for which
//     f32 is enough; the great ones keep what their roundings lose.  That adds up to 2^-42, so
//     that the rounding to f32 is as good as always that of the exact value, and rotated keys
//     get the codes that a program in 64 bits gives them (2^-35, a last bit off in one value of
//     some thousands, took 41.3 us where this takes 43.2).
//     For q a lane takes both halves of its pairs, so that q may be rotated in place;
//     k's other half is read by the lane that needs it (it is in L1).
//
// Measured on GB300 (copy rate 6792 GB/s): 8190 tokens of 32 heads of 128, bf16, to Q4_0
// 38.9 us, 4.4 TB/s, issue (0.7 of the cycles).  8192 tokens, 8 heads to Q8_0 with 32 of q
// rotated, 43.2 us, 4.3 TB/s, the latency of angles and loads (0.5 of the cycles issue); to
// Q4_0 44.0 us; q alone 25.4 us, 5.3 TB/s.
#pragma once

#include "kv4.h"
#include "kv_common.cuh"

namespace kv {

struct StoreParams {
    Cache c;            // BITS = 4: Cache4::rows
    int dim, blocks;    // elements of a head, stored blocks of a row
    const void *in[2];  // k, v; strides in elements
    int64_t row[2], head[2];
    const int64_t *slots;
    int64_t n;
    int lanes;  // of one token's k and v: heads * blocks * (32 / E)
    int kv_y;   // blocks along y that store; those behind rotate q
    // rotation
    const void *q;
    void *out;
    int64_t q_row, q_head, out_row, out_head;
    int q_lanes, q_items;  // of one token, and of one of its heads
    const int64_t *positions;
    const uint64_t *turns;
    const float4 *circle;  // cos and sin of k / 256 of a turn, then what they lack
    float factor;
    int half;  // pairs of a head
    int interleaved, back;
};

namespace store {

template <typename T>
union Piece {
    uint4 v;
    T t[16 / sizeof(T)];
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// cos and sin of t / 2^64 turns, rounded to f32 once
__device__ __forceinline__ void turn(uint64_t t, const float4 *circle, float *c, float *s) {
    const uint32_t k = static_cast<uint32_t>((t + (1ull << 55)) >> 56);  // the nearest point
    const int64_t r = static_cast<int64_t>(t - (static_cast<uint64_t>(k) << 56));  // within +-2^55
    const float4 z = __ldg(circle + (k & 255u));
    const int hi = static_cast<int>(r >> 25);  // within +-2^30
    const float h = __int2float_rn(hi);
    // what h lacks, in units of 2^25
    const float l = __fadd_rn(__int2float_rn(hi - static_cast<int>(h)),
                              __fmul_rn(__uint2float_rn(static_cast<uint32_t>(r) & 0x1FFFFFFu), 0x1p-25f));
    // 2 pi / 2^39 in two parts
    constexpr float k1 = 0x1.921fb6p-37f, k2 = -0x1.777a5cp-62f;
    const float x = __fmul_rn(h, k1);
    const float low = __fadd_rn(__fmaf_rn(h, k1, -x), __fmaf_rn(l, k1, __fmul_rn(h, k2)));  // the angle is x + low
    // cos = 1 + n + g, sin = x + sl: n exact, the others below 4e-7
    const float x2 = __fmul_rn(x, x), n = -0.5f * x2;
    const float g = __fmaf_rn(__fmul_rn(x2, x2), 1.0f / 24.0f, -0.5f * __fmaf_rn(2.0f * x, low, __fmaf_rn(x, x, -x2)));
    const float sl = __fmaf_rn(__fmul_rn(x2, x), __fmaf_rn(x2, 1.0f / 120.0f, -1.0f / 6.0f), low);
    // C cos - S sin = C - S x + C n + ..., S cos + C sin = S + C x + S n + ...: the great terms with what their roundings
    // lose, in falling order (or the first is 0 and the third with it), so that a sum less its first term is exact
    const float C = z.x, S = z.y;
    const float p = __fmul_rn(S, x), q = __fmul_rn(C, x), u = __fmul_rn(C, n), v = __fmul_rn(S, n);
    const float a = __fsub_rn(C, p), b = __fadd_rn(S, q);
    const float c1 = __fadd_rn(a, u), s1 = __fadd_rn(b, v);
    const float ce = __fadd_rn(__fsub_rn(__fsub_rn(C, a), p), __fsub_rn(u, __fsub_rn(c1, a)));
    const float se = __fadd_rn(__fadd_rn(__fsub_rn(S, b), q), __fsub_rn(v, __fsub_rn(s1, b)));
    const float pe = __fsub_rn(__fmaf_rn(C, n, -u), __fmaf_rn(S, x, -p)), qe = __fadd_rn(__fmaf_rn(S, n, -v), __fmaf_rn(C, x, -q));
    const float cr = __fmaf_rn(C, g, __fmaf_rn(-S, sl, __fmaf_rn(z.z, n, __fmaf_rn(-z.w, x, z.z))));
    const float sr = __fmaf_rn(S, g, __fmaf_rn(C, sl, __fmaf_rn(z.w, n, __fmaf_rn(z.z, x, z.w))));
    *c = __fadd_rn(c1, __fadd_rn(__fadd_rn(ce, pe), cr));
    *s = __fadd_rn(s1, __fadd_rn(__fadd_rn(se, qe), sr));
}

// The largest x and the largest -x (and 0) of a lane's elements, NaN if one is.
template <int E>
__device__ __forceinline__ float2 extremes(const float (&y)[E]) {
    float2 m = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < E; ++j) {
        m.x = max_nan(m.x, y[j]);
        m.y = max_nan(m.y, -y[j]);
    }
    return m;
}
__device__ __forceinline__ __half2 pair2(__half a, __half b) { return __halves2half2(a, b); }
__device__ __forceinline__ __nv_bfloat162 pair2(__nv_bfloat16 a, __nv_bfloat16 b) { return __halves2bfloat162(a, b); }
template <typename T2>
__device__ __forceinline__ T2 extremes_of_pairs(const uint4 &v) {
    const T2 *p = reinterpret_cast<const T2 *>(&v);
    const T2 a = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
    const T2 b = __hneg2(__hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3])));
    return __hmax2_nan(pair2(a.x, b.x), pair2(a.y, b.y));
}
// The largest |x|, twice.
template <int E>
__device__ __forceinline__ float2 magnitude(const float (&y)[E]) {
    float m = fabsf(y[0]);
#pragma unroll
    for (int j = 1; j < E; ++j) m = max_nan(m, fabsf(y[j]));
    return make_float2(m, m);
}
// over the PER lanes of a block; ONE: both numbers are the same
template <int PER, bool ONE>
__device__ __forceinline__ float2 over_block(float2 m) {
#pragma unroll
    for (int d = 1; d < PER; d *= 2) {
        m.x = max_nan(m.x, __shfl_xor_sync(~0u, m.x, d));
        if (!ONE) m.y = max_nan(m.y, __shfl_xor_sync(~0u, m.y, d));
    }
    if (ONE) m.y = m.x;
    return m;
}

constexpr float kRound = 12582912.0f;  // 1.5 * 2^23

// E codes of 4 bits.  `low`: x / d may be below -8.5 (d is subnormal).  Codes j and j + E / 2 are cut off at 15 together,
// as halves of a word.
template <int E>
__device__ __forceinline__ uint32_t pack_4(const float (&y)[E], float inv, bool low) {
    uint32_t w = 0;
#pragma unroll
    for (int j = E / 2 - 1; j >= 0; --j) {
        float z[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (not as f32x2: its product and sum come out fused)
            z[i] = __fadd_rn(__fmul_rn(y[j + i * (E / 2)], inv), kRound + 8.0f);
            if (low) z[i] = fmaxf(z[i], kRound);
        }
        w = w * 16u + __vminu2(__byte_perm(__float_as_uint(z[0]), __float_as_uint(z[1]), 0x5410u), 0x000F000Fu);
    }
    if constexpr (E == 4) w = (w & 0xFFu) | (w >> 8);
    return w;
}

// Four codes of 8 bits, for any block: NaN becomes 0 (as kv_cache.cu)
__device__ __forceinline__ uint32_t pack_8(const float *y, float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = max(-127, min(127, __float2int_rn(__fmul_rn(y[i], inv))));
        w |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * i);
    }
    return w;
}
__device__ __forceinline__ uint32_t pack_8_usual(const float *y, float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__fadd_rn(__fmul_rn(y[i], inv), kRound));
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040u), __byte_perm(c[2], c[3], 0x0040u), 0x5410u);
}

template <typename T, bool VEC>
__device__ __forceinline__ uint4 load(const T *p) {
    Piece<T> x;
    if constexpr (VEC) {
        x.v = *reinterpret_cast<const uint4 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) x.t[i] = p[i];
    }
    return x.v;
}

// Element e of a head: its pair, and whether its sine counts negative (the first of the pair).
__device__ __forceinline__ int pair_of(const StoreParams &p, int e, int *other, bool *first) {
    if (p.interleaved) {
        *other = e ^ 1;
        *first = (e & 1) == 0;
        return e >> 1;
    }
    *first = e < p.half;
    *other = *first ? e + p.half : e - p.half;
    return *first ? e : e - p.half;
}

template <typename T>
__device__ __forceinline__ void rotate_pair(T &a, T &b, float c, float s) {
    const float x = to_f32(a), y = to_f32(b);
    a = from_f32<T>(__fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)));
    b = from_f32<T>(__fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)));
}

}  // namespace store

// N angles' cosines or sines, at 4 N bytes' alignment (16 at most)
template <int N>
__device__ __forceinline__ void load_angles(const float *p, float (&c)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + j);
            c[j] = x.x;
            c[j + 1] = x.y;
            c[j + 2] = x.z;
            c[j + 3] = x.w;
        }
    } else {
        static_assert(N == 2, "pairs of 2, 4 or 8");
        const float2 x = *reinterpret_cast<const float2 *>(p);
        c[0] = x.x;
        c[1] = x.y;
    }
}

// One lane's item of one head of q (VEC): a piece, or two that hold each other's pairs (b is of the second, or unused).
struct Item {
    int a, b;       // their first elements; b < 0: there is none
    int first;      // the first pair, below 0: they stay as they are
};
template <int E>
__device__ __forceinline__ Item item_of(const StoreParams &p, int item) {
    if (p.interleaved) return {item * E, -1, item * E < 2 * p.half ? item * E / 2 : -1};
    if (item * E < p.half) return {item * E, item * E + p.half, item * E};
    return {item * E + p.half, -1, -1};
}
template <typename T, int E = 16 / sizeof(T)>
__device__ __forceinline__ void rotate_item(const StoreParams &p, const Item &it, const uint4 &va, const uint4 &vb, T *dst,
                                            const float *cs, const float *sn) {
    using namespace store;
    Piece<T> x, y;
    x.v = va;
    y.v = vb;
    if (it.b >= 0) {
        float c[E], s[E];
        load_angles<E>(cs + it.first, c);
        load_angles<E>(sn + it.first, s);
#pragma unroll
        for (int j = 0; j < E; ++j) rotate_pair(x.t[j], y.t[j], c[j], s[j]);
        *reinterpret_cast<uint4 *>(dst + it.b) = y.v;
    } else if (it.first >= 0) {
        float c[E / 2], s[E / 2];
        load_angles<E / 2>(cs + it.first, c);
        load_angles<E / 2>(sn + it.first, s);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) rotate_pair(x.t[2 * j], x.t[2 * j + 1], c[j], s[j]);
    }
    *reinterpret_cast<uint4 *>(dst + it.a) = x.v;
}
// any alignment: an item is a pair, or an element that stays
template <typename T>
__device__ __forceinline__ void rotate_item(const StoreParams &p, const T *src, T *dst, int item, const float *cs, const float *sn) {
    using namespace store;
    if (item < p.half) {
        const int a = p.interleaved ? 2 * item : item, b = p.interleaved ? a + 1 : a + p.half;
        T x = src[a], y = src[b];
        rotate_pair(x, y, cs[item], sn[item]);
        dst[a] = x;
        dst[b] = y;
    } else {
        dst[item + p.half] = src[item + p.half];
    }
}

// The angles of a block's tokens, by all its threads
__device__ __forceinline__ void turn_all(const StoreParams &p, float *angles, int tokens, int64_t first, int tid) {
    const int pairs = static_cast<int>(min(static_cast<int64_t>(tokens), p.n - first)) * p.half;
    for (int i = tid; i < pairs; i += blockDim.x * blockDim.y) {
        const int t = i / p.half, k = i - t * p.half;
        float c, s;
        store::turn(static_cast<uint64_t>(__ldg(p.positions + first + t)) * __ldg(p.turns + k), p.circle, &c, &s);
        angles[i] = __fmul_rn(c, p.factor);
        s = __fmul_rn(s, p.factor);
        angles[tokens * p.half + i] = p.back ? -s : s;
    }
}

// Lane `at` of q's, U tokens: loads, then the angles, then the rest.
template <typename T, bool VEC, int U>
__device__ __forceinline__ void rotate_q(const StoreParams &p, float *angles, int at, int64_t first, int tid) {
    constexpr int E = 16 / sizeof(T);
    const int tokens = blockDim.y * U;
    const int h = at / max(p.q_items, 1), item = at - h * p.q_items;
    const T *src = static_cast<const T *>(p.q) + (first + threadIdx.y) * p.q_row + h * p.q_head;
    T *dst = static_cast<T *>(p.out) + (first + threadIdx.y) * p.out_row + h * p.out_head;
    const int64_t step = blockDim.y * p.q_row, step_out = blockDim.y * p.out_row;
    // tokens of this lane
    const int64_t left = p.n - first - threadIdx.y;
    const int mine = at >= p.q_lanes || left <= 0 ? 0 : left > (U - 1) * static_cast<int64_t>(blockDim.y) ? U
                                                        : static_cast<int>((left + blockDim.y - 1) / blockDim.y);
    if constexpr (VEC) {
        const Item it = item_of<E>(p, item);
        uint4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            a[u] = u < mine ? store::load<T, true>(src + u * step + it.a) : make_uint4(0, 0, 0, 0);
            b[u] = u < mine && it.b >= 0 ? store::load<T, true>(src + u * step + it.b) : make_uint4(0, 0, 0, 0);
        }
        turn_all(p, angles, tokens, first, tid);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = u * blockDim.y + threadIdx.y;
            if (u < mine) rotate_item<T>(p, it, a[u], b[u], dst + u * step_out, angles + t * p.half, angles + (tokens + t) * p.half);
        }
    } else {
        turn_all(p, angles, tokens, first, tid);
        __syncthreads();
        for (int u = 0; u < mine; ++u) {
            const int t = u * blockDim.y + threadIdx.y;
            rotate_item<T>(p, src + u * step, dst + u * step_out, item, angles + t * p.half, angles + (tokens + t) * p.half);
        }
    }
}

// q alone: of the registers that keys and values take, it has none.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(256) kv_rotate_kernel(const StoreParams p) {
    extern __shared__ __align__(16) float angles[];  // cos, then sin, [token of the block][pair]
    rotate_q<T, VEC, U>(p, angles, blockIdx.y * blockDim.x + threadIdx.x, static_cast<int64_t>(blockIdx.x) * (blockDim.y * U),
                        threadIdx.y * blockDim.x + threadIdx.x);
}

// U tokens a lane.  Six blocks an SM with one (40 registers, a few bytes spilled): 8192 tokens rotated and written to Q8_0
// 43.2 us; five 43.9, four 49.7, eight 52.7 (to Q4_0 44.0, 43.5, 49.4, 51.7).
template <typename T, int BITS, bool ROT, bool VEC, int U>
__global__ void __launch_bounds__(256, U == 1 ? 6 : 1) kv_store_kernel(const StoreParams p) {
    using namespace store;
    constexpr int E = 16 / sizeof(T), PER = 32 / E;  // elements a lane, lanes a block
    extern __shared__ __align__(16) float angles[];  // ROT: cos, then sin, [token of the block][pair]
    // of each token's row of head 0: its first byte of codes (-1: there is no row) and of scales
    __shared__ int64_t code_at[8 * U], scale_at[8 * U];
    const int tokens = blockDim.y * U, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
    const bool stores = static_cast<int>(blockIdx.y) < p.kv_y;
    const int at = (stores ? blockIdx.y : blockIdx.y - p.kv_y) * blockDim.x + threadIdx.x;

    if constexpr (ROT) {
        if (!stores) {
            rotate_q<T, VEC, U>(p, angles, at, first, tid);
            return;
        }
    }
    // ---- keys and values
    const int per_head = p.blocks * PER;
    const int h = at / per_head, in_row = at - h * per_head, e0 = in_row * E, b = in_row / PER;
    const bool live = at < p.lanes && e0 < p.dim;
    // a whole piece of the other halves of k's pairs (VEC, not interleaved)
    const bool turns_piece = ROT && e0 < 2 * p.half;
    const bool apart = ROT && VEC && turns_piece && !p.interleaved;
    const int other0 = e0 < p.half ? e0 + p.half : e0 - p.half;
    Piece<T> raw[U][2], oth[ROT && VEC ? U : 1];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const T *src = static_cast<const T *>(p.in[s]) + (first + threadIdx.y) * p.row[s] + h * p.head[s];
        const int64_t step = static_cast<int64_t>(blockDim.y) * p.row[s];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool there = live && first + threadIdx.y + u * blockDim.y < p.n;
            raw[u][s].v = there ? load<T, VEC>(src + e0 + u * step) : make_uint4(0, 0, 0, 0);
            if constexpr (ROT && VEC)
                if (s == 0) oth[u].v = there && apart ? load<T, true>(src + other0 + u * step) : make_uint4(0, 0, 0, 0);
        }
    }
    if (tid < tokens) {  // row of head 0 of each token, -1 if there is none
        int64_t r = -1;
        const int64_t slot = first + tid < p.n ? __ldg(p.slots + first + tid) : -1;
        if (slot >= 0 && slot < p.c.slots) {
            int64_t page;
            int place;
            if ((slot >> 32) == 0) {
                const uint32_t s32 = static_cast<uint32_t>(slot), pg = s32 / static_cast<uint32_t>(p.c.page_size);
                page = pg;
                place = static_cast<int>(s32 - pg * static_cast<uint32_t>(p.c.page_size));
            } else {
                page = slot / p.c.page_size;
                place = static_cast<int>(slot - page * p.c.page_size);
            }
            r = row_of(p.c, page, 0, place);
        }
        code_at[tid] = r < 0 ? -1 : r * p.c.dim;
        scale_at[tid] = r * (4 * p.c.blocks);
    }
    // the lane's places in its head's row: codes of k and v, the scale that it writes
    const int nb = p.blocks, lane = threadIdx.x & 31, of = lane & (PER - 1), first_lane = lane - of;  // (blockDim.x: whole warps)
    const int64_t head_row = h * p.c.stride_head;
    const int k_place = BITS == 8 ? e0 : E == 8 ? 4 * (of * nb + b) : 4 * ((of >> 1) * nb + b) + 2 * (of & 1);
    const int v_place = BITS == 8 ? e0 : E == 8 ? 2 * (2 * of * nb + b) : 2 * (of * nb + b);
    unsigned char *const k_lane = reinterpret_cast<unsigned char *>(p.c.k_codes) + head_row * p.c.dim + k_place;
    unsigned char *const v_lane = reinterpret_cast<unsigned char *>(p.c.v_codes) + head_row * p.c.dim + v_place;
    // 4 bits: k's is the block's first lane's, v's its second's; 8 bits: the second's and the fourth's
    const bool values_scale = BITS == 4 ? of & 1 : of & 2;
    unsigned char *const s_lane = reinterpret_cast<unsigned char *>(values_scale ? p.c.v_scales : p.c.k_scales) +
                                  head_row * (4 * p.c.blocks) + b * (BITS == 4 ? 2 : 4);
    if constexpr (ROT) turn_all(p, angles, tokens, first, tid);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int t = u * blockDim.y + threadIdx.y;
        const int64_t codes = code_at[t];
        float y[2][E];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < E; ++j) y[s][j] = to_f32(raw[u][s].t[j]);
        if constexpr (ROT) {
            if (live && turns_piece && first + t < p.n) {
                const float *cs = angles + t * p.half, *sn = angles + (tokens + t) * p.half;
                if (VEC && !p.interleaved) {
                    const int i0 = e0 < p.half ? e0 : e0 - p.half;
                    const uint32_t sign = e0 < p.half ? 0x80000000u : 0u;
                    float c[E], s[E];
                    load_angles<E>(cs + i0, c);
                    load_angles<E>(sn + i0, s);
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        y[0][j] = __fadd_rn(__fmul_rn(y[0][j], c[j]),
                                            __fmul_rn(to_f32(oth[VEC ? u : 0].t[j]), __uint_as_float(__float_as_uint(s[j]) ^ sign)));
                } else if (VEC) {
                    float c[E / 2], s[E / 2];
                    load_angles<E / 2>(cs + e0 / 2, c);
                    load_angles<E / 2>(sn + e0 / 2, s);
#pragma unroll
                    for (int j = 0; j < E; j += 2) {
                        const float a = y[0][j], z = y[0][j + 1];
                        y[0][j] = __fsub_rn(__fmul_rn(a, c[j / 2]), __fmul_rn(z, s[j / 2]));
                        y[0][j + 1] = __fadd_rn(__fmul_rn(z, c[j / 2]), __fmul_rn(a, s[j / 2]));
                    }
                } else {
                    const T *src = static_cast<const T *>(p.in[0]) + (first + t) * p.row[0] + h * p.head[0];
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        if (e0 + j < 2 * p.half) {
                            int other;
                            bool low;
                            const int i = pair_of(p, e0 + j, &other, &low);
                            const float s = low ? -sn[i] : sn[i];
                            y[0][j] = __fadd_rn(__fmul_rn(y[0][j], cs[i]), __fmul_rn(to_f32(src[other]), s));
                        }
                }
            }
        }
        float2 m[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (sizeof(T) == 2 && !(ROT && s == 0)) {  // (as they came)
                if constexpr (sizeof(T) == 2) {
                    using T2 = decltype(pair2(raw[0][0].t[0], raw[0][0].t[0]));
                    T2 x = extremes_of_pairs<T2>(raw[u][s].v);
#pragma unroll
                    for (int d = 1; d < PER; d *= 2) x = __hmax2_nan(x, __shfl_xor_sync(~0u, x, d));
                    m[s] = make_float2(to_f32(x.x), to_f32(x.y));
                }
            } else {
                m[s] = BITS == 8 ? over_block<PER, true>(magnitude(y[s])) : over_block<PER, false>(extremes(y[s]));
            }
        }
        const bool nan = m[0].x != m[0].x || m[1].x != m[1].x || m[0].y != m[0].y || m[1].y != m[1].y;
        if (__any_sync(~0u, nan)) {  // of those that are numbers
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                m[s] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    m[s].x = fmaxf(m[s].x, y[s][j]);
                    m[s].y = fmaxf(m[s].y, -y[s][j]);
                }
                m[s] = over_block<PER, false>(m[s]);
            }
        }
        if constexpr (BITS == 4) {
            // the block's two divisions: k's in its first lane, v's in its second
            const float2 mine = of & 1 ? m[1] : m[0];
            const float top = mine.y > mine.x ? -mine.y : mine.x;
            const __half d = __float2half_rn(__fmul_rn(top, -0.125f));
            const float f = __half2float(d);
            const float ratio = f != 0.0f ? __frcp_rn(f) : 0.0f;
            const float inv[2] = {__shfl_sync(~0u, ratio, first_lane), __shfl_sync(~0u, ratio, first_lane + 1)};
            // 1 / d of an ordinary d is 2^14 at most; an infinite one leaves 0
            const bool usual = !nan && fabsf(ratio) <= 16384.0f && fabsf(f) < INFINITY;
            uint32_t w[2];
            if (__all_sync(~0u, usual)) {
                w[0] = pack_4(y[0], inv[0], false);
                w[1] = pack_4(y[1], inv[1], false);
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        const float z = __fmul_rn(y[s][j], inv[s]);
                        if (!(fabsf(z) < INFINITY)) y[s][j] = 0.0f;  // NaN, or what an infinite d makes of it
                        if (inv[s] == 0.0f) y[s][j] = 0.0f;
                    }
                w[0] = pack_4(y[0], inv[0], true);
                w[1] = pack_4(y[1], inv[1], true);
            }
            if (codes >= 0 && at < p.lanes) {
                if constexpr (E == 8) {
                    *reinterpret_cast<uint32_t *>(k_lane + codes) = w[0];
                    *reinterpret_cast<uint16_t *>(v_lane + codes) = static_cast<uint16_t>(w[1]);
                    *reinterpret_cast<uint16_t *>(v_lane + codes + 2 * nb) = static_cast<uint16_t>(w[1] >> 16);
                } else {
                    *reinterpret_cast<uint16_t *>(k_lane + codes) = static_cast<uint16_t>(w[0]);
                    *reinterpret_cast<uint16_t *>(v_lane + codes) = static_cast<uint16_t>(w[1]);
                }
                if (of < 2) *reinterpret_cast<__half *>(s_lane + scale_at[t]) = d;
            }
        } else {
            const float amax[2] = {fmaxf(m[0].x, m[0].y), fmaxf(m[1].x, m[1].y)};
            // as q8kv_write_kernel: 1 / amax and amax / 127 of k, then of v, a division a lane
            const float a = of & 2 ? amax[1] : amax[0], num = of & 1 ? a : 1.0f, den = of & 1 ? 127.0f : a;
            float ratio = den > 0.0f ? __fdiv_rn(num, den) : 0.0f;
            if (!(of & 1)) ratio = __fmul_rn(127.0f, ratio);
            const float inv[2] = {__shfl_sync(~0u, ratio, first_lane), __shfl_sync(~0u, ratio, first_lane + 2)};
            const bool usual = !nan && amax[0] < INFINITY && amax[1] < INFINITY && inv[0] < INFINITY && inv[1] < INFINITY;
            uint32_t w[2][E / 4];
            if (__all_sync(~0u, usual)) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < E / 4; ++j) w[s][j] = pack_8_usual(y[s] + 4 * j, inv[s]);
            } else {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < E / 4; ++j) w[s][j] = pack_8(y[s] + 4 * j, inv[s]);
            }
            if (live && codes >= 0) {
                if constexpr (E == 8) {
                    *reinterpret_cast<uint2 *>(k_lane + codes) = make_uint2(w[0][0], w[0][1]);
                    *reinterpret_cast<uint2 *>(v_lane + codes) = make_uint2(w[1][0], w[1][1]);
                } else {
                    *reinterpret_cast<uint32_t *>(k_lane + codes) = w[0][0];
                    *reinterpret_cast<uint32_t *>(v_lane + codes) = w[1][0];
                }
            }
            if (codes >= 0 && at < p.lanes && (of == 1 || of == 3)) *reinterpret_cast<float *>(s_lane + scale_at[t]) = ratio;
        }
    }
}

// Tokens a lane of a large call: of writes (8190 tokens of 32 heads x 128 in bf16: 38.9 us, 41.0 with two, 46.6 with one), and
// of what only rotates (f32, 5003 tokens of 12 heads of 80: 7.2 us, 8.4 with two, 8.9 with one)
constexpr int kStoreTokens = 4;

template <typename T, int BITS, bool ROT>
void launch_store(const StoreParams &p, bool vec, const Shape &s, size_t smem, cudaStream_t stream) {
    if (!vec)
        kv_store_kernel<T, BITS, ROT, false, 1><<<s.grid, s.block, smem, stream>>>(p);
    else if (ROT || !s.many)
        kv_store_kernel<T, BITS, ROT, true, 1><<<s.grid, s.block, smem, stream>>>(p);
    else
        kv_store_kernel<T, BITS, ROT, true, ROT ? 1 : kStoreTokens><<<s.grid, s.block, smem, stream>>>(p);
}

}  // namespace kv
