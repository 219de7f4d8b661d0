// Attention of wide draft trees over a Q8_0 cache on the 5th-generation tensor
// cores (../../include/q8kv.h): up to 128 query rows (node, head of the group) of
// one kv head at a time, bf16 queries and outputs.
//
//     S[r, j] = q[r] . K[j],   O[r] += P[r, j] V[j],   P = exp2(scale log2(e) S + E - M)
//
// Work is the line of units of kv_attend.cuh with 128-row items and tiles of 128
// keys, one CTA per SM.  With 128 rows a code meets 128 multiplications on each
// side, so the products belong to tcgen05.mma and the rest of the SM keeps it fed:
//   * eight convert warps take 16 keys of a tile each.  cp.async brings the codes
//     and scales of two tiles to come while they turn this one's into f16 operands in
//     shared memory, K a tile ahead of V.  A key's row is normalised by a power of two
//     (one for the warp's 16 keys, or one per key where some of them are drafted) that
//     goes into the softmax, and code times scale is formed with the scale in two
//     f16 parts.  K is kept in two f16 parts, 22 bits, since a score's error is a
//     weight's relative one and lse is f32; V is rounded once to 11 bits, as outputs
//     are bf16.  (f32 and f16 outputs stay with kv_attend.cuh.)  K and V tiles have
//     the same layout, 128-byte rows of a key's 64 e, swizzled: K is read K-major, V
//     MN-major.
//   * one lane of a warp that stays together issues the MMAs: S = Q K^T of tile g
//     (lower part, then upper), then O += P V of tile g - 1.
//   * two softmax warpgroups take alternate tiles, a thread a row, each with its own
//     S, O (f32) and, in place of S, P (f16) in tensor memory: 2 x (128 + 128)
//     columns, all of them.  While one exponentiates, the other's products run.
//     P is 2^7 at the maximum, so that f16 holds weights down to 2^-31 of the largest,
//     and the maximum only moves when P would pass 2^15: O is rarely rescaled.
//   * at an item's end each warpgroup adds half of the columns of both O.
// All hand-overs are mbarriers, every wait is bounded (2 s); one that runs out is
// recorded in the plan's error word and the CTA leaves, once its MMAs have ended and
// its parts of cut items are counted: the tickets are whole after every call.
//
// 16 requests of 700 .. 5000 tokens, trees of 31 nodes, 32 heads over 8 of 128: 87.3 us,
// 239 TFLOP/s of the two products, 1.2 TB/s of cache.  A tile takes 5600 cycles, of
// which the MMAs run 1400; turning its codes into operands bounds it, then 8 us until a
// CTA's first scores are there and 10 us of joining cut items at the end.
#pragma once

#include "kv_attend.cuh"

namespace kv {

constexpr int kTcRows = 128, kTcKeys = 128;
constexpr int kTcSoftWarps = 8, kTcConvWarps = 8;
constexpr int kTcWarpKeys = 128 / kTcConvWarps;  // keys of a tile that a convert warp takes
constexpr int kTcMmaWarp = kTcSoftWarps + kTcConvWarps;
constexpr int kTcThreads = (kTcMmaWarp + 1) * 32;
constexpr int kTcHalf = kTcKeys * 128;          // 128 rows of 64 f16
constexpr int kTcErrWait = 1;
constexpr uint64_t kTcDrainNs = 2000000000ull;  // for MMAs that were issued: they end by themselves, whatever a plan's waits are
constexpr float kTcTop = 7.0f;                  // log2 of P at the row's maximum when that is taken
constexpr float kTcSlack = 15.0f;               // and how far P may grow before it is taken anew (f16 ends at 2^16)
constexpr int kTcItemUnits = 4;                 // an item's fixed cost in tiles (16 requests of 700 .. 5000 tokens, 124 rows:
                                                // 149, 114, 88.4, 86.5, 86.0, 89.6 us with 1 .. 6; 24 of 300 .. 3000, 68 rows: 83.1 with 4,
                                                // 83.6 with 5)

template <int DP>
struct TcSmem {
    static constexpr int kTile = DP / 64 * kTcHalf;   // one operand of 128 rows: 64 e after 64 e
    static constexpr int kQ = 0, kK = kTile, kLo = 2 * kTile, kV = 3 * kTile, kMeta = 4 * kTile;
    static constexpr int kMetaTile = kTcKeys * 16;    // per key: K's factor, E, 2^-E, flag
    // a convert warp's keys of a tile as they are in the cache: codes of K and V, scales of both
    // (a row's pitch is 16 mod 128 bytes: 8 lanes read 16 bytes of 8 rows)
    static constexpr int kRaw = kMeta + 4 * kMetaTile, kRawPitch = DP + 16;
    static constexpr int kRawV = kTcWarpKeys * kRawPitch, kRawS = 2 * kTcWarpKeys * kRawPitch;
    static constexpr int kRawWarp = 2 * kTcWarpKeys * kRawPitch + 2 * kTcWarpKeys * (DP / 32) * 4;
    static constexpr int kUsed = kRaw + 2 * kTcConvWarps * kRawWarp;  // of two tiles
    static constexpr int kTotal = kUsed + 1024;  // the swizzled tiles begin on 1024 bytes
    static constexpr int kPart = kTcRows * (DP + 2);  // floats of a partial result: O by 4 columns x 128 rows, m, l
};

__device__ __forceinline__ uint32_t tc_smem(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void tc_bar_init(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void tc_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc_smem(bar)) : "memory");
}
// whether the phase of `parity` is over, after at most about `ns` (the hardware may give up earlier)
__device__ __forceinline__ bool tc_try(uint64_t *bar, uint32_t parity, uint32_t ns) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(tc_smem(bar)), "r"(parity), "r"(ns)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ uint64_t tc_now() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// The phase of `parity`; false if the CTA is leaving or the time is up.  A warp sleeps up to 1 ms at a time, so the
// clock is hardly ever read.
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, const volatile int *leave, uint64_t wait_ns) {
    if (tc_try(bar, parity, 0)) return true;
    const uint32_t nap = static_cast<uint32_t>(wait_ns < 1000000 ? wait_ns : 1000000);
    const uint64_t t0 = tc_now();
    for (;;) {
        if (tc_try(bar, parity, nap)) return true;
        if (leave != nullptr && *leave) return false;
        if (tc_now() - t0 > wait_ns) return false;
    }
}
// one lane of a warp that is together
__device__ __forceinline__ bool tc_elect() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand of 128-byte rows, 128-byte swizzle (rows in eights 1024 bytes apart); `next`: bytes to the next
// 64 elements along M or N, where a row runs along it.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t next) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(next >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// place of 16 bytes, the c-th of a row, in an operand's tile
__device__ __forceinline__ uint32_t tc_place(int row, int c) {
    return static_cast<uint32_t>((c >> 3) * kTcHalf + row * 128 + (((c ^ row) & 7) << 4));
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc_smem(bar)) : "memory");
}
// 32 columns of the thread's lane
__device__ __forceinline__ void tc_ld32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 16 columns of the thread's lane, not waited for
__device__ __forceinline__ void tc_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_st32(uint32_t at, const float (&v)[32]) {
    uint32_t r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t at, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// two f16 codes times a scale in two parts, rounded once, and what that leaves (exact but for c * lo's last bits)
__device__ __forceinline__ uint32_t tc_scaled(uint32_t codes, uint32_t hi, uint32_t lo, uint32_t *rest) {
    uint32_t t, y;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(t) : "r"(codes), "r"(lo));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(codes), "r"(hi), "r"(t));
    if (rest != nullptr) {
        uint32_t d;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(codes), "r"(hi), "r"(y ^ 0x80008000u));
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(*rest) : "r"(d), "r"(t));
    }
    return y;
}

// power of two with exponent e
__device__ __forceinline__ float tc_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Counts a part of a cut item, tiles first .. first + tiles_k - 1 of the line, that its CTA will not write: as the joins
// of the kernel count it, so that the item's tickets are 0 again when all of its CTAs have come.
static __device__ __noinline__ void tc_count(const Split split, unsigned *ticket, unsigned *group_tickets, int64_t first, int64_t tiles_k) {
    auto arrive = [](unsigned *at, unsigned count) -> bool {
        const bool last = atomicAdd(at, 1u) == count - 1;
        if (last) *at = 0;
        return last;
    };
    const int c0 = static_cast<int>(split.owner(first)), c1 = static_cast<int>(split.owner(first + tiles_k - 1));
    if (c1 - c0 < kJoinGroup) {
        arrive(ticket, c1 - c0 + 1);
    } else {
        const int grp = blockIdx.x / kJoinGroup, lo = max(c0, grp * kJoinGroup), hi = min(c1, grp * kJoinGroup + kJoinGroup - 1);
        if (arrive(group_tickets + 2 * grp + (c0 < grp * kJoinGroup ? 0 : 1), hi - lo + 1))
            arrive(ticket, c1 / kJoinGroup - c0 / kJoinGroup + 1);
    }
}

// A convert warp's place: an item, and which of its tiles here.
struct TcTile {
    Place w;
    int64_t kt;
    int n, i;  // the item's tiles of this CTA, and which of them
    bool any;
};

template <int DP>
__global__ void __launch_bounds__(kTcThreads, 1) q8kv_attend_tc_kernel(const AttendParams p) {
    using T = __nv_bfloat16;
    using S = TcSmem<DP>;
    constexpr int PARTS = DP / 16, KPL = 32 / PARTS, NL = kTcWarpKeys / KPL;  // 16-byte pieces of a row, keys of a load, loads
    constexpr int NB = DP / 32, WK = kTcWarpKeys;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *const smem = smem_raw + ((1024u - (tc_smem(smem_raw) & 1023u)) & 1023u);
    __shared__ __align__(8) uint64_t k_full[2], k_free[2], v_full, v_free[2], s_full[2], p_full[2];
    __shared__ __align__(8) uint64_t soft_bar;            // among the softmax warps
    __shared__ uint32_t tmem_at;
    __shared__ int leave, is_last;
    __shared__ int64_t scan_units[kTcThreads / 32], scan_items[kTcThreads / 32];
    __shared__ int64_t start_b, start_item, start_unit;
    __shared__ float row_mul[4][kTcRows];                // by item
    __shared__ float2 row_ml[2][kTcRows];                // a warpgroup's maximum and sum
    __shared__ TcTile tiles[kTcConvWarps][2];
    __shared__ Place places[kTcSoftWarps];
    __shared__ uint32_t there_bits[4][kTcConvWarps];     // by tile: the keys that are there
    __shared__ uint32_t plain_keys[4][kTcConvWarps];     // by tile: whether all rows see a warp's keys, with one normaliser

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const volatile int *leaving = &leave;

    // ---- the CTA's share of the line of units (as in kv_attend.cuh)
    Split split;
    int64_t u, u_end;
    Place w;
    {
        const int per = (p.requests + kTcThreads - 1) / kTcThreads;
        const int b0 = min(tid * per, p.requests), b1 = min(b0 + per, p.requests);
        int64_t units = 0, items = 0;
        auto units_in = [&](const Place &x) { return static_cast<int64_t>(p.c.heads) * x.tiles_r * (x.tiles_k + kTcItemUnits); };
        for (int b = b0; b < b1; ++b) {
            load_request<kTcRows, kTcKeys>(p, b, w);
            units += units_in(w);
            items += static_cast<int64_t>(p.c.heads) * w.tiles_r;
        }
        int64_t iu = units, ii = items;
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
        if (tid == 0) {
            for (int i = 0; i < 2; ++i) {
                tc_bar_init(k_full + i, kTcConvWarps);
                tc_bar_init(k_free + i, 1);
                tc_bar_init(v_free + i, 1);
                tc_bar_init(s_full + i, 1);
                tc_bar_init(p_full + i, 4);
            }
            tc_bar_init(&soft_bar, kTcSoftWarps);
            tc_bar_init(&v_full, kTcConvWarps);
            leave = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();
        int64_t total = 0, before_u = 0, before_i = 0;
        for (int i = 0; i < kTcThreads / 32; ++i) {
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
        if (u >= before_u && u < before_u + units) {
            int b = b0;
            for (; b < b1; ++b) {
                load_request<kTcRows, kTcKeys>(p, b, w);
                const int64_t n = units_in(w);
                if (u < before_u + n) break;
                before_u += n;
                before_i += static_cast<int64_t>(p.c.heads) * w.tiles_r;
            }
            start_b = b;
            start_unit = before_u;
            start_item = before_i;
        }
        __syncthreads();
        load_request<kTcRows, kTcKeys>(p, static_cast<int>(start_b), w);
        const int64_t k = (u - start_unit) / (w.tiles_k + kTcItemUnits);
        w.h = static_cast<int>(k / w.tiles_r);
        w.rt = static_cast<int>(k - static_cast<int64_t>(w.h) * w.tiles_r);
        w.item = start_item + k;
        w.first = start_unit + k * (w.tiles_k + kTcItemUnits) + kTcItemUnits;
    }
    auto advance = [&](Place &x) {
        x.first += x.tiles_k + kTcItemUnits;
        ++x.item;
        if (++x.rt == x.tiles_r) {
            x.rt = 0;
            if (++x.h == p.c.heads) {
                x.h = 0;
                do load_request<kTcRows, kTcKeys>(p, x.b + 1, x);
                while (x.tiles_r == 0);
            }
        }
    };
    // the CTA's tiles of item x: kt0 .. kt1 - 1
    auto tiles_of = [&](const Place &x, int64_t *kt0) -> int {
        *kt0 = max(u, x.first) - x.first;
        return static_cast<int>(max(min(u_end, x.first + x.tiles_k) - x.first, *kt0) - *kt0);
    };
    auto more = [&](const Place &x) { return x.first + x.tiles_k < u_end; };

    if (warp == kTcMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(&tmem_at)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_at;
    const uint32_t base = tc_smem(smem);
    bool bad = false;

    if (warp == kTcMmaWarp) {
        // ================ the MMAs.  The warp stays together and one lane issues: the operands' descriptors are then
        // uniform and need no moves between register files, which held the issue to 200 cycles an MMA.
        constexpr uint32_t idesc_s = (1u << 4) | (static_cast<uint32_t>(kTcKeys >> 3) << 17) | (static_cast<uint32_t>(kTcRows >> 4) << 24);
        constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(DP >> 3) << 17) | (static_cast<uint32_t>(kTcRows >> 4) << 24);
        const bool first_lane = tc_elect();
        const uint64_t dq = tc_desc(base + S::kQ, 16), dk = tc_desc(base + S::kK, 16), dl = tc_desc(base + S::kLo, 16),
                       dv = tc_desc(base + S::kV, kTcHalf);
        // 64 e further, 16 e further, 16 keys further, as descriptors count
        constexpr uint64_t kHalfStep = kTcHalf >> 4, kStep = 32 >> 4, kKeyStep = 2048 >> 4;
        auto scores = [&](uint32_t d) {  // S = Q K^T, lower part first
#pragma unroll
            for (int e = 0; e < DP / 16; ++e)
                tc_mma_ss(d, dq + (e / 4) * kHalfStep + (e % 4) * kStep, dl + (e / 4) * kHalfStep + (e % 4) * kStep, idesc_s, e == 0 ? 0u : 1u);
#pragma unroll
            for (int e = 0; e < DP / 16; ++e)
                tc_mma_ss(d, dq + (e / 4) * kHalfStep + (e % 4) * kStep, dk + (e / 4) * kHalfStep + (e % 4) * kStep, idesc_s, 1u);
        };
        auto products = [&](uint32_t d, uint32_t a, uint32_t add) {  // O += P V
            tc_mma_ts(d, a, dv, idesc_o, add);
#pragma unroll
            for (int k = 1; k < kTcKeys / 16; ++k) tc_mma_ts(d, a + k * 8, dv + k * kKeyStep, idesc_o, 1u);
        };
        int64_t g = 0;                    // tile of the CTA
        int64_t scored = -1, summed = -1; // the last tiles whose scores and whose O += P V were issued
        int last_first = 0;               // whether tile g - 1 was its warpgroup's first of an item
        auto second = [&](int64_t t, bool first) -> bool {
            const uint32_t x = static_cast<uint32_t>(t) & 1u, ph = static_cast<uint32_t>(t >> 1) & 1u;
            bool ok = tc_wait(p_full + x, ph, leaving, p.wait_ns) && tc_wait(&v_full, static_cast<uint32_t>(t) & 1u, leaving, p.wait_ns);
            ok = __all_sync(~0u, ok);
            if (!ok) return false;
            tc_after();
            if (first_lane) {
                products(tmem + 256 + x * 128, tmem + x * 128, first ? 0u : 1u);
                tc_commit(v_free + x);
            }
            __syncwarp();
            summed = t;
            return true;
        };
        for (;;) {
            int64_t kt0;
            const int n = tiles_of(w, &kt0);
            for (int i = 0; i < n && !bad; ++i, ++g) {
                const uint32_t x = static_cast<uint32_t>(g) & 1u, ph = static_cast<uint32_t>(g >> 1) & 1u;
                if (!__all_sync(~0u, tc_wait(k_full + x, ph, leaving, p.wait_ns))) {
                    bad = true;
                    break;
                }
                tc_after();
                if (first_lane) {
                    scores(tmem + x * 128);
                    tc_commit(k_free + x);
                    tc_commit(s_full + x);
                }
                __syncwarp();
                scored = g;
                if (g > 0 && !second(g - 1, last_first != 0)) {
                    bad = true;
                    break;
                }
                last_first = i < 2;
            }
            if (bad || !more(w)) break;
            advance(w);
        }
        if (!bad && g > 0 && !second(g - 1, last_first != 0)) bad = true;
        if (bad) leave = 1;
        // What was issued has to end, and its last arrivals to be there, before the tensor memory, the operands and the
        // barriers go back: also of a CTA that leaves because a wait ran out, so not with that wait's bound.
        auto drain = [&](uint64_t *bars, int64_t t) {
            if (t >= 0 && !tc_wait(bars + (t & 1), static_cast<uint32_t>(t >> 1) & 1u, nullptr, kTcDrainNs)) bad = true;
        };
        drain(k_free, scored);
        drain(s_full, scored);
        drain(v_free, summed);
        if (bad && lane == 0) atomicOr(p.err, kTcErrWait);
    } else if (warp >= kTcSoftWarps) {
        // ================ convert
        const int cw = warp - kTcSoftWarps, part = lane % PARTS, sub = lane / PARTS;
        const bool live = part * 16 < p.c.dim;
        const int ct = tid - kTcSoftWarps * 32;  // thread among the convert warps
        unsigned char *const raws = smem + S::kRaw + cw * (2 * S::kRawWarp);  // by tile % 2: K, V, scales of K [key][NB], of V
        for (int i = lane; i < 2 * S::kRawWarp / 16; i += 32) reinterpret_cast<uint4 *>(raws)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
        // A tile of the CTA: its item and its number there.  The warp keeps two in shared memory, this one and the
        // next but one: in registers they would push the codes out.
        TcTile *const here = tiles[cw], *const ahead = tiles[cw] + 1;
        auto settle = [&](TcTile &t) {  // to the first item with tiles, from t.w on
            for (;;) {
                t.n = tiles_of(t.w, &t.kt);
                t.i = 0;
                t.any = t.n > 0;
                if (t.any || !more(t.w)) return;
                advance(t.w);
            }
        };
        auto step = [&](TcTile *at) {
            __syncwarp();
            if (lane == 0 && at->any) {
                ++at->kt;
                if (++at->i == at->n) {
                    at->any = more(at->w);
                    if (at->any) {
                        TcTile t = *at;
                        advance(t.w);
                        settle(t);
                        *at = t;
                    }
                }
            }
            __syncwarp();
        };
        // row of the lane's key in a tile, or kNoRow
        auto find = [&](const TcTile *t) -> uint32_t {
            if (!t->any) return kNoRow;
            const int64_t pos = t->kt * kTcKeys + cw * WK + lane;
            const int64_t keys = min(static_cast<int64_t>(t->w.prefix) + t->w.nodes, static_cast<int64_t>(p.table_cols) * p.c.page_size);
            if (lane >= WK || pos >= keys) return kNoRow;
            const uint32_t at = static_cast<uint32_t>(pos), col = (__umulhi(at, p.page_mul) + at) >> p.page_shift;
            const int page = __ldg(p.table + static_cast<int64_t>(t->w.b) * p.table_row + col);
            if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.pages)) return kNoRow;
            return static_cast<uint32_t>(row_of(p.c, page, t->w.h, static_cast<int>(at - col * p.c.page_size)));
        };
        const bool wide_scales = NB == 4 && p.c.blocks == 4;
        auto codes = [&](const int8_t *from, uint32_t to, uint32_t row) {  // the warp's rows of one array
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const uint32_t r = __shfl_sync(~0u, row, j * KPL + sub);
                if (r != kNoRow && live)
                    cp_async16(to + (j * KPL + sub) * S::kRawPitch + part * 16, from + static_cast<uint64_t>(r) * static_cast<uint32_t>(p.c.dim) + part * 16);
            }
        };
        auto issue_a = [&](uint32_t row, int64_t g) {  // codes of K, scales of both; an absent key's scales are 0
            unsigned char *raw = raws + (g & 1) * S::kRawWarp;
            float *raw_s = reinterpret_cast<float *>(raw + S::kRawS);
            codes(p.c.k_codes, tc_smem(raw), row);
            const uint32_t at = tc_smem(raw_s) + lane * (NB * 4);
            if (row != kNoRow) {
                const float *ks = p.c.k_scales + static_cast<uint64_t>(row) * static_cast<uint32_t>(p.c.blocks);
                const float *vs = p.c.v_scales + static_cast<uint64_t>(row) * static_cast<uint32_t>(p.c.blocks);
                if (wide_scales) {
                    cp_async16(at, ks);
                    cp_async16(at + WK * NB * 4, vs);
                } else {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        if (b < p.c.blocks) {
                            cp_async4(at + 4 * b, ks + b);
                            cp_async4(at + WK * NB * 4 + 4 * b, vs + b);
                        }
                }
            } else if (lane < WK) {
#pragma unroll
                for (int b = 0; b < NB; ++b) raw_s[lane * NB + b] = raw_s[WK * NB + lane * NB + b] = 0.0f;
            }
            cp_commit();
        };
        auto issue_b = [&](uint32_t row, int64_t g) {  // codes of V
            codes(p.c.v_codes, tc_smem(raws) + static_cast<uint32_t>(g & 1) * S::kRawWarp + S::kRawV, row);
            cp_commit();
        };
        // exponent e with scales below 2^(e + 7): codes times scale / 2^e stay below 2^14
        auto exponent = [](uint32_t bits) -> int { return max(min(static_cast<int>(bits >> 23) - 127 - 6, 120), -100); };
        // Converting, a lane has one key (lane % WK) and every second piece of its row: 8 lanes store 16 bytes of 8 keys,
        // which the swizzle puts into 8 different banks' lines.
        static_assert(WK == 16, "two lanes a key");
        const int key = lane & 15, odd_piece = lane >> 4;
        auto store = [&](uint32_t tile, int piece, const uint32_t (&o)[8]) {
            const int r = cw * WK + key;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + tc_place(r, 2 * piece)), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + tc_place(r, 2 * piece + 1)), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
        };
        // a piece of 16 codes times scale / 2^e to the tile, and what that rounds off
        auto convert = [&](uint32_t tile, int piece, const unsigned char *from, float scale, uint32_t (*rest)[8]) {
            const uint4 c = *reinterpret_cast<const uint4 *>(from + key * S::kRawPitch + piece * 16);
            const __half hi = __float2half_rn(scale), lo = __float2half_rn(scale - __half2float(hi));
            const uint32_t h2 = pack_half2(__half2float(hi), __half2float(hi)), l2 = pack_half2(__half2float(lo), __half2float(lo));
            const uint32_t in[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = tc_scaled(unbias(__byte_perm(in[i / 2], 0x64646464u, i % 2 ? 0x4342u : 0x4140u)), h2, l2, rest ? &(*rest)[i] : nullptr);
            store(tile, piece, o);
        };
        auto waited = [&](uint64_t *bar, int64_t phase) -> bool {  // whole warps
            if (!tc_wait(bar, static_cast<uint32_t>(phase) & 1u, leaving, p.wait_ns)) bad = true;
            bad = __any_sync(~0u, bad);
            return !bad;
        };

        int item_no = -1;
        float v_scale[NB] = {};  // the lane's key's scales of V, normalised, of the tile whose K was converted last
        // q and K of tile g
        auto do_k = [&](int64_t g, uint32_t row, uint32_t row_after) -> bool {
            const TcTile &t = *here;
            // the scores of the tile before, which end its use of q and K (and tile g - 4's of the rings' entries)
            if (g > 0 && !waited(k_free + ((g - 1) & 1), (g - 1) >> 1)) return false;
            const bool all_before = t.kt * kTcKeys + (cw + 1) * WK <= t.w.prefix;
            if (t.i == 0) {
                ++item_no;
                constexpr int TPR = kTcConvWarps * 32 / kTcRows, H = DP / 8 / TPR;  // threads a row, a thread's groups of 8
                const int r = ct / TPR, g0 = ct % TPR * H;
                const int rows = min(kTcRows, t.w.nodes * p.group - t.w.rt * kTcRows);
                const int idx = t.w.rt * kTcRows + r, node = idx / p.group, hq = t.w.h * p.group + idx - node * p.group;
                const T *src = static_cast<const T *>(p.q) + (static_cast<int64_t>(t.w.row0) + node) * p.q_row + hq * p.q_head;
                union Eight {
                    uint4 u;
                    T t[8];
                };
                auto eight = [&](int k) -> Eight {  // the k-th of the thread's groups
                    const int e = 8 * (g0 + k);
                    Eight y;
                    y.u = make_uint4(0, 0, 0, 0);
                    if (r < rows && e < p.c.dim) {
                        if (p.q_vec) {
                            y.u = __ldg(reinterpret_cast<const uint4 *>(src + e));
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) y.t[j] = src[e + j];
                        }
                    }
                    return y;
                };
                uint32_t top = 0;
#pragma unroll 4
                for (int k = 0; k < H; ++k) {
                    const Eight y = eight(k);
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(to_f32(y.t[j])) & 0x7FFFFFFFu);
                }
#pragma unroll
                for (int d = 1; d < TPR; d *= 2) top = max(top, __shfl_xor_sync(~0u, top, d));
                const int ex = min(max(static_cast<int>(top >> 23) - 127 - 10, -100), 100);
                const float down = copysignf(tc_pow2(-ex), p.scale_log2);
#pragma unroll 4
                for (int k = 0; k < H; ++k) {
                    const Eight y = eight(k);
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = pack_half2(to_f32(y.t[2 * e]) * down, to_f32(y.t[2 * e + 1]) * down);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + S::kQ + tc_place(r, g0 + k)), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
                }
                if (g0 == 0)
                    row_mul[item_no & 3][r] = fmaxf(tc_pow2(ex) * fabsf(p.scale_log2), 1e-37f);
            }
            if (g <= 2)
                cp_wait<2>();
            else
                cp_wait<3>();  // V of g - 1, K of g + 1 and V of g may be on their way
            __syncwarp();
            const unsigned char *raw = raws + (g & 1) * S::kRawWarp;
            const float *raw_s = reinterpret_cast<const float *>(raw + S::kRawS);
            const int x = static_cast<int>(g & 1), ring = static_cast<int>(g & 3);
            float4 *meta = reinterpret_cast<float4 *>(smem + S::kMeta + ring * S::kMetaTile) + cw * WK;
            const uint32_t there = __ballot_sync(~0u, row != kNoRow);
            bool plain = all_before && there == (1u << WK) - 1u;
            // ---- normalisers: of each key, and of all keys if every row sees them
            float k_scale[NB];
            {
                uint32_t bk = 0, bv = 0;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    k_scale[b] = raw_s[key * NB + b];
                    v_scale[b] = raw_s[WK * NB + key * NB + b];
                    bk = max(bk, __float_as_uint(k_scale[b]) & 0x7FFFFFFFu);
                    bv = max(bv, __float_as_uint(v_scale[b]) & 0x7FFFFFFFu);
                }
                // a scale that is not finite: the key's rows are 0 here, and the softmax makes NaN of who sees it
                const bool odd = bk >= 0x7F800000u || bv >= 0x7F800000u;
                plain = plain && !__any_sync(~0u, odd);
                if (plain) {
                    bk = __reduce_max_sync(~0u, bk);
                    bv = __reduce_max_sync(~0u, bv);
                }
                const int ek = exponent(odd ? 0 : bk), ev = exponent(odd ? 0 : bv);
                if (lane < WK) meta[key] = make_float4(tc_pow2(ek), static_cast<float>(ev), tc_pow2(-ev), odd ? 1.0f : 0.0f);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    v_scale[b] = odd ? 0.0f : v_scale[b] * tc_pow2(-ev);
                    k_scale[b] = odd ? 0.0f : k_scale[b] * tc_pow2(-ek);
                }
            }
            // ---- K
            const uint32_t kb = base + S::kK;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint32_t rest[8];
                convert(kb, 2 * b + odd_piece, raw, k_scale[b], &rest);
                store(base + S::kLo, 2 * b + odd_piece, rest);
            }
            if (lane == 0) {
                there_bits[ring][cw] = there;
                plain_keys[ring][cw] = plain;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc_arrive(k_full + x);
            // (after the fence, which would wait for these copies: 2000 cycles a tile)
            issue_a(row_after, g + 2);
            return true;
        };
        // V of tile g
        auto do_v = [&](int64_t g, const float (&scale)[NB], uint32_t row_after) -> bool {
            cp_wait<3>();  // K of g + 1 .. g + 2 and V of g + 1 may be on their way
            __syncwarp();
            if (g >= 1 && !waited(v_free + ((g - 1) & 1), (g - 1) >> 1)) return false;
#pragma unroll
            for (int b = 0; b < NB; ++b) convert(base + S::kV, 2 * b + odd_piece, raws + (g & 1) * S::kRawWarp + S::kRawV, scale[b], nullptr);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc_arrive(&v_full);
            issue_b(row_after, g + 2);
            return true;
        };
        if (lane == 0) {
            TcTile t;
            t.w = w;
            settle(t);
            *here = t;
            *ahead = t;
        }
        __syncwarp();
        if (here->any) {
            // r0, r1, r2: rows of the tiles g + 1, g + 2 and g + 3 of the loop below; `here` is tile g + 1, `ahead` g + 3
            // (g = -1: only the first tile's K)
            uint32_t r0 = find(here);
            issue_a(r0, 0);
            issue_b(r0, 0);
            step(ahead);
            uint32_t r1 = find(ahead);
            issue_a(r1, 1);
            issue_b(r1, 1);
            step(ahead);
            uint32_t r2 = find(ahead);
            int64_t keys = 0;  // tiles whose K is converted
            for (int64_t g = -1;; ++g) {
                float scale[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) scale[b] = v_scale[b];
                if (here->any) {
                    if (!do_k(keys++, r0, r2)) break;
                } else {
                    cp_commit();  // in the place of K's group
                }
                if (g >= 0 && !do_v(g, scale, r1)) break;
                if (g + 1 == keys) break;
                step(here);
                step(ahead);
                r0 = r1;
                r1 = r2;
                r2 = find(ahead);
            }
        }
        cp_wait<0>();
        if (bad) {
            leave = 1;
            if (lane == 0) atomicOr(p.err, kTcErrWait);
        }
    } else {
        // ================ softmax: warpgroup x takes tiles g = x mod 2
        const int x = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128, to = tmem + lanes + 256 + x * 128;
        const int64_t pitch = S::kPart;
        int64_t g = 0;
        int item_no = 0;
        bool first_item = true;
        uint32_t soft_phase = 0;
        bool counted = false;  // the item's part, if it is one
        Place &pl = places[warp];  // the warp's copy
        if (lane == 0) pl = w;
        __syncwarp();
        // all softmax warps; false (in whole warps) if the CTA is leaving
        auto soft_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) tc_arrive(&soft_bar);
            const bool ok = tc_wait(&soft_bar, soft_phase, leaving, p.wait_ns);
            soft_phase ^= 1u;
            if (!ok) leave = 1;  // at once: a warp that leaves may come here a few times more
            return __all_sync(~0u, ok);
        };
        for (;;) {
            int64_t kt0;
            const int n = tiles_of(pl, &kt0);
            if (n > 0) {
                const int idx = pl.rt * kTcRows + r;
                const bool whole = n == pl.tiles_k;
                float m = -INFINITY, l = 0.0f;
                bool have = false;  // O holds something
                float mul = 0.0f;
                for (int i = 0; i < n; ++i, ++g) {
                    if (static_cast<int>(g & 1) != x) continue;
                    const int ring = static_cast<int>(g & 3);
                    if (!tc_wait(s_full + x, static_cast<uint32_t>(g >> 1) & 1u, leaving, p.wait_ns)) bad = true;
                    if (__any_sync(~0u, bad)) {
                        bad = true;
                        break;
                    }
                    tc_after();
                    if (!have) mul = row_mul[item_no & 3][r];
                    const float4 *meta = reinterpret_cast<const float4 *>(smem + S::kMeta + ring * S::kMetaTile);
                    // for each convert warp's keys, whether all rows see them; and which of 32 keys this row sees
                    uint32_t fast = 0, see[4];
#pragma unroll
                    for (int q = 0; q < kTcConvWarps; ++q) fast |= plain_keys[ring][q] << q;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        see[q] = there_bits[ring][2 * q] | there_bits[ring][2 * q + 1] << 16;
                        const int64_t j0 = (kt0 + i) * kTcKeys + 32 * q - pl.prefix;
                        if (j0 + 32 > 0)
                            see[q] &= sees(p.mask, p.mask_row, p.mask_words, p.group, pl.nodes, pl.row0, static_cast<int>(j0), idx);
                    }
                    // ---- the row's maximum of s + E
                    float top = -INFINITY;
                    auto look = [&](int c16, const uint32_t (&v)[16]) {
                        const float4 *mt = meta + 16 * c16;
                        if ((fast >> (c16 * 16 / WK)) & 1u) {
                            float t0 = __uint_as_float(v[0]), t1 = __uint_as_float(v[1]);
#pragma unroll
                            for (int e = 2; e < 16; e += 2) {
                                t0 = fmaxf(t0, __uint_as_float(v[e]));
                                t1 = fmaxf(t1, __uint_as_float(v[e + 1]));
                            }
                            const float4 c = mt[0];
                            top = fmaxf(top, fmaf(fmaxf(t0, t1), mul * c.x, c.y));
                        } else {
                            const int q = c16 >> 1;
                            const uint32_t bits = (q == 0 ? see[0] : q == 1 ? see[1] : q == 2 ? see[2] : see[3]) >> (16 * (c16 & 1));
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float4 c = mt[e];
                                if ((bits >> e) & 1u) {
                                    top = fmaxf(top, fmaf(__uint_as_float(v[e]), mul * c.x, c.y));
                                    if (c.w != 0.0f) l = NAN;
                                }
                            }
                        }
                    };
                    {
                        uint32_t va[16], vb[16];
                        tc_ld16(ts, va);
                        tc_wait_ld();
#pragma unroll 1
                        for (int c16 = 0; c16 < 8; c16 += 2) {
                            tc_ld16(ts + 16 * (c16 + 1), vb);
                            look(c16, va);
                            tc_wait_ld();
                            if (c16 + 2 < 8) tc_ld16(ts + 16 * (c16 + 2), va);
                            look(c16 + 1, vb);
                            tc_wait_ld();
                        }
                    }
                    // ---- move the maximum?
                    float f = 1.0f;
                    if (top > m + kTcSlack || m == -INFINITY) {
                        f = m == -INFINITY ? 0.0f : ex2(m - (top - kTcTop));
                        m = top - kTcTop;
                    }
                    const float z = m == -INFINITY ? 0.0f : m;
                    l *= f;
                    if (have && __any_sync(~0u, f != 1.0f)) {
#pragma unroll 1
                        for (int q = 0; q < DP / 32; ++q) {
                            float v[32];
                            tc_ld32(to + 32 * q, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= f;
                            tc_st32(to + 32 * q, v);
                        }
                    }
                    have = true;
                    // ---- P, 16 keys at a time, the next 16 scores on their way
                    auto weigh = [&](int c16, const uint32_t (&v)[16]) {
                        uint32_t o[8];
                        const int q = c16 >> 1;
                        const float4 *mt = meta + 16 * c16;
                        if ((fast >> (c16 * 16 / WK)) & 1u) {
                            const float4 c = mt[0];
                            const float a = mul * c.x, d = c.y - z;
                            float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float p0 = ex2(fmaf(__uint_as_float(v[e]), a, d)), p1 = ex2(fmaf(__uint_as_float(v[e + 1]), a, d));
                                sum0 += p0;
                                sum1 += p1;
                                o[e / 2] = pack_half2(p0, p1);
                            }
                            l = fmaf(sum0 + sum1, c.z, l);
                        } else {
                            const uint32_t bits = (q == 0 ? see[0] : q == 1 ? see[1] : q == 2 ? see[2] : see[3]) >> (16 * (c16 & 1));
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float4 c0 = mt[e], c1 = mt[e + 1];
                                const float p0 = (bits >> e) & 1u ? ex2(fmaf(__uint_as_float(v[e]), mul * c0.x, c0.y - z)) : 0.0f;
                                const float p1 = (bits >> (e + 1)) & 1u ? ex2(fmaf(__uint_as_float(v[e + 1]), mul * c1.x, c1.y - z)) : 0.0f;
                                l = fmaf(p0, c0.z, l);
                                l = fmaf(p1, c1.z, l);
                                o[e / 2] = pack_half2(p0, p1);
                            }
                        }
                        tc_st8(ts + 8 * c16, o);
                    };
                    {
                        uint32_t va[16], vb[16];
                        tc_ld16(ts, va);
                        tc_wait_ld();
#pragma unroll 1
                        for (int c16 = 0; c16 < 8; c16 += 2) {
                            // (P's columns 8 c16 .. lie before the scores that are still to come)
                            tc_ld16(ts + 16 * (c16 + 1), vb);
                            weigh(c16, va);
                            tc_wait_ld();
                            if (c16 + 2 < 8) tc_ld16(ts + 16 * (c16 + 2), va);
                            weigh(c16 + 1, vb);
                            tc_wait_ld();
                        }
                    }
                    tc_wait_st();
                    tc_before();
                    __syncwarp();
                    if (lane == 0) tc_arrive(p_full + x);
                }
                if (bad) break;
                // ---- the item's results: both O must be complete
                row_ml[x][r] = make_float2(m, l);
                // (a barrier each, by turns: one for all could be two phases behind here, which looks like none)
                for (int back = 1; back <= 2 && back <= n; ++back) {
                    const int64_t t = g - back;
                    if (!tc_wait(v_free + static_cast<int>(t & 1), static_cast<uint32_t>(t >> 1) & 1u, leaving, p.wait_ns)) bad = true;
                }
                if (__any_sync(~0u, bad)) {
                    bad = true;
                    break;
                }
                tc_after();
                if (!soft_sync()) {
                    bad = true;
                    break;
                }
                const float2 ml0 = row_ml[0][r], ml1 = row_ml[1][r];
                const bool has[2] = {n > 1 || static_cast<int>((g - 1) & 1) == 0, n > 1 || static_cast<int>((g - 1) & 1) == 1};
                const float top = fmaxf(ml0.x, ml1.x), z = top == -INFINITY ? 0.0f : top;
                const float f0 = ex2(ml0.x - z), f1 = ex2(ml1.x - z);
                const float sum = fmaf(f0, ml0.y, f1 * ml1.y);
                const int rows = min(kTcRows, pl.nodes * p.group - pl.rt * kTcRows);
                const int node = idx / p.group, hq = pl.h * p.group + idx - node * p.group;
                const int64_t row = static_cast<int64_t>(pl.row0) + node;
                T *out = static_cast<T *>(p.out) + row * p.out_row + hq * p.out_head;
                const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (first_item ? 0 : 1);
                first_item = false;
                auto finish = [&](int e0, const float (&v)[32], float total) {  // columns e0 .. e0 + 31
                    const float inv = total > 0.0f ? __frcp_rn(total) : total == 0.0f ? 0.0f : total;
                    if (r >= rows) return;
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        if (e0 + e < p.c.dim) {
                            union {
                                uint4 u;
                                T t[8];
                            } y;
#pragma unroll
                            for (int k = 0; k < 8; ++k) y.t[k] = from_f32<T>(v[e + k] * inv);
                            if (p.out_vec) {
                                *reinterpret_cast<uint4 *>(out + e0 + e) = y.u;
                            } else {
#pragma unroll
                                for (int k = 0; k < 8; ++k) out[e0 + e + k] = y.t[k];
                            }
                        }
                    }
                };
                auto finish_lse = [&](float mm, float total) {
                    if (x == 0 && r < rows && p.lse) p.lse[row * p.heads_q + hq] = (mm + log2f(total)) * 0.693147180559945f;
                };
                // warpgroup x has the columns x * DP / 2 ..
#pragma unroll 1
                for (int q = 0; q < DP / 64; ++q) {
                    const int e0 = x * (DP / 2) + 32 * q;
                    float v[32], a[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0.0f;
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (has[y]) {  // a warpgroup without a tile has nothing in its O
                            tc_ld32(tmem + lanes + 256 + y * 128 + e0, a);
                            const float f = y ? f1 : f0;
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = fmaf(f, a[e], v[e]);
                        }
                    if (whole) {
                        finish(e0, v, sum);
                    } else {
                        float4 *part = reinterpret_cast<float4 *>(p.partial + slot * pitch) + e0 / 4 * kTcRows + r;
#pragma unroll
                        for (int e = 0; e < 8; ++e) part[e * kTcRows] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                }
                if (whole)
                    finish_lse(z, sum);
                else if (x == 0)
                    reinterpret_cast<float2 *>(p.partial + slot * pitch + kTcRows * DP)[r] = make_float2(top, sum);
                tc_before();
                if (!soft_sync()) {  // both O are read: the next item's products may replace them
                    bad = true;
                    break;
                }
                tc_after();
                if (!whole && pl.item < p.tickets_n) {
                    auto join = [&](int parts, int64_t head, int64_t at, int64_t step, bool last) {
                        if (bad) return;
                        auto part_of = [&](int i) { return p.partial + (i == 0 ? head : at + i * step) * pitch; };
                        float up = -INFINITY, total = 0.0f;
                        for (int i = 0; i < parts; ++i) up = fmaxf(up, __ldcg(reinterpret_cast<const float2 *>(part_of(i) + kTcRows * DP) + r).x);
                        const float zz = up == -INFINITY ? 0.0f : up;
                        for (int i = 0; i < parts; ++i) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part_of(i) + kTcRows * DP) + r);
                            total = fmaf(ex2(ml.x - zz), ml.y, total);
                        }
#pragma unroll 1
                        for (int q = 0; q < DP / 64; ++q) {
                            const int e0 = x * (DP / 2) + 32 * q;
                            float v[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = 0.0f;
                            for (int i = 0; i < parts; ++i) {
                                const float f = ex2(__ldcg(reinterpret_cast<const float2 *>(part_of(i) + kTcRows * DP) + r).x - zz);
                                const float4 *src = reinterpret_cast<const float4 *>(part_of(i)) + e0 / 4 * kTcRows + r;
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    if (e == 4) asm volatile("" ::: "memory");
                                    const float4 y = __ldcg(src + e * kTcRows);
                                    v[4 * e] = fmaf(f, y.x, v[4 * e]);
                                    v[4 * e + 1] = fmaf(f, y.y, v[4 * e + 1]);
                                    v[4 * e + 2] = fmaf(f, y.z, v[4 * e + 2]);
                                    v[4 * e + 3] = fmaf(f, y.w, v[4 * e + 3]);
                                }
                            }
                            if (last) {
                                finish(e0, v, total);
                            } else {
                                float4 *to4 = reinterpret_cast<float4 *>(p.partial + head * pitch) + e0 / 4 * kTcRows + r;
#pragma unroll
                                for (int e = 0; e < 8; ++e) to4[e * kTcRows] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                            }
                        }
                        if (last) {
                            finish_lse(zz, total);
                        } else {
                            if (!soft_sync()) bad = true;  // everybody has read the first part's maximum
                            if (x == 0) reinterpret_cast<float2 *>(p.partial + head * pitch + kTcRows * DP)[r] = make_float2(up, total);
                        }
                    };
                    auto arrive = [&](unsigned *ticket, unsigned count) -> bool {
                        __threadfence();
                        if (!soft_sync()) bad = true;
                        if (tid == 0) {  // (also if the CTA is leaving: its output is undefined, but the tickets are not)
                            const unsigned t = atomicAdd(ticket, 1u);
                            is_last = t == count - 1;
                            if (is_last) *ticket = 0;
                        }
                        __syncwarp();
                        if (!soft_sync()) bad = true;
                        const bool yes = *const_cast<volatile int *>(&is_last) != 0;
                        if (!soft_sync()) bad = true;
                        if (yes) __threadfence();
                        return yes;
                    };
                    const int c0 = static_cast<int>(split.owner(pl.first)), c1 = static_cast<int>(split.owner(pl.first + pl.tiles_k - 1));
                    const int slot_c0 = split.begin(c0) >= pl.first - kTcItemUnits ? 2 * c0 : 2 * c0 + 1;
                    if (c1 - c0 < kJoinGroup) {
                        if (arrive(p.tickets + pl.item, c1 - c0 + 1)) join(c1 - c0 + 1, slot_c0, 2 * c0, 2, true);
                    } else {
                        const int grp = blockIdx.x / kJoinGroup, g0 = c0 / kJoinGroup, g1 = c1 / kJoinGroup;
                        const int lo = max(c0, grp * kJoinGroup), hi = min(c1, grp * kJoinGroup + kJoinGroup - 1);
                        if (arrive(p.group_tickets + 2 * grp + (c0 < grp * kJoinGroup ? 0 : 1), hi - lo + 1)) {
                            join(hi - lo + 1, lo == c0 ? slot_c0 : 2 * lo, 2 * lo, 2, false);
                            if (arrive(p.tickets + pl.item, g1 - g0 + 1)) join(g1 - g0 + 1, slot_c0, 2 * kJoinGroup * g0, 2 * kJoinGroup, true);
                        }
                    }
                }
                ++item_no;
            }
            counted = true;
            if (bad || !more(pl)) break;
            counted = false;
            __syncwarp();
            if (lane == 0) {
                Place next = pl;
                advance(next);
                pl = next;
            }
            __syncwarp();
        }
        if (bad) {
            leave = 1;
            if (lane == 0) atomicOr(p.err, kTcErrWait);
            // what the first thread has not counted yet
            if (tid == 0) {
                Place y = pl;
                for (;;) {
                    int64_t kt0;
                    const int n = tiles_of(y, &kt0);
                    if (!counted && n > 0 && n != y.tiles_k && y.item < p.tickets_n)
                        tc_count(split, p.tickets + y.item, p.group_tickets, y.first, y.tiles_k);
                    if (!more(y)) break;
                    advance(y);
                    counted = false;
                }
            }
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == kTcMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

}  // namespace kv
