// Verification of drafted tokens (../../include/q8kv.h).
//
// Per visited node: the row's maximum, its whole-number weights w = trunc(2^40
// exp(z - max)) and their sums, then the tests of the node's children; at the end
// one prefix search.  Everything that is summed is a 64-bit whole number, so the
// split over threads and CTAs cannot change a result.
//
// One cluster of 16 CTAs walks one request and only reads the rows that the walk
// visits, and the first child's of each: a tree of many nodes costs its accepted
// path, not its size.  What bounds it is the longest path of the batch, a chain of
// rows each with a load, a sum, exchanges over the cluster and the tests; so a row is
// spread over 128 warps, and the CTAs are small (256 threads, 32 KB) so that the
// clusters of 30 and more requests are resident together and those that go on get the
// SMs of those that have ended.  (8 CTAs a request are slower at every size: 57.7 us
// to 32.6 for one tree, 233 to 206 for 128.)  A CTA owns a contiguous part of the
// vocabulary and each of its 8 warps a contiguous part of that, so the search at the
// end goes cluster -> CTA -> warp -> 128 tokens.  A lane keeps the row's first logits
// in shared memory between the maximum and the sum (all of a 131072-token
// vocabulary), so a row is read once, all of a lane's loads in flight.  While a row is
// summed the first child's takes its place, and that row's maximum is told with this
// row's sum: on a path along first children a step takes 8400 cycles instead of 10600.
// Maxima and sums cross the cluster through distributed shared memory, the first time
// once all of its CTAs are known to run; every CTA runs
// the children's tests itself, on the same numbers, and reaches the same verdict.
//
// Vocabulary 128256, f32: 32 trees of 24 nodes, paths up to 9 rows, 57 us (49 MB
// of visited rows, 13 % of the copy rate; 4.5 us a row of the longest path and the start); 2
// chains of 6 with draft probabilities 24 us, 8 trees of 24 with them 40 us.  Beyond 131072
// tokens rows do not fit shared memory, none is brought early and part of each is read
// twice: 32 trees at 151936 83 us, at 262144 112 us.
//
// A 64-bit conversion per logit runs at the few-per-cycle rate of the FP64 pipe
// (4 us for an eighth of a 128256-token row).  The weight is split by two f32
// fused multiply-adds rounded toward zero instead: e 2^20 + 2^23 has the upper 20
// bits in its mantissa, the remainder gives the lower 20 the same way, and lanes
// add both as 32-bit numbers.
#include "kv_common.cuh"

#include <cooperative_groups.h>

#include <new>

namespace cg = cooperative_groups;

namespace kv {

namespace {

constexpr int kCluster = 16;                // CTAs of a request
constexpr int kNodes = 256;                // of a request, that fit the shared copy
constexpr int kVerifyWarps = 8;
constexpr int kHeld = 1024;                // logits of a warp's part that are kept
constexpr int kVerifySmem = kVerifyWarps * kHeld * 4;

struct VerifyParams {
    const void *logits;
    const float *draft;
    const int32_t *tokens, *parents;
    const float *uniforms, *temperature;
    const int32_t *starts;
    int32_t *path, *count, *next;
    int64_t logits_row, draft_row, rows;
    int requests, vocab, seg;  // seg: tokens of a warp, a multiple of 4
    int vec;                   // four logits (and draft probabilities) may be loaded at once
    int ahead;                 // rows are whole in shared memory, in fours: the likeliest next one is brought early
};

// The row that the walk stands on: what its weights are made of.
struct Row {
    float inv;       // 1 / temperature
    float top;       // largest z
    int best;        // its first index, if greedy
    bool greedy;
    float per;       // f32(2^40 / W), drafts only
    float less;      // a
};

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// z of one logit: NaN counts as -inf, -0 as 0
__device__ __forceinline__ float scaled(float l, float inv) {
    const float z = __fadd_rn(__fmul_rn(l, inv), 0.0f);
    return z == z ? z : -INFINITY;
}

// e of a logit, not greedy, of a row whose largest z is not -inf
__device__ __forceinline__ float soft(const Row &r, float z) {
    return fminf(expf(z - r.top), 1.0f);  // 1 for inf - inf
}

// the same for logit i of any such row
__device__ __forceinline__ float share(const Row &r, float z, int i) {
    return r.greedy ? (i == r.best ? 1.0f : 0.0f) : soft(r, z);
}

// Whole-number weight trunc(2^40 e), 0 <= e <= 1, as 2^20 hi + lo.
struct Weight {
    uint32_t hi, lo;  // plus kWeightBias each, so that a sum can take that off once
};
constexpr uint32_t kWeightBias = 0x4B000000u;  // the bits of 2^23
__device__ __forceinline__ Weight split_weight(float e) {
    const float y = __fmaf_rz(e, 1048576.0f, 8388608.0f);
    const float r = __fmaf_rn(e, 1048576.0f, 8388608.0f - y);  // exact, in [0, 1)
    const float x = __fmaf_rz(r, 1048576.0f, 8388608.0f);
    return {__float_as_uint(y), __float_as_uint(x)};
}
__device__ __forceinline__ int64_t weight(float e) {
    const Weight w = split_weight(e);
    return (static_cast<int64_t>(w.hi - kWeightBias) << 20) + (w.lo - kWeightBias);
}

__device__ __forceinline__ float residual(const Row &r, float e, float q) {
    return fmaxf(__fsub_rn(__fmul_rn(e, r.per), __fmul_rn(r.less, q)), 0.0f);
}

// four logits as they are in memory
template <typename T>
struct Four {
    using type = uint2;
};
template <>
struct Four<float> {
    using type = float4;
};
template <typename T>
__device__ __forceinline__ void unpack4(const typename Four<T>::type &v, float (&x)[4]) {
    if constexpr (sizeof(T) == 4) {
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        union {
            uint2 u;
            T t[4];
        } y;
        y.u = v;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = to_f32(y.t[k]);
    }
}

// z of four logits, all -inf unless `in`; top becomes the largest
template <typename T>
__device__ __forceinline__ float4 scaled4(const typename Four<T>::type &v, bool in, float inv, float &top) {
    float x[4];
    unpack4<T>(v, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = in ? scaled(x[j], inv) : -INFINITY;
    top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
    return make_float4(x[0], x[1], x[2], x[3]);
}

// copies into the place that `old` was read from, after that has arrived
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t to, const void *from, const float4 &old) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES), "f"(old.x), "f"(old.y), "f"(old.z), "f"(old.w) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T>
__device__ __forceinline__ void load4(const T *p, int i, int n, bool vec, float (&x)[4], float fill) {
    if (vec && i + 4 <= n) {
        unpack4<T>(__ldg(reinterpret_cast<const typename Four<T>::type *>(p + i)), x);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = i + k < n ? to_f32(p[i + k]) : fill;
    }
}

// the cluster's barrier in two halves, for the order of execution alone
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

template <typename T, bool DRAFTS>
__global__ void __launch_bounds__(kVerifyWarps * 32, 4) q8kv_verify_kernel(const VerifyParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ float4 held[];           // [warp][kHeld / 128][lane]
    // what the CTAs tell one another: each writes to its place in everybody's copy
    __shared__ uint32_t x_max[2][kCluster];
    __shared__ int32_t x_best[2][kCluster];
    __shared__ int64_t x_sum[2][kCluster];
    __shared__ uint32_t warp_max[kVerifyWarps];
    __shared__ int32_t warp_best[kVerifyWarps];
    __shared__ int64_t warp_w[kVerifyWarps];   // sums of the warps' weights as they stand
    __shared__ int64_t cta_w[kCluster];     // and of all CTAs'
    __shared__ int32_t s_tokens[kNodes], s_parents[kNodes];
    __shared__ float s_uniforms[kNodes];
    __shared__ int verdict, child;             // of the last test

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster.block_rank());
    constexpr int ctas = kCluster;
    const int b = blockIdx.x / ctas;
    int64_t row0, row1;
    if (p.starts) {
        row0 = min(max(static_cast<int64_t>(p.starts[b]), static_cast<int64_t>(0)), p.rows);
        row1 = min(max(static_cast<int64_t>(p.starts[b + 1]), row0), p.rows);
    } else {
        row0 = p.rows / p.requests * b;
        row1 = row0 + p.rows / p.requests;
    }
    const int nodes = static_cast<int>(row1 - row0);
    if (nodes == 0) {  // the whole cluster
        if (rank == 0 && tid == 0) {
            p.count[b] = 0;
            p.next[b] = -1;
        }
        return;
    }
    // Another CTA's shared memory may be written once that CTA runs: waited for before the first exchange, behind the
    // first row's loads.
    cluster_arrive();
    bool started = false;
    const int32_t *tokens = p.tokens + row0, *parents = p.parents + row0;
    const float *uniforms = p.uniforms + row0;
    int32_t *path = p.path + row0;
    if (nodes <= kNodes) {
        for (int i = tid; i < nodes; i += kVerifyWarps * 32) {
            s_tokens[i] = tokens[i];
            s_parents[i] = parents[i];
            s_uniforms[i] = uniforms[i];
        }
        tokens = s_tokens;
        parents = s_parents;
        uniforms = s_uniforms;
    }
    __syncthreads();
    if (rank == 0)
        for (int i = tid; i < nodes; i += blockDim.x) path[i] = i == 0 ? 0 : -1;

    Row r;
    const float t = p.temperature ? p.temperature[b] : 1.0f;
    r.greedy = !(t > 0.0f);
    r.best = 0;
    r.inv = r.greedy ? 1.0f : __frcp_rn(t);
    const int seg = p.seg, chunk = seg * kVerifyWarps;
    const int64_t lo64 = static_cast<int64_t>(rank) * chunk + static_cast<int64_t>(warp) * seg;
    const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(p.vocab)));
    const int hi_end = static_cast<int>(min(lo64 + seg, static_cast<int64_t>(p.vocab)));

    int parity = 0;
    // What a step of the walk tells the cluster: the lanes' sums (then in warp_w, cta_w and the result), the warps'
    // warp_max and warp_best of a row (then in top and best), or both.
    uint32_t top_bits = 0;
    int best = 0;
    auto exchange = [&](bool sums, bool tops, int64_t mine) -> int64_t {
        if (sums) {
            mine = warp_sum(mine);
            if (lane == 0) warp_w[warp] = mine;
        }
        __syncthreads();
        if (!started) cluster_wait();
        started = true;
        if (tid < ctas) {
            if (sums) {
                int64_t s = 0;
#pragma unroll
                for (int i = 0; i < kVerifyWarps; ++i) s += warp_w[i];
                *cluster.map_shared_rank(&x_sum[parity][rank], tid) = s;
            }
            if (tops) {
                uint32_t m = warp_max[0];
                int first = r.greedy ? warp_best[0] : 0;
#pragma unroll
                for (int i = 1; i < kVerifyWarps; ++i) {
                    if (r.greedy && warp_max[i] > m) first = warp_best[i];
                    m = max(m, warp_max[i]);
                }
                *cluster.map_shared_rank(&x_max[parity][rank], tid) = m;
                if (r.greedy) *cluster.map_shared_rank(&x_best[parity][rank], tid) = first;
            }
        }
        cluster.sync();
        if (tops) {
            const uint32_t m = lane < ctas ? x_max[parity][lane] : 0;
            top_bits = __reduce_max_sync(~0u, m);
            if (r.greedy) best = __reduce_min_sync(~0u, m == top_bits ? x_best[parity][lane & (kCluster - 1)] : INT32_MAX);
        }
        int64_t s = 0;
        if (sums) {
            s = lane < ctas ? x_sum[parity][lane] : 0;
            if (tid < ctas) cta_w[tid] = s;
            __syncthreads();
            s = warp_sum(s);
        }
        parity ^= 1;
        return s;
    };

    int cur = 0, count = 0;
    int64_t total = 0;
    bool rest = false;  // drafts: the weights are the residual's
    bool ready = false; // the row is in shared memory and its maximum known
    for (;;) {
        const T *l = static_cast<const T *>(p.logits) + (row0 + cur) * p.logits_row;
        const float *q = DRAFTS ? p.draft + (row0 + cur) * p.draft_row : nullptr;
        // warp 0 looks up the first nodes after this one: those that are children, and their tokens' logits
        int child_tok = -1;
        float child_l = 0.0f, child_q = 0.0f, child_u = 0.0f;
        if (warp == 0) {
            const int node = cur + 1 + lane;
            const bool is_child = node < nodes && parents[node] == cur;
            const int tok = is_child ? tokens[node] : -1;
            if (tok >= 0 && tok < p.vocab) {
                child_tok = tok;
                child_l = to_f32(l[tok]);
                child_u = uniforms[node];
                if (DRAFTS) child_q = q[tok];
            }
        }
        float4 *mine = held + warp * (kHeld / 4) + lane;
        const int held_end = min(hi_end, lo + kHeld);
        // the warp's largest of a row whose lanes have `top`: and, if greedy, the first index that has it
        auto peak = [&](float top, const T *row) {
            const uint32_t most = __reduce_max_sync(~0u, ordered(top));
            if (lane == 0) warp_max[warp] = most;
            if (r.greedy) {
                int first = INT32_MAX;
                for (int i = lo; i < hi_end && first == INT32_MAX; i += 128) {
                    float x[4];
                    if (i < held_end) {
                        const float4 v = mine[(i - lo) / 4];
                        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
                    } else {
                        load4(row, i + lane * 4, hi_end, p.vec, x, -INFINITY);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = scaled(x[j], r.inv);
                    }
#pragma unroll
                    for (int j = 3; j >= 0; --j)
                        if (i + lane * 4 + j < hi_end && ordered(x[j]) == most) first = i + lane * 4 + j;
                }
                first = __reduce_min_sync(~0u, first);
                if (lane == 0) warp_best[warp] = first;
            }
        };
        if (!ready) {  // ---- the row's maximum
            float top = -INFINITY;
            auto look = [&](int i) -> float4 {
                float x[4];
                load4(l, i, hi_end, p.vec, x, -INFINITY);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = scaled(x[j], r.inv);
                top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
                return make_float4(x[0], x[1], x[2], x[3]);
            };
            if (p.vec && ((held_end - lo) & 3) == 0) {
                // all of the lane's loads at once: with a test for the row's end at each they would follow one another
                using V = typename Four<T>::type;
                V v[kHeld / 128];
#pragma unroll
                for (int k = 0; k < kHeld / 128; ++k) {
                    const int i = lo + 128 * k + 4 * lane;
                    if (i < held_end) v[k] = __ldg(reinterpret_cast<const V *>(l + i));
                }
#pragma unroll
                for (int k = 0; k < kHeld / 128; ++k) {
                    if (lo + 128 * k >= held_end) break;
                    mine[32 * k] = scaled4<T>(v[k], lo + 128 * k + 4 * lane < held_end, r.inv, top);
                }
            } else {
                for (int i = lo; i < held_end; i += 128) mine[(i - lo) / 4] = look(i + lane * 4);
            }
#pragma unroll 4
            for (int i = lo + kHeld; i < hi_end; i += 128) look(i + lane * 4);
            peak(top, l);
            exchange(false, true, 0);
            r.top = unordered(top_bits);
            r.best = best;
        }
        // ---- the row of the first child, the likeliest to be next, takes this row's place as that is summed, and its
        // maximum is found and told along with the sum: on a path along first children a step has one exchange and
        // waits for no row.  L2 starts on it now.
        const uint32_t kids = __ballot_sync(~0u, cur + 1 + lane < nodes && parents[cur + 1 + lane] == cur);
        const int next = p.ahead && kids != 0 ? cur + __ffs(kids) : -1;
        const T *next_l = static_cast<const T *>(p.logits) + (row0 + cur + __ffs(kids)) * p.logits_row;
        if (kids != 0) {
            constexpr int kLine = 128 / sizeof(T);
            for (int i = lo + lane * kLine; i < held_end; i += 32 * kLine) asm volatile("prefetch.global.L2 [%0];" ::"l"(next_l + i));
        }
        r.less = 0.0f;

        // sum of the lane's weights (of the residual's once `rest`): at most 2^10 logits a lane, so 32 bits a half
        // `fresh`: of a row that is in shared memory, and leaves it for the next one
        auto sum = [&](bool fresh) -> int64_t {
            const bool leaves = fresh && next >= 0;
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
            if (r.greedy || r.top == -INFINITY) {
                if (leaves)
                    for (int i = lo; i < hi_end; i += 128)
                        if (i + 4 * lane < hi_end) cp_async<4 * sizeof(T)>(to + 4 * (i - lo), next_l + i + 4 * lane, mine[(i - lo) / 4]);
                // one logit has all the weight
                if (r.top == -INFINITY || lane != 0 || r.best < lo || r.best >= hi_end) return 0;
                return weight(DRAFTS && rest ? residual(r, 1.0f, q[r.best]) : 1.0f);
            }
            const uint32_t n = 4 * static_cast<uint32_t>((hi_end - lo + 127) / 128);  // weights that the lane adds
            uint32_t hi = 0 - n * kWeightBias, lo_bits = hi;
            auto add = [&](const float4 &v, int i) {
                const float x[4] = {v.x, v.y, v.z, v.w};
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (DRAFTS && rest) load4(q, i + lane * 4, hi_end, p.vec, y, 0.0f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = soft(r, x[j]);  // 0 past the warp's end, where z is -inf
                    const Weight w = split_weight(DRAFTS && rest ? residual(r, e, y[j]) : e);
                    hi += w.hi;
                    lo_bits += w.lo;
                }
            };
            if (fresh) {
#pragma unroll 4
                for (int i = lo; i < held_end; i += 128) {
                    const float4 v = mine[(i - lo) / 4];
                    add(v, i);
                    if (leaves && i + 4 * lane < hi_end) cp_async<4 * sizeof(T)>(to + 4 * (i - lo), next_l + i + 4 * lane, v);
                }
            }
            for (int i = fresh ? lo + kHeld : lo; i < hi_end; i += 128) {
                float x[4];
                load4(l, i + lane * 4, hi_end, p.vec, x, -INFINITY);
                add(make_float4(scaled(x[0], r.inv), scaled(x[1], r.inv), scaled(x[2], r.inv), scaled(x[3], r.inv)), i);
            }
            return (static_cast<int64_t>(hi) << 20) + lo_bits;
        };
        rest = false;
        {
            const int64_t w = sum(true);
            if (next >= 0) {
                cp_async_wait();  // the lane's own
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kHeld / 128; ++k) {
                    if (lo + 128 * k >= hi_end) break;
                    mine[32 * k] = scaled4<T>(*reinterpret_cast<const typename Four<T>::type *>(mine + 32 * k),
                                               lo + 128 * k + 4 * lane < hi_end, r.inv, top);
                }
                peak(top, next_l);
            }
            total = exchange(true, next >= 0, w);
        }
        if (DRAFTS) r.per = static_cast<float>(1099511627776.0 / static_cast<double>(total));

        // ---- the children, in index order.  Warp 0 tests until one is accepted (verdict 1), none is
        // left (0) or, with draft probabilities, one is refused (2)
        float norm = 1.0f;
        int from = cur + 1;
        bool open = true;
        for (;;) {
            if (warp == 0) {
                int said = 0, who = nodes;
                for (int i0 = from; i0 < nodes && said == 0 && open && total > 0; i0 += 32) {
                    // every lane looks up its node's token; then they are tested in order
                    int tok = child_tok;
                    float lx = child_l, qx = child_q, u = child_u;
                    if (i0 != cur + 1) {
                        const int node = i0 + lane;
                        tok = node < nodes && parents[node] == cur ? tokens[node] : -1;
                        if (tok < 0 || tok >= p.vocab) tok = -1;
                        lx = tok >= 0 ? to_f32(l[tok]) : 0.0f;
                        u = tok >= 0 ? uniforms[node] : 0.0f;
                        qx = DRAFTS && tok >= 0 ? q[tok] : 0.0f;
                    }
                    const bool valid = tok >= 0;
                    const float e = valid ? share(r, scaled(lx, r.inv), tok) : 0.0f;
                    int64_t wx = weight(e);
                    if (!DRAFTS) {
                        // a sibling before with the same token was refused when this one is tested: its weight is gone
                        bool twin = (__match_any_sync(~0u, valid ? tok : -1 - lane) & ((1u << lane) - 1u)) != 0;
                        for (int j = cur + 1; j < i0; ++j) twin |= parents[j] == cur && tokens[j] == tok;
                        if (twin) wx = 0;
                    }
                    uint32_t todo = __ballot_sync(~0u, valid);  // an invalid token has no weight and was never drawn
                    while (todo != 0 && said == 0) {
                        const int at = __ffs(todo) - 1;
                        todo &= todo - 1;
                        bool ok;
                        if constexpr (DRAFTS) {
                            ok = __fmul_rn(__fmul_rn(u, qx), norm) < residual(r, e, qx);
                        } else {
                            ok = static_cast<double>(u) * static_cast<double>(total) < static_cast<double>(wx);
                        }
                        ok = __shfl_sync(~0u, ok, at);
                        if (ok || DRAFTS) {
                            who = i0 + at;
                            said = ok ? 1 : 2;
                        } else {
                            total -= __shfl_sync(~0u, wx, at);
                            if (lane == at) {
                                cta_w[tok / chunk] -= wx;
                                if (tok / chunk == rank) warp_w[tok % chunk / seg] -= wx;
                            }
                            __syncwarp();  // the next one's lane may change the same words
                        }
                    }
                }
                if (lane == 0) {
                    verdict = said;
                    child = who;
                }
            }
            __syncthreads();
            const int said = verdict, who = child;
            __syncthreads();
            if (!DRAFTS || said != 2) {
                if (said == 1) {
                    cur = who;
                    ready = who == next;
                    if (ready) {
                        r.top = unordered(top_bits);
                        r.best = best;
                    }
                    ++count;
                    if (rank == 0 && tid == 0) path[count] = who;
                }
                open = said == 1;  // goes on with the accepted child's row
                break;
            }
            // refused: take the draft's share out, once more
            r.less = __fadd_rn(r.less, norm);
            rest = true;
            const int64_t left = exchange(true, false, sum(false));
            from = who + 1;
            if (left == 0) {
                // nothing is left: the target's own weights, and no other child
                rest = false;
                r.less = 0.0f;
                total = exchange(true, false, sum(false));
                open = false;
            } else {
                total = left;
                norm = static_cast<float>(static_cast<double>(left) * (1.0 / 1099511627776.0));
            }
        }
        if (open) continue;

        // ---- the next token: the first whose prefix sum exceeds the target
        __syncthreads();
        total = 0;
        for (int i = 0; i < ctas; ++i) total += cta_w[i];
        if (total == 0) {
            if (rank == 0 && tid == 0) p.next[b] = -1;
        } else {
            int64_t want = __double2ll_rz(static_cast<double>(uniforms[0]) * static_cast<double>(total));
            want = max(static_cast<int64_t>(0), min(want, total - 1));
            int owner = 0;
            while (owner < ctas - 1 && want >= cta_w[owner]) want -= cta_w[owner++];
            if (owner == rank) {
                int ow = 0;
                while (ow < kVerifyWarps - 1 && want >= warp_w[ow]) want -= warp_w[ow++];
                if (ow == warp) {
                    for (int i = lo + lane * 4;; i += 128) {  // ends: the warp's weights exceed `want`
                        float x[4], y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        int64_t w[4];
                        load4(l, i, hi_end, p.vec, x, -INFINITY);
                        if (DRAFTS && rest) load4(q, i, hi_end, p.vec, y, 0.0f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float e = share(r, scaled(x[j], r.inv), i + j < hi_end ? i + j : -1);
                            w[j] = weight(DRAFTS && rest ? residual(r, e, y[j]) : e);
                        }
                        if (!DRAFTS) {
                            // refused children have no weight
                            for (int j0 = cur + 1; j0 < nodes; j0 += 32) {
                                const bool is_child = j0 + lane < nodes && parents[j0 + lane] == cur;
                                const int tok = is_child ? tokens[j0 + lane] : -1;
                                uint32_t todo = __ballot_sync(~0u, is_child);
                                while (todo != 0) {
                                    const int x0 = __shfl_sync(~0u, tok, __ffs(todo) - 1);
                                    todo &= todo - 1;
#pragma unroll
                                    for (int j = 0; j < 4; ++j) w[j] = i + j == x0 ? 0 : w[j];
                                }
                            }
                        }
                        const int64_t mine = w[0] + w[1] + w[2] + w[3];
                        int64_t upto = mine;
#pragma unroll
                        for (int d = 1; d < 32; d *= 2) {
                            const int64_t a = __shfl_up_sync(~0u, upto, d);
                            if (lane >= d) upto += a;
                        }
                        const uint32_t over = __ballot_sync(~0u, upto > want);
                        if (over != 0) {
                            if (lane == __ffs(over) - 1) {
                                int64_t at = upto - mine;
                                int j = 0;
                                while (j < 3 && at + w[j] <= want) at += w[j++];
                                p.next[b] = i + j;
                            }
                            break;
                        }
                        want -= __shfl_sync(~0u, upto, 31);
                        if (i - lane * 4 + 128 >= hi_end) break;  // not reached: the sums are exact
                    }
                }
            }
        }
        if (rank == 0 && tid == 0) p.count[b] = count;
        break;
    }
    cluster.sync();  // no CTA leaves while another may read its shared memory
}

template <typename T>
cudaError_t launch(const VerifyParams &p, cudaStream_t stream) {
    auto *fn = p.draft ? q8kv_verify_kernel<T, true> : q8kv_verify_kernel<T, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.requests) * kCluster);
    cfg.blockDim = dim3(kVerifyWarps * 32);
    cfg.dynamicSmemBytes = kVerifySmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

// Clusters of 16 are beyond the size that every GPU takes: allowed per kernel, when a plan is made.
template <typename T>
cudaError_t allow_clusters() {
    cudaError_t e = cudaSuccess;
    for (auto *fn : {q8kv_verify_kernel<T, true>, q8kv_verify_kernel<T, false>}) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kVerifySmem);
    }
    return e;
}

}  // namespace

}  // namespace kv

struct q8kv_verify_s {
    int device = 0;
    int max_requests = 0, vocab = 0;
    int64_t max_rows = 0;
};

extern "C" {

q8mv_status_t q8kv_verify_plan(q8kv_verify_plan_t *out, int32_t max_requests, int64_t max_rows, int32_t vocab,
                               int device) {
    if (out == nullptr) return Q8MV_ERR_INVALID_ARG;
    *out = nullptr;
    if (max_requests < 1 || max_requests > 65535 || max_rows < 1 || max_rows > (1 << 20) || vocab < 1 ||
        vocab > (1 << 22))
        return Q8MV_ERR_INVALID_ARG;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(device);
    if (st != Q8MV_OK) return st;
    q8kv_verify_s *p = new (std::nothrow) q8kv_verify_s();
    if (p == nullptr) return Q8MV_ERR_OUT_OF_MEMORY;
    p->device = scope.device();
    p->max_requests = max_requests;
    p->max_rows = max_rows;
    p->vocab = vocab;
    cudaError_t e = kv::allow_clusters<float>();
    if (e == cudaSuccess) e = kv::allow_clusters<__half>();
    if (e == cudaSuccess) e = kv::allow_clusters<__nv_bfloat16>();
    if (e != cudaSuccess) {
        delete p;
        return q8i::cuda_status(e);
    }
    *out = p;
    return Q8MV_OK;
}

q8mv_status_t q8kv_verify(q8kv_verify_plan_t plan, const q8kv_verify_args_t *a, cudaStream_t stream) {
    if (plan == nullptr || a == nullptr) return Q8MV_ERR_INVALID_ARG;
    if (a->reserved != 0 || !kv::valid_type(a->type) || a->vocab != plan->vocab) return Q8MV_ERR_INVALID_ARG;
    if (a->requests < 0 || a->requests > plan->max_requests || a->rows < 0 || a->rows > plan->max_rows)
        return Q8MV_ERR_INVALID_ARG;
    const int64_t most = 1LL << 40;
    if (a->logits_row < 0 || a->logits_row > most || a->draft_row < 0 || a->draft_row > most)
        return Q8MV_ERR_INVALID_ARG;
    if (a->requests == 0) return Q8MV_OK;
    if (a->starts == nullptr && a->rows % a->requests != 0) return Q8MV_ERR_INVALID_ARG;
    if (!a->count || !a->next_token) return Q8MV_ERR_INVALID_ARG;
    const int size = kv::type_size(a->type);
    if (a->rows > 0) {
        if (!a->logits || !a->tokens || !a->parents || !a->uniforms || !a->path) return Q8MV_ERR_INVALID_ARG;
        if (!kv::aligned(a->logits, size)) return Q8MV_ERR_INVALID_ARG;
    }
    if (!kv::aligned(a->draft_probs, 4) || !kv::aligned(a->tokens, 4) || !kv::aligned(a->parents, 4) ||
        !kv::aligned(a->uniforms, 4) || !kv::aligned(a->temperature, 4) || !kv::aligned(a->starts, 4) ||
        !kv::aligned(a->path, 4) || !kv::aligned(a->count, 4) || !kv::aligned(a->next_token, 4))
        return Q8MV_ERR_INVALID_ARG;
    // every CTA of a cluster decides from the inputs: none of them may be written meanwhile
    {
        const int64_t R = a->rows, B = a->requests;
        const kv::Range in[] = {
            {a->logits, R > 0 ? ((R - 1) * a->logits_row + a->vocab) * size : 0},
            {a->draft_probs, a->draft_probs && R > 0 ? ((R - 1) * a->draft_row + a->vocab) * 4 : 0},
            {a->tokens, 4 * R}, {a->parents, 4 * R}, {a->uniforms, 4 * R},
            {a->temperature, a->temperature ? 4 * B : 0}, {a->starts, a->starts ? 4 * (B + 1) : 0}};
        const kv::Range outs[] = {{a->path, 4 * R}, {a->count, 4 * B}, {a->next_token, 4 * B}};
        for (int i = 0; i < 3; ++i) {
            for (const kv::Range &x : in)
                if (kv::overlap(outs[i], x)) return Q8MV_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if (kv::overlap(outs[i], outs[j])) return Q8MV_ERR_INVALID_ARG;
        }
    }
    kv::VerifyParams p = {};
    p.logits = a->logits;
    p.draft = a->draft_probs;
    p.tokens = a->tokens;
    p.parents = a->parents;
    p.uniforms = a->uniforms;
    p.temperature = a->temperature;
    p.starts = a->starts;
    p.path = a->path;
    p.count = a->count;
    p.next = a->next_token;
    p.logits_row = a->logits_row;
    p.draft_row = a->draft_row;
    p.rows = a->rows;
    p.requests = a->requests;
    p.vocab = a->vocab;
    constexpr int parts = kv::kCluster * kv::kVerifyWarps;
    p.seg = static_cast<int>(kv::ceil_div(kv::ceil_div(a->vocab, parts), 4) * 4);
    p.vec = kv::aligned(a->logits, 4 * size) && a->logits_row % 4 == 0 && kv::aligned(a->draft_probs, 16) &&
            a->draft_row % 4 == 0;
    p.ahead = p.vec && p.seg <= kv::kHeld && a->vocab % 4 == 0;
    cudaError_t e;
    if (a->type == Q8KV_F32)
        e = kv::launch<float>(p, stream);
    else if (a->type == Q8KV_F16)
        e = kv::launch<__half>(p, stream);
    else
        e = kv::launch<__nv_bfloat16>(p, stream);
    return q8i::cuda_status(e);
}

q8mv_status_t q8kv_verify_destroy(q8kv_verify_plan_t p) {
    if (p == nullptr) return Q8MV_OK;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(p->device);
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceSynchronize());
    delete p;
    return st;
}

}  // extern "C"
