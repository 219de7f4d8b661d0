// Writing, reading and moving rows of the Q8_0 cache (../../include/q8kv.h), and
// the device check of the q8kv plans.
//
// All three are streams without reuse, bound by HBM for many rows and by one
// round trip for few.  Every lane handles 16 bytes of the wide side (8 16-bit
// elements or 4 f32), so its loads or stores are one full vector and a warp's
// are contiguous; a 32-element block is then 4 or 8 neighbouring lanes and its
// amax takes 2 or 3 shuffles.  Keys and values of the same place are handled by
// the same lane, which keeps two independent loads in flight.  A large write has
// to be short of instructions too (a kernel with 20 an element took 50 us where
// this one takes 38).
//
// 8190 tokens of 32 heads x 128, bf16: written in 37.7 us, read in 34.2 us (5.6 and
// 6.1 TB/s, 82 and 90 % of the copy rate; a write issues in 0.73 of the cycles, 15
// instructions an element).  32768 tokens of 8 heads read: 35.0 us (5.9 TB/s).  64
// requests' 9 rows of 256 heads moved from anywhere to anywhere: 29 us (85 MB, 2.9 TB/s:
// rows of 128 and 16 bytes, 2 KB apart, of which DRAM moves 64 at a time, which is 20
// us; neither more blocks an SM nor more rows in flight change the rest, the loads'
// latency), up a path as a verification leaves them 15 us.  A few rows: 2.1, 2.5 and 3.5
// us.
#include "kv_common.cuh"

namespace kv {

namespace {

// Tokens a lane takes of a large call, for loads in flight.  8190 tokens of 32 heads x 128 bf16 written: 44.7, 39.3,
// 37.7 us with 1, 2, 4; read: 39.6, 34.2, 34.6, 34.8 with 1, 2, 4, 8; 32768 tokens of 8 heads read: 41.6, 35.0, 35.5,
// 35.8.  A call that leaves less than four blocks an SM with that takes one a lane: 8 tokens of 8 heads, written and
// read, 4.1 us, and 6.0 with several.
constexpr int kManyBlocks = 152 * 4;
constexpr int kWriteTokens = 4, kReadTokens = 2;

struct IoParams {
    Cache c;
    const void *in[2];   // k, v (write)
    void *out[2];        // k, v (read)
    int64_t row[2];      // strides of `in`, in elements
    int64_t head[2];
    const int64_t *slots;
    int64_t n;
    int lanes;           // lanes of one token: heads * blocks * (32 / E)
};

// The place of token slot s, or false if it is outside the cache.
__device__ __forceinline__ bool place_of(const Cache &c, int64_t slot, int64_t *page, int *place) {
    if (slot < 0 || slot >= c.slots) return false;
    if ((slot >> 32) == 0) {  // the usual case, without a 64-bit division
        const uint32_t s = static_cast<uint32_t>(slot), p = s / static_cast<uint32_t>(c.page_size);
        *page = p;
        *place = static_cast<int>(s - p * static_cast<uint32_t>(c.page_size));
    } else {
        *page = slot / c.page_size;
        *place = static_cast<int>(slot - *page * c.page_size);
    }
    return true;
}

// 16 bytes of T as they are in memory
template <typename T>
union Piece {
    uint4 v;
    T t[16 / sizeof(T)];
};

template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_piece(const T *p) {
    Piece<T> x;
    if constexpr (VEC) {
        x.v = __ldg(reinterpret_cast<const uint4 *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) x.t[i] = p[i];
    }
    return x.v;
}

// Four codes rint(x * id).  Usually x * id is within +-127.5 and the sum with
// 1.5 * 2^23 leaves it, rounded to even, in the low byte; a conversion would run at
// an eighth of that rate.
__device__ __forceinline__ uint32_t pack4(const float *x, float id) {
    constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], id), kRound));
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040u), __byte_perm(c[2], c[3], 0x0040u), 0x5410u);
}

// The same for blocks with NaN (0), infinities or an overflowing 127 (1 / amax).
__device__ __noinline__ uint32_t pack4_any(float x0, float x1, float x2, float x3, float id) {
    const float x[4] = {x0, x1, x2, x3};
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i) {
        const int c = max(-127, min(127, __float2int_rn(__fmul_rn(x[i], id))));  // NaN becomes 0
        w |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * i);
    }
    return w;
}

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The largest |x| of a lane's elements, NaN if one is: 16-bit types in pairs.
__device__ __forceinline__ float amax_of(const Piece<float> &x) {
    return max_nan(max_nan(fabsf(x.t[0]), fabsf(x.t[1])), max_nan(fabsf(x.t[2]), fabsf(x.t[3])));
}
template <typename T2, typename P>
__device__ __forceinline__ float amax_of_pairs(const P &x) {
    const T2 *p = reinterpret_cast<const T2 *>(x.t);
    const T2 m = __hmax2_nan(__hmax2_nan(__habs2(p[0]), __habs2(p[1])), __hmax2_nan(__habs2(p[2]), __habs2(p[3])));
    return max_nan(to_f32(m.x), to_f32(m.y));
}
__device__ __forceinline__ float amax_of(const Piece<__half> &x) { return amax_of_pairs<__half2>(x); }
__device__ __forceinline__ float amax_of(const Piece<__nv_bfloat16> &x) { return amax_of_pairs<__nv_bfloat162>(x); }

// Row of head 0 for each of the block's tokens, -1 if there is none: one thread a token does the divisions.
template <int U>
__device__ __forceinline__ void find_rows(const IoParams &p, int64_t (&rows)[8 * U]) {
    const int t = threadIdx.y * blockDim.x + threadIdx.x;
    if (t < static_cast<int>(blockDim.y) * U) {
        const int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.y * U) + t;
        int64_t page;
        int place;
        rows[t] = i < p.n && place_of(p.c, __ldg(p.slots + i), &page, &place) ? row_of(p.c, page, 0, place) : -1;
    }
}

// d = amax / 127, c = rint(x * (127 * (1 / amax))), every step rounded.
// U tokens a lane: their loads, which do not wait for the slots, are all in flight.
// For many rows the issue slots bound it, next to HBM: a warp stays together
// (shuffles of all lanes, one vote for blocks that are not ordinary), 16-bit
// elements are compared in pairs and a NaN shows in the maximum.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(256) q8kv_write_kernel(const IoParams p) {
    constexpr int E = 16 / sizeof(T), PER = 32 / E;  // elements a lane, lanes a block
    __shared__ int64_t rows[8 * U];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (blockDim.y * U) + threadIdx.y;
    const int at = blockIdx.y * blockDim.x + threadIdx.x;
    const int per_head = p.c.blocks * PER;
    const int h = at / per_head, in_row = at - h * per_head, e0 = in_row * E, b = in_row / PER;
    const bool live = at < p.lanes && e0 < p.c.dim;
    Piece<T> raw[U][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const T *src = static_cast<const T *>(p.in[s]) + first * p.row[s] + h * p.head[s] + e0;
        const int64_t step = static_cast<int64_t>(blockDim.y) * p.row[s];
#pragma unroll
        for (int u = 0; u < U; ++u)
            raw[u][s].v = live && first + u * blockDim.y < p.n ? load_piece<T, VEC>(src + u * step) : make_uint4(0, 0, 0, 0);
    }
    find_rows<U>(p, rows);
    __syncthreads();
    const int lane = threadIdx.x & 31, of = lane & (PER - 1), first_lane = lane - of;  // (blockDim.x: whole warps)
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r0 = rows[u * blockDim.y + threadIdx.y];
        const int64_t r = r0 + h * p.c.stride_head;
        const bool there = live && r0 >= 0;
        float amax[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            amax[s] = amax_of(raw[u][s]);
#pragma unroll
            for (int d = 1; d < PER; d *= 2) amax[s] = max_nan(amax[s], __shfl_xor_sync(~0u, amax[s], d));
        }
        const bool nan = amax[0] != amax[0] || amax[1] != amax[1];
        if (__any_sync(~0u, nan)) {  // the largest of those that are numbers
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                amax[s] = 0.0f;
#pragma unroll
                for (int j = 0; j < E; ++j) amax[s] = fmaxf(amax[s], fabsf(to_f32(raw[u][s].t[j])));
#pragma unroll
                for (int d = 1; d < PER; d *= 2) amax[s] = fmaxf(amax[s], __shfl_xor_sync(~0u, amax[s], d));
            }
        }
        // the block's four divisions, one in each of its first four lanes: 1 / amax and amax / 127 of k, then of v
        const float a = of & 2 ? amax[1] : amax[0], num = of & 1 ? a : 1.0f, den = of & 1 ? 127.0f : a;
        float ratio = den > 0.0f ? __fdiv_rn(num, den) : 0.0f;
        if (!(of & 1)) ratio = __fmul_rn(127.0f, ratio);
        const float id[2] = {__shfl_sync(~0u, ratio, first_lane), __shfl_sync(~0u, ratio, first_lane + 2)};
        const bool usual = !nan && amax[0] < INFINITY && amax[1] < INFINITY && id[0] < INFINITY && id[1] < INFINITY;
        uint32_t w[2][E / 4];
        if (__all_sync(~0u, usual)) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < E / 4; ++j) {
                    const T *t = raw[u][s].t + 4 * j;
                    const float x[4] = {to_f32(t[0]), to_f32(t[1]), to_f32(t[2]), to_f32(t[3])};
                    w[s][j] = pack4(x, id[s]);
                }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < E / 4; ++j) {
                    const T *t = raw[u][s].t + 4 * j;
                    w[s][j] = pack4_any(to_f32(t[0]), to_f32(t[1]), to_f32(t[2]), to_f32(t[3]), id[s]);
                }
        }
        if (there) {
            const int64_t at_code = r * p.c.dim + e0;
            if constexpr (E == 8) {
                *reinterpret_cast<uint2 *>(p.c.k_codes + at_code) = make_uint2(w[0][0], w[0][1]);
                *reinterpret_cast<uint2 *>(p.c.v_codes + at_code) = make_uint2(w[1][0], w[1][1]);
            } else {
                *reinterpret_cast<uint32_t *>(p.c.k_codes + at_code) = w[0][0];
                *reinterpret_cast<uint32_t *>(p.c.v_codes + at_code) = w[1][0];
            }
        }
        if (r0 >= 0 && at < p.lanes && (of & 1)) {
            if (of == 1) p.c.k_scales[r * p.c.blocks + b] = ratio;
            if (of == 3) p.c.v_scales[r * p.c.blocks + b] = ratio;
        }
    }
}

template <typename T, int U>
__global__ void __launch_bounds__(256) q8kv_read_kernel(const IoParams p) {
    constexpr int E = 16 / sizeof(T);
    __shared__ int64_t rows[8 * U];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (blockDim.y * U) + threadIdx.y;
    const int at = blockIdx.y * blockDim.x + threadIdx.x;
    find_rows<U>(p, rows);
    __syncthreads();
    if (at >= p.lanes) return;
    const int per_head = p.c.dim / E;
    const int h = at / per_head, e0 = (at - h * per_head) * E, b = e0 / 32;
    uint32_t w[U][2][E / 4] = {};
    float d[U][2] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r0 = rows[u * blockDim.y + threadIdx.y];
        if (r0 >= 0) {
            const int64_t r = r0 + h * p.c.stride_head;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int8_t *codes = (s == 0 ? p.c.k_codes : p.c.v_codes) + r * p.c.dim + e0;
                if constexpr (E == 8) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(codes);
                    w[u][s][0] = v.x;
                    w[u][s][1] = v.y;
                } else {
                    w[u][s][0] = *reinterpret_cast<const uint32_t *>(codes);
                }
                d[u][s] = ((s == 0 ? p.c.k_scales : p.c.v_scales) + r * p.c.blocks)[b];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * blockDim.y;
        if (i >= p.n) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Piece<T> x;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = static_cast<int8_t>(w[u][s][j / 4] >> (8 * (j % 4)));
                x.t[j] = from_f32<T>(__fmul_rn(static_cast<float>(c), d[u][s]));
            }
            T *out = static_cast<T *>(p.out[s]) + (i * p.c.heads + h) * p.c.dim + e0;
            *reinterpret_cast<uint4 *>(out) = x.v;
        }
    }
}

struct MoveParams {
    Cache c;
    const int64_t *src, *dst;
    int path;
    int scale_pieces;  // of one row and array: blocks / 4 of 16 bytes, or `blocks` of 4
    int lanes;         // of one token: heads * 2 * (dim / 16 + scale_pieces)
};

constexpr int kMoveBatch = 8, kMovePairs = 32;

// V bytes of every row of a request, pairs g .. g + kMoveBatch - 1: all loaded before any is stored, unless one of them
// is read by a later one.
template <typename V>
__device__ __forceinline__ void move_batch(char *base, int64_t pitch, const int64_t *from, const int64_t *to, bool meet) {
    if (!meet) {
        V v[kMoveBatch];
#pragma unroll
        for (int i = 0; i < kMoveBatch; ++i)
            if (from[i] >= 0) v[i] = *reinterpret_cast<const V *>(base + from[i] * pitch);
#pragma unroll
        for (int i = 0; i < kMoveBatch; ++i)
            if (from[i] >= 0) *reinterpret_cast<V *>(base + to[i] * pitch) = v[i];
    } else {
        for (int i = 0; i < kMoveBatch; ++i)
            if (from[i] >= 0) *reinterpret_cast<V *>(base + to[i] * pitch) = *reinterpret_cast<const V *>(base + from[i] * pitch);
    }
}

// One lane owns one 16-byte piece of codes or of scales (one scale, where a row's
// are not whole pieces) of every row that its request moves, so the order of a request's pairs is the lane's own program
// order and needs no barrier.  Eight pairs are loaded before any is stored,
// unless one of them is read by a later one of the eight.  The pairs' rows are
// found once per block, 32 at a time.
__global__ void __launch_bounds__(256, 3) q8kv_move_kernel(const MoveParams p) {
    __shared__ int64_t from[kMovePairs], to[kMovePairs];  // of head 0; -1: the pair is skipped
    __shared__ int meets[kMovePairs / kMoveBatch];
    const int64_t *src = p.src + static_cast<int64_t>(blockIdx.y) * p.path;
    const int64_t *dst = p.dst + static_cast<int64_t>(blockIdx.y) * p.path;
    const int at = blockIdx.x * blockDim.x + threadIdx.x;
    const int pieces = p.c.dim / 16, scales = p.scale_pieces, per_head = 2 * (pieces + scales);
    const bool mine = at < p.lanes;
    const int h = mine ? at / per_head : 0, in = mine ? at - h * per_head : 0;
    const bool wide = in < 2 * pieces || scales < p.c.blocks;
    // address of the lane's piece in row 0 of its head, and the bytes of one row of its array
    char *base;
    int64_t pitch;
    if (in < 2 * pieces) {
        base = reinterpret_cast<char *>(in < pieces ? p.c.k_codes : p.c.v_codes) + (in < pieces ? in : in - pieces) * 16;
        pitch = p.c.dim;
    } else {
        const int s = in - 2 * pieces;
        base = reinterpret_cast<char *>(s < scales ? p.c.k_scales : p.c.v_scales) + (s < scales ? s : s - scales) * (wide ? 16 : 4);
        pitch = 4LL * p.c.blocks;
    }
    base += h * p.c.stride_head * pitch;
    for (int i0 = 0; i0 < p.path; i0 += kMovePairs) {
        const int n = min(kMovePairs, p.path - i0);
        __syncthreads();
        if (threadIdx.x < kMovePairs) {  // one warp
            const int i = threadIdx.x;
            int64_t page, f = -1, t = -1;
            int place;
            if (i < n && place_of(p.c, dst[i0 + i], &page, &place)) {
                t = row_of(p.c, page, 0, place);
                if (place_of(p.c, src[i0 + i], &page, &place)) f = row_of(p.c, page, 0, place);
            }
            from[i] = f;
            to[i] = f >= 0 ? t : -1;
            __syncwarp();
            bool meet = false;
            for (int j = i & ~(kMoveBatch - 1); j < i; ++j) meet |= f >= 0 && f == to[j];
            const unsigned any = __ballot_sync(~0u, meet);
            if (i < kMovePairs / kMoveBatch) meets[i] = (any >> (i * kMoveBatch)) & ((1u << kMoveBatch) - 1u);
        }
        __syncthreads();
        if (!mine) continue;
        for (int g = 0; g < n; g += kMoveBatch) {
            const bool meet = meets[g / kMoveBatch] != 0;
            if (wide)
                move_batch<uint4>(base, pitch, from + g, to + g, meet);
            else
                move_batch<float>(base, pitch, from + g, to + g, meet);
        }
    }
}

// Threads of one token along x (a multiple of 32, at most 256), tokens along y.
// `tokens` tokens a thread once that leaves several blocks an SM, else one.
struct Shape {
    dim3 grid, block;
    bool many;
};

Shape shape(int lanes, int64_t n, int tokens) {
    const unsigned x = lanes >= 256 ? 256u : static_cast<unsigned>((lanes + 31) / 32 * 32);
    const unsigned y = 256u / x;
    Shape s;
    s.block = dim3(x, y);
    const int64_t across = ceil_div(lanes, x);
    s.many = ceil_div(n, tokens * y) * across >= kManyBlocks;
    s.grid = dim3(static_cast<unsigned>(ceil_div(n, s.many ? tokens * y : y)), static_cast<unsigned>(across));
    return s;
}

template <typename T>
void launch_write(const IoParams &p, bool vec, const Shape &s, cudaStream_t stream) {
    if (!vec)
        q8kv_write_kernel<T, false, 1><<<s.grid, s.block, 0, stream>>>(p);
    else if (s.many)
        q8kv_write_kernel<T, true, kWriteTokens><<<s.grid, s.block, 0, stream>>>(p);
    else
        q8kv_write_kernel<T, true, 1><<<s.grid, s.block, 0, stream>>>(p);
}

template <typename T>
void launch_read(const IoParams &p, const Shape &s, cudaStream_t stream) {
    if (s.many)
        q8kv_read_kernel<T, kReadTokens><<<s.grid, s.block, 0, stream>>>(p);
    else
        q8kv_read_kernel<T, 1><<<s.grid, s.block, 0, stream>>>(p);
}

bool valid_stride(int64_t s) { return s >= 0 && s < (1LL << 40); }

}  // namespace

q8mv_status_t DeviceScope::enter(int device) {
    q8mv_status_t st = q8i::cuda_status(cudaGetDevice(&prev_));
    if (st != Q8MV_OK) return st;
    device_ = device < 0 ? prev_ : device;
    int count = 0, major = 0, minor = 0;
    st = q8i::cuda_status(cudaGetDeviceCount(&count));
    if (st != Q8MV_OK) return st;
    if (device_ >= count) {
        device_ = prev_;
        return Q8MV_ERR_INVALID_ARG;
    }
    st = q8i::cuda_status(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device_));
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device_));
    if (st == Q8MV_OK && (major != 10 || minor != 3)) st = Q8MV_ERR_UNSUPPORTED_DEVICE;
    if (st == Q8MV_OK && device_ != prev_) st = q8i::cuda_status(cudaSetDevice(device_));
    if (st != Q8MV_OK) device_ = prev_;
    return st;
}

}  // namespace kv

extern "C" {

q8mv_status_t q8kv_cache_write(const q8kv_cache_t *cache, int64_t n, const void *k, const void *v, int32_t type,
                               int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head, const int64_t *slots,
                               cudaStream_t stream) {
    kv::IoParams p = {};
    if (!kv::make_cache(cache, &p.c) || n < 0 || n >= (1LL << 31) || !kv::valid_type(type)) return Q8MV_ERR_INVALID_ARG;
    if (!kv::valid_stride(k_row) || !kv::valid_stride(k_head) || !kv::valid_stride(v_row) || !kv::valid_stride(v_head))
        return Q8MV_ERR_INVALID_ARG;
    if (n == 0 || p.c.slots == 0) return Q8MV_OK;
    const int size = kv::type_size(type);
    if (!k || !v || !slots || !kv::aligned(k, size) || !kv::aligned(v, size) || !kv::aligned(slots, 8))
        return Q8MV_ERR_INVALID_ARG;
    p.in[0] = k;
    p.in[1] = v;
    p.row[0] = k_row;
    p.row[1] = v_row;
    p.head[0] = k_head;
    p.head[1] = v_head;
    p.slots = slots;
    p.n = n;
    p.lanes = p.c.heads * p.c.blocks * (size == 4 ? 8 : 4);
    const int64_t e = 16 / size;
    const bool vec = kv::aligned(k, 16) && kv::aligned(v, 16) &&
                     ((k_row | k_head | v_row | v_head) & (e - 1)) == 0;
    kv::Shape s = kv::shape(p.lanes, n, kv::kWriteTokens);
    if (!vec && s.many) {  // element-wise loads: one token a thread
        s.many = false;
        s.grid.x = static_cast<unsigned>(kv::ceil_div(n, s.block.y));
    }
    if (type == Q8KV_F32)
        kv::launch_write<float>(p, vec, s, stream);
    else if (type == Q8KV_F16)
        kv::launch_write<__half>(p, vec, s, stream);
    else
        kv::launch_write<__nv_bfloat16>(p, vec, s, stream);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t q8kv_cache_read(const q8kv_cache_t *cache, int64_t n, const int64_t *slots, void *k_out, void *v_out,
                              int32_t type, cudaStream_t stream) {
    kv::IoParams p = {};
    if (!kv::make_cache(cache, &p.c) || n < 0 || n >= (1LL << 31) || !kv::valid_type(type)) return Q8MV_ERR_INVALID_ARG;
    if (n == 0) return Q8MV_OK;
    if (!slots || !k_out || !v_out || !kv::aligned(slots, 8) || !kv::aligned(k_out, 16) || !kv::aligned(v_out, 16))
        return Q8MV_ERR_INVALID_ARG;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.slots = slots;
    p.n = n;
    const int size = kv::type_size(type);
    p.lanes = p.c.heads * p.c.dim * size / 16;
    const kv::Shape s = kv::shape(p.lanes, n, kv::kReadTokens);
    if (type == Q8KV_F32)
        kv::launch_read<float>(p, s, stream);
    else if (type == Q8KV_F16)
        kv::launch_read<__half>(p, s, stream);
    else
        kv::launch_read<__nv_bfloat16>(p, s, stream);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t q8kv_cache_move(const q8kv_cache_t *cache, int64_t batch, int64_t path, const int64_t *src,
                              const int64_t *dst, cudaStream_t stream) {
    kv::MoveParams p = {};
    if (!kv::make_cache(cache, &p.c) || batch < 0 || batch > 65535 || path < 0 || path >= (1LL << 31))
        return Q8MV_ERR_INVALID_ARG;
    if (batch == 0 || path == 0 || p.c.slots == 0) return Q8MV_OK;
    if (!src || !dst || !kv::aligned(src, 8) || !kv::aligned(dst, 8)) return Q8MV_ERR_INVALID_ARG;
    p.src = src;
    p.dst = dst;
    p.path = static_cast<int>(path);
    p.scale_pieces = p.c.blocks % 4 == 0 ? p.c.blocks / 4 : p.c.blocks;
    p.lanes = p.c.heads * 2 * (p.c.dim / 16 + p.scale_pieces);
    const int threads = p.lanes >= 256 ? 256 : (p.lanes + 31) / 32 * 32;
    kv::q8kv_move_kernel<<<dim3(static_cast<unsigned>(kv::ceil_div(p.lanes, threads)), static_cast<unsigned>(batch)),
                           threads, 0, stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

}  // extern "C"
