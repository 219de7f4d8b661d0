// Writing, reading and moving rows of the Q8_0 cache (../../include/q8kv.h), and
// the device check of the q8kv plans.
//
// All three are streams without reuse, bound by HBM for many rows and by one
// round trip for few.  Every lane handles 16 bytes of the wide side (8 16-bit
// elements or 4 f32), so its loads or stores are one full vector and a warp's
// are contiguous; a 32-element block is then 4 or 8 neighbouring lanes and its
// amax takes 2 or 3 shuffles.  Keys and values of the same place are handled by
// the same lane, which keeps two independent loads in flight.
#include "kv_common.cuh"

namespace kv {

namespace {

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

template <typename T, bool VEC>
__device__ __forceinline__ void load_elems(const T *p, float (&x)[16 / sizeof(T)]) {
    constexpr int E = 16 / sizeof(T);
    if constexpr (VEC) {
        union {
            uint4 u;
            T t[E];
        } v;
        v.u = __ldg(reinterpret_cast<const uint4 *>(p));
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = to_f32(v.t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = to_f32(p[i]);
    }
}

__device__ __forceinline__ uint32_t pack4(const float *x, float id) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // NaN becomes 0; the clamp only acts where 127 / amax overflows (amax < 4e-37)
        const int c = max(-127, min(127, __float2int_rn(__fmul_rn(x[i], id))));
        w |= (static_cast<uint32_t>(c) & 0xFFu) << (8 * i);
    }
    return w;
}

// d = amax / 127, c = rint(x * (127 / amax)): the recipe of q8mv_quantize_rows.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) q8kv_write_kernel(const IoParams p) {
    constexpr int E = 16 / sizeof(T), PER = 32 / E;  // elements a lane, lanes a block
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int at = blockIdx.y * blockDim.x + threadIdx.x;
    int64_t page = 0;
    int place = 0;
    // whole groups of PER lanes share (token, head, block), so they leave together
    if (i >= p.n || at >= p.lanes || !place_of(p.c, p.slots[i], &page, &place)) return;
    const unsigned group = ((1u << PER) - 1u) << ((threadIdx.y * blockDim.x + threadIdx.x) & 31 & ~(PER - 1));
    const int per_head = p.c.blocks * PER;
    const int h = at / per_head, in_row = at - h * per_head, e0 = in_row * E, b = in_row / PER;
    const bool live = e0 < p.c.dim;
    const int64_t r = row_of(p.c, page, h, place);
    float x[2][E];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const T *src = static_cast<const T *>(p.in[s]) + i * p.row[s] + h * p.head[s] + e0;
        if (live) {
            load_elems<T, VEC>(src, x[s]);
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) x[s][j] = 0.0f;
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < E; ++j) amax = fmaxf(amax, fabsf(x[s][j]));
#pragma unroll
        for (int d = 1; d < PER; d *= 2) amax = fmaxf(amax, __shfl_xor_sync(group, amax, d));
        const float id = amax > 0.0f ? __fdiv_rn(127.0f, amax) : 0.0f;
        int8_t *codes = (s == 0 ? p.c.k_codes : p.c.v_codes) + r * p.c.dim + e0;
        float *scales = (s == 0 ? p.c.k_scales : p.c.v_scales) + r * p.c.blocks + b;
        if (live) {
            if constexpr (E == 8)
                *reinterpret_cast<uint2 *>(codes) = make_uint2(pack4(x[s], id), pack4(x[s] + 4, id));
            else
                *reinterpret_cast<uint32_t *>(codes) = pack4(x[s], id);
        }
        if ((in_row & (PER - 1)) == 0) *scales = __fdiv_rn(amax, 127.0f);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) q8kv_read_kernel(const IoParams p) {
    constexpr int E = 16 / sizeof(T);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int at = blockIdx.y * blockDim.x + threadIdx.x;
    if (i >= p.n || at >= p.lanes) return;
    const int per_head = p.c.dim / E;
    const int h = at / per_head, e0 = (at - h * per_head) * E, b = e0 / 32;
    int64_t page = 0;
    int place = 0;
    const bool live = place_of(p.c, p.slots[i], &page, &place);
    uint32_t w[2][E / 4] = {};
    float d[2] = {};
    if (live) {
        const int64_t r = row_of(p.c, page, h, place);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int8_t *codes = (s == 0 ? p.c.k_codes : p.c.v_codes) + r * p.c.dim + e0;
            if constexpr (E == 8) {
                const uint2 u = *reinterpret_cast<const uint2 *>(codes);
                w[s][0] = u.x;
                w[s][1] = u.y;
            } else {
                w[s][0] = *reinterpret_cast<const uint32_t *>(codes);
            }
            d[s] = ((s == 0 ? p.c.k_scales : p.c.v_scales) + r * p.c.blocks)[b];
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        union {
            uint4 u;
            T t[E];
        } v;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int c = static_cast<int8_t>(w[s][j / 4] >> (8 * (j % 4)));
            v.t[j] = from_f32<T>(__fmul_rn(static_cast<float>(c), d[s]));
        }
        T *out = static_cast<T *>(p.out[s]) + (i * p.c.heads + h) * p.c.dim + e0;
        *reinterpret_cast<uint4 *>(out) = v.u;
    }
}

struct MoveParams {
    Cache c;
    const int64_t *src, *dst;
    int path;
    int lanes;  // lanes of one token: heads * (2 * dim / 16 + 2 * blocks)
};

constexpr int kMoveBatch = 8;

// One lane owns one 16-byte piece of codes or one scale of every row that its
// request moves, so the order of a request's pairs is the lane's own program
// order and needs no barrier.  Eight pairs are loaded before any is stored,
// unless one of them is read by a later one of the eight.
__global__ void __launch_bounds__(256) q8kv_move_kernel(const MoveParams p) {
    const int64_t *src = p.src + static_cast<int64_t>(blockIdx.y) * p.path;
    const int64_t *dst = p.dst + static_cast<int64_t>(blockIdx.y) * p.path;
    const int at = blockIdx.x * blockDim.x + threadIdx.x;
    const int pieces = p.c.dim / 16, per_head = 2 * pieces + 2 * p.c.blocks;
    const bool mine = at < p.lanes;
    const int h = mine ? at / per_head : 0, in = mine ? at - h * per_head : 0;
    const bool wide = in < 2 * pieces;
    // byte address of the lane's piece in row 0, and the bytes of one row of its array
    char *base;
    int64_t pitch;
    if (wide) {
        base = reinterpret_cast<char *>(in < pieces ? p.c.k_codes : p.c.v_codes) + (in < pieces ? in : in - pieces) * 16;
        pitch = p.c.dim;
    } else {
        const int s = in - 2 * pieces;
        base = reinterpret_cast<char *>(s < p.c.blocks ? p.c.k_scales + s : p.c.v_scales + s - p.c.blocks);
        pitch = 4LL * p.c.blocks;
    }
    for (int i0 = 0; i0 < p.path; i0 += kMoveBatch) {
        const int n = min(kMoveBatch, p.path - i0);
        int64_t from[kMoveBatch], to[kMoveBatch];
        bool meet = false;
#pragma unroll
        for (int i = 0; i < kMoveBatch; ++i) {
            const int64_t s = i < n ? src[i0 + i] : -1, d = i < n ? dst[i0 + i] : -1;
            int64_t page;
            int place;
            const bool ok = place_of(p.c, d, &page, &place);
            to[i] = ok ? row_of(p.c, page, h, place) : -1;
            from[i] = ok && place_of(p.c, s, &page, &place) ? row_of(p.c, page, h, place) : -1;
        }
#pragma unroll
        for (int i = 0; i < kMoveBatch; ++i)
#pragma unroll
            for (int j = i + 1; j < kMoveBatch; ++j) meet |= from[j] >= 0 && from[i] >= 0 && from[j] == to[i];
        if (!mine) continue;
        if (wide) {
            if (!meet) {
                uint4 v[kMoveBatch];
#pragma unroll
                for (int i = 0; i < kMoveBatch; ++i)
                    if (from[i] >= 0) v[i] = *reinterpret_cast<const uint4 *>(base + from[i] * pitch);
#pragma unroll
                for (int i = 0; i < kMoveBatch; ++i)
                    if (from[i] >= 0) *reinterpret_cast<uint4 *>(base + to[i] * pitch) = v[i];
            } else {
#pragma unroll
                for (int i = 0; i < kMoveBatch; ++i)
                    if (from[i] >= 0)
                        *reinterpret_cast<uint4 *>(base + to[i] * pitch) =
                            *reinterpret_cast<const uint4 *>(base + from[i] * pitch);
            }
        } else {
            if (!meet) {
                float v[kMoveBatch];
#pragma unroll
                for (int i = 0; i < kMoveBatch; ++i)
                    if (from[i] >= 0) v[i] = *reinterpret_cast<const float *>(base + from[i] * pitch);
#pragma unroll
                for (int i = 0; i < kMoveBatch; ++i)
                    if (from[i] >= 0) *reinterpret_cast<float *>(base + to[i] * pitch) = v[i];
            } else {
#pragma unroll
                for (int i = 0; i < kMoveBatch; ++i)
                    if (from[i] >= 0)
                        *reinterpret_cast<float *>(base + to[i] * pitch) =
                            *reinterpret_cast<const float *>(base + from[i] * pitch);
            }
        }
    }
}

// Threads of one token along x (a multiple of 32, at most 256), tokens along y.
void shape(int lanes, int64_t n, dim3 *grid, dim3 *block) {
    const unsigned x = lanes >= 256 ? 256u : static_cast<unsigned>((lanes + 31) / 32 * 32);
    const unsigned y = 256u / x;
    *block = dim3(x, y);
    *grid = dim3(static_cast<unsigned>(ceil_div(n, y)), static_cast<unsigned>(ceil_div(lanes, x)));
}

template <typename T>
void launch_write(const IoParams &p, bool vec, dim3 grid, dim3 block, cudaStream_t stream) {
    if (vec)
        q8kv_write_kernel<T, true><<<grid, block, 0, stream>>>(p);
    else
        q8kv_write_kernel<T, false><<<grid, block, 0, stream>>>(p);
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
    dim3 grid, block;
    kv::shape(p.lanes, n, &grid, &block);
    if (type == Q8KV_F32)
        kv::launch_write<float>(p, vec, grid, block, stream);
    else if (type == Q8KV_F16)
        kv::launch_write<__half>(p, vec, grid, block, stream);
    else
        kv::launch_write<__nv_bfloat16>(p, vec, grid, block, stream);
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
    dim3 grid, block;
    kv::shape(p.lanes, n, &grid, &block);
    if (type == Q8KV_F32)
        kv::q8kv_read_kernel<float><<<grid, block, 0, stream>>>(p);
    else if (type == Q8KV_F16)
        kv::q8kv_read_kernel<__half><<<grid, block, 0, stream>>>(p);
    else
        kv::q8kv_read_kernel<__nv_bfloat16><<<grid, block, 0, stream>>>(p);
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
    p.lanes = p.c.heads * (2 * (p.c.dim / 16) + 2 * p.c.blocks);
    const int threads = p.lanes >= 256 ? 256 : (p.lanes + 31) / 32 * 32;
    kv::q8kv_move_kernel<<<dim3(static_cast<unsigned>(kv::ceil_div(p.lanes, threads)), static_cast<unsigned>(batch)),
                           threads, 0, stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

}  // extern "C"
