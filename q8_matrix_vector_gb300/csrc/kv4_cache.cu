// Writing, reading and moving rows of the Q4_0 cache (../../include/q4kv.h).
#include "kv_store.cuh"

namespace kv {

namespace {

struct ReadParams {
    Cache c;  // Cache4::rows
    int dim, blocks;
    void *out[2];
    const int64_t *slots;
    int64_t n;
    int lanes;  // of one token: heads * dim / E
};

// 8190 tokens of 32 heads of 128 to bf16: 34.9 us, 4.9 TB/s.  3.5 bytes are written for each that is read, so that the
// GPU's write rate bounds it (a plain fill of 1 GB: 4.1 TB/s).
constexpr int kReadTokens4 = 2;

// A lane gives 16 bytes of a key and of its value: 8 elements are one unit of a key and two of a value, 4 half of one
// and one.
template <typename T, int U>
__global__ void __launch_bounds__(256) q4kv_read_kernel(const ReadParams p) {
    constexpr int E = 16 / sizeof(T);
    __shared__ int64_t rows[8 * U];
    const int tokens = blockDim.y * U, tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
    const int at = blockIdx.y * blockDim.x + threadIdx.x;
    if (tid < tokens) {
        const int64_t slot = first + tid < p.n ? __ldg(p.slots + first + tid) : -1;
        int64_t r = -1;
        if (slot >= 0 && slot < p.c.slots) {
            const int64_t page = slot / p.c.page_size;
            r = row_of(p.c, page, 0, static_cast<int>(slot - page * p.c.page_size));
        }
        rows[tid] = r;
    }
    __syncthreads();
    if (at >= p.lanes) return;
    const int per_head = p.dim / E, nb = p.blocks;
    const int h = at / per_head, e0 = (at - h * per_head) * E, b = e0 / 32, i = e0 % 32;
    uint32_t w[U][2] = {};
    float d[U][2] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r0 = rows[u * blockDim.y + threadIdx.y];
        if (r0 >= 0) {
            const int64_t r = r0 + h * p.c.stride_head;
            const unsigned char *kc = reinterpret_cast<const unsigned char *>(p.c.k_codes) + r * p.c.dim + 4 * (i / 8 * nb + b);
            const unsigned char *vc = reinterpret_cast<const unsigned char *>(p.c.v_codes) + r * p.c.dim + 2 * (i / 4 * nb + b);
            if constexpr (E == 8) {
                w[u][0] = *reinterpret_cast<const uint32_t *>(kc);
                w[u][1] = *reinterpret_cast<const uint16_t *>(vc) |
                          static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(vc + 2 * nb)) << 16;
            } else {
                w[u][0] = *reinterpret_cast<const uint16_t *>(kc + i % 8 / 2);
                w[u][1] = *reinterpret_cast<const uint16_t *>(vc);
            }
            d[u][0] = __half2float((reinterpret_cast<const __half *>(p.c.k_scales) + r * (2 * p.c.blocks))[b]);
            d[u][1] = __half2float((reinterpret_cast<const __half *>(p.c.v_scales) + r * (2 * p.c.blocks))[b]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t token = first + u * blockDim.y + threadIdx.y;
        if (token >= p.n) break;
        const bool there = rows[u * blockDim.y + threadIdx.y] >= 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            store::Piece<T> x;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                // 2^23 + c, less 2^23 + 8
                const float c = __uint_as_float(0x4B000000u | ((w[u][s] >> (4 * j)) & 15u)) - 8388616.0f;
                x.t[j] = from_f32<T>(there ? __fmul_rn(c, d[u][s]) : 0.0f);
            }
            *reinterpret_cast<uint4 *>(static_cast<T *>(p.out[s]) + (token * p.c.heads + h) * p.dim + e0) = x.v;
        }
    }
}

template <typename T>
void launch_read4(const ReadParams &p, const Shape &s, cudaStream_t stream) {
    if (s.many)
        q4kv_read_kernel<T, kReadTokens4><<<s.grid, s.block, 0, stream>>>(p);
    else
        q4kv_read_kernel<T, 1><<<s.grid, s.block, 0, stream>>>(p);
}

}  // namespace

}  // namespace kv

extern "C" {

q8mv_status_t q4kv_cache_write(const q4kv_cache_t *cache, int64_t n, const void *k, const void *v, int32_t type,
                               int64_t k_row, int64_t k_head, int64_t v_row, int64_t v_head, const int64_t *slots,
                               cudaStream_t stream) {
    kv::Cache4 c = {};
    kv::StoreParams p = {};
    if (!kv::make_cache4(cache, &c) || n < 0 || n >= (1LL << 31) || !kv::valid_type(type)) return Q8MV_ERR_INVALID_ARG;
    if (!kv::valid_stride(k_row) || !kv::valid_stride(k_head) || !kv::valid_stride(v_row) || !kv::valid_stride(v_head))
        return Q8MV_ERR_INVALID_ARG;
    if (n == 0 || c.rows.slots == 0) return Q8MV_OK;
    const int size = kv::type_size(type);
    if (!k || !v || !slots || !kv::aligned(k, size) || !kv::aligned(v, size) || !kv::aligned(slots, 8))
        return Q8MV_ERR_INVALID_ARG;
    p.c = c.rows;
    p.dim = c.dim;
    p.blocks = c.blocks;
    p.in[0] = k;
    p.in[1] = v;
    p.row[0] = k_row;
    p.row[1] = v_row;
    p.head[0] = k_head;
    p.head[1] = v_head;
    p.slots = slots;
    p.n = n;
    p.lanes = c.rows.heads * c.blocks * (size == 4 ? 8 : 4);
    const int64_t e = 16 / size;
    const bool vec = kv::aligned(k, 16) && kv::aligned(v, 16) && ((k_row | k_head | v_row | v_head) & (e - 1)) == 0;
    kv::Shape s = kv::shape(p.lanes, n, kv::kStoreTokens);
    if (!vec && s.many) {  // element-wise loads: one token a thread
        s.many = false;
        s.grid.x = static_cast<unsigned>(kv::ceil_div(n, s.block.y));
    }
    p.kv_y = static_cast<int>(s.grid.y);
    if (type == Q8KV_F32)
        kv::launch_store<float, 4, false>(p, vec, s, 0, stream);
    else if (type == Q8KV_F16)
        kv::launch_store<__half, 4, false>(p, vec, s, 0, stream);
    else
        kv::launch_store<__nv_bfloat16, 4, false>(p, vec, s, 0, stream);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t q4kv_cache_read(const q4kv_cache_t *cache, int64_t n, const int64_t *slots, void *k_out, void *v_out,
                              int32_t type, cudaStream_t stream) {
    kv::Cache4 c = {};
    if (!kv::make_cache4(cache, &c) || n < 0 || n >= (1LL << 31) || !kv::valid_type(type)) return Q8MV_ERR_INVALID_ARG;
    if (n == 0) return Q8MV_OK;
    if (!slots || !k_out || !v_out || !kv::aligned(slots, 8) || !kv::aligned(k_out, 16) || !kv::aligned(v_out, 16))
        return Q8MV_ERR_INVALID_ARG;
    kv::ReadParams p = {c.rows, c.dim, c.blocks, {k_out, v_out}, slots, n, c.rows.heads * c.dim * kv::type_size(type) / 16};
    const kv::Shape s = kv::shape(p.lanes, n, kv::kReadTokens4);
    if (type == Q8KV_F32)
        kv::launch_read4<float>(p, s, stream);
    else if (type == Q8KV_F16)
        kv::launch_read4<__half>(p, s, stream);
    else
        kv::launch_read4<__nv_bfloat16>(p, s, stream);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t q4kv_cache_move(const q4kv_cache_t *cache, int64_t batch, int64_t path, const int64_t *src,
                              const int64_t *dst, cudaStream_t stream) {
    kv::Cache4 c = {};
    if (!kv::make_cache4(cache, &c)) return Q8MV_ERR_INVALID_ARG;
    return kv::cache_move(c.rows, batch, path, src, dst, stream);
}

}  // extern "C"
