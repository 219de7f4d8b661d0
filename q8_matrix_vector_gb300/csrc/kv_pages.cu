// Pages of a cache (../../include/kvpage.h): who holds which, and copies of their
// contents.
//
// The bookkeeping is small whole-number work whose time is latency: launches,
// round trips to L2 and barriers, not bytes.  What has to be ordered (which page is
// the k-th free one, which request gets it) is one thread-block cluster's work, so
// that a step needs one launch: its CTAs take a share of the requests and of the pages
// each, exchange their counts through distributed shared memory and go on without the
// host or a second kernel.  Nothing is read that another CTA writes in the same phase.
// Counts of holders change by atomics: whole numbers, any order.
//
// Copies are HBM's: every thread has four 16-byte loads in flight before their stores.
//
// Measured on GB300: extend 5.5 us for 12 requests and 6.8 for 144, fork and free 3 each,
// compact of 16384 pages 8.3; 4035 pages of 36 KB copied in 53 us, 5.6 TB/s (copy rate 6.8).
#include "../../include/kvpage.h"
#include "kv4.h"
#include "kv_common.cuh"

#include <algorithm>
#include <cooperative_groups.h>
#include <new>

namespace cg = cooperative_groups;

struct kvpage_s {
    int device = 0;
    int pages = 0, page_size = 0, requests = 0, columns = 0;
    int *work = nullptr;
};

namespace kv {

namespace {

constexpr int kThreads = 512, kPer = 4;  // of a CTA that counts; pages a thread takes at a time
constexpr int kCluster = 8;
constexpr int kTile = kThreads * kPer;
constexpr int kFewColumns = 4;  // a thread looks at so many alone

struct PageParams {
    int *refs, *table, *held;
    int pages, page_size, requests, columns;
    const int *lengths, *tokens;
    int64_t *slots;
    int width, slots_here;
    int *src, *dst, *ok, *count;
    // workspace
    int *amount;         // [requests] fresh pages wanted, -1: refused
    int *fresh, *old;    // [pages] pages given out, and what they replace (-1: nothing)
    int *dense;          // [1] L
};

// Sum over the block before this thread, and of all of it.
__device__ __forceinline__ int scan(int x, int *total, int *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int in = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(~0u, in, d);
        if (lane >= d) in += y;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warp_sums[warp] = in;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return before + in - x;
}

// Every CTA's number reaches every CTA: the sum of those before this one, and of all.  `box` has a place for each.
__device__ __forceinline__ int exchange(cg::cluster_group &cluster, int *box, int mine, int *total) {
    const int ranks = cluster.num_blocks(), me = cluster.block_rank();
    if (ranks == 1) {
        *total = mine;
        return 0;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < ranks) cluster.map_shared_rank(box, threadIdx.x)[me] = mine;
    cluster.sync();
    int before = 0, all = 0;
    for (int r = 0; r < ranks; ++r) {
        if (r < me) before += box[r];
        all += box[r];
    }
    *total = all;
    return before;
}

// refs of the thread's kPer pages from p0, -1 past `end`
__device__ __forceinline__ void load_refs(const int *refs, int p0, int end, int (&r)[kPer]) {
    if (p0 + kPer <= end && (reinterpret_cast<uintptr_t>(refs + p0) & 15) == 0) {
        const int4 x = *reinterpret_cast<const int4 *>(refs + p0);
        r[0] = x.x;
        r[1] = x.y;
        r[2] = x.z;
        r[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) r[i] = p0 + i < end ? refs[p0 + i] : -1;
    }
}

// x / page_size; 64-bit divisions take a hundred instructions
__device__ __forceinline__ int64_t pages_of(const PageParams &p, int64_t x) {
    return (x >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(p.page_size)) : x / p.page_size;
}

// A request's span of columns: those that will be written.
struct Span {
    int64_t length, tokens;
    int held, first, need;  // need > columns: refused
};
__device__ __forceinline__ Span span_of(const PageParams &p, int b) {
    Span s;
    s.length = max(p.lengths[b], 0);
    s.tokens = max(p.tokens[b], 0);
    s.held = min(max(p.held[b], 0), p.columns);
    const int64_t need = s.tokens > 0 ? pages_of(p, s.length + s.tokens + p.page_size - 1) : 0;
    s.need = static_cast<int>(min(need, static_cast<int64_t>(p.columns) + 1));
    s.first = static_cast<int>(min(pages_of(p, s.length), static_cast<int64_t>(s.held)));
    return s;
}

// Whether a held column gets a fresh page; *page: what is there now, -1 if it is none.
__device__ __forceinline__ bool replaced(const PageParams &p, int b, int c, int *page) {
    const int x = p.table[static_cast<int64_t>(b) * p.columns + c];
    *page = static_cast<unsigned>(x) < static_cast<unsigned>(p.pages) ? x : -1;
    return *page < 0 || p.refs[*page] > 1;
}

__device__ __forceinline__ int64_t slot_at(const PageParams &p, int b, int64_t position) {
    const int64_t c = pages_of(p, position);
    const int64_t page = p.table[static_cast<int64_t>(b) * p.columns + c];
    return page * p.page_size + position - c * p.page_size;
}

__global__ void __launch_bounds__(kThreads, 1) kvpage_extend_kernel(const PageParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // waited for before the first exchange: nobody's shared memory is written before it runs
    __shared__ int warp_sums[kThreads / 32], box[3][kCluster], starts[kThreads];
    const int ranks = cluster.num_blocks(), me = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.requests + ranks - 1) / ranks;
    const int b0 = min(me * per, p.requests), b1 = min(b0 + per, p.requests);
    // the first refs of the CTA's pages, on their way while the requests are looked at
    const int share = ((p.pages + ranks - 1) / ranks + kPer - 1) / kPer * kPer;
    const int p0 = static_cast<int>(min(static_cast<int64_t>(me) * share, static_cast<int64_t>(p.pages)));
    const int p1 = min(p0 + share, p.pages);
    int r0[kPer], r[kPer];
    load_refs(p.refs, p0 + threadIdx.x * kPer, p1, r0);
    // ---- how many pages each request wants: a thread each, or its warp where many columns are to be looked at (amounts
    // stay here if a tile holds them)
    const bool few = b1 - b0 <= kThreads;
    int mine = 0;
    for (int t0 = b0; t0 < b1; t0 += kThreads) {
        const int b = t0 + threadIdx.x;
        int n = 0, first = 0, end = 0;  // held columns first .. end - 1 may be replaced
        if (b < b1) {
            const Span s = span_of(p, b);
            if (s.need <= p.columns) {
                n = max(s.need - s.held, 0);
                first = s.first;
                end = max(min(s.held, s.need), first);
            } else {
                n = -1;
            }
        }
        int page;
        if (end - first <= kFewColumns)
            for (int c = first; c < end; ++c) n += replaced(p, b, c, &page);
        for (unsigned many = __ballot_sync(~0u, end - first > kFewColumns); many != 0; many &= many - 1) {
            const int who = __ffs(many) - 1, rb = t0 + warp * 32 + who;
            const int c0 = __shfl_sync(~0u, first, who), c1 = __shfl_sync(~0u, end, who);
            int k = 0;
            for (int c = c0 + lane; c < c1; c += 32) k += replaced(p, rb, c, &page);
            k = __reduce_add_sync(~0u, k);
            if (lane == who) n += k;
        }
        if (b < b1) (few ? starts[threadIdx.x] : p.amount[b]) = n;
        mine += max(n, 0);
    }
    int total;
    scan(mine, &total, warp_sums);
    cluster.barrier_wait();
    int wanted, free_pages = 0;
    const int before = exchange(cluster, box[0], total, &wanted);
    // ---- the lowest free pages in order
    if (wanted > 0) {
        int at = 0;
        if (ranks > 1) {  // how many there are before the CTA's
            int count = 0;
            for (int t = p0 + threadIdx.x * kPer; t < p1; t += kTile) {
                load_refs(p.refs, t, p1, r);
#pragma unroll
                for (int i = 0; i < kPer; ++i) count += r[i] == 0;
            }
            scan(count, &total, warp_sums);
            at = exchange(cluster, box[1], total, &free_pages);
        }
        for (int t0 = p0; t0 < p1 && at < wanted; t0 += kTile) {  // (the same for all threads)
            const int t = t0 + threadIdx.x * kPer;
            if (t0 == p0) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) r[i] = r0[i];
            } else {
                load_refs(p.refs, t, p1, r);
            }
            int n = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) n += r[i] == 0;
            int k = at + scan(n, &total, warp_sums);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (r[i] == 0) {
                    if (k < wanted) p.fresh[k] = t + i;
                    ++k;
                }
            at += total;
        }
        // the list is there
        if (ranks > 1) {
            cluster.sync();
        } else {
            free_pages = at;  // (at least `wanted`, or all)
            __syncthreads();
        }
    }
    // ---- the requests take them
    int served = 0, base = before;
    for (int t0 = b0; t0 < b1; t0 += kThreads) {
        const int b = t0 + threadIdx.x;
        const int n = b >= b1 ? 0 : few ? starts[threadIdx.x] : p.amount[b];
        int k = base + scan(max(n, 0), &total, warp_sums);
        const bool fits = n >= 0 && (n == 0 || k + n <= free_pages);
        if (fits && n > 0) served = max(served, k + n);
        starts[threadIdx.x] = fits ? k : -1;
        base += total;
        Span s = {};
        if (b < b1) s = span_of(p, b);
        const bool goes = b < b1 && fits && s.need > s.first;
        const int64_t col = pages_of(p, s.length);
        const int part = s.length != col * p.page_size && col < p.columns ? static_cast<int>(col) : -1;  // its page has tokens
        int from = -1, to = -1;
        // column c gets page p.fresh[at]
        auto give = [&](int rb, int c, int at, int old, int part_c, int *f, int *g) {
            const int x = p.fresh[at];
            p.table[static_cast<int64_t>(rb) * p.columns + c] = x;
            p.old[at] = old;
            if (c == part_c && old >= 0) {
                *f = old;
                *g = x;
            }
        };
        if (goes && s.need - s.first <= kFewColumns)
            for (int c = s.first; c < s.need; ++c) {
                int page = -1;
                if (c >= s.held || replaced(p, b, c, &page)) give(b, c, k++, page, part, &from, &to);
            }
        for (unsigned many = __ballot_sync(~0u, goes && s.need - s.first > kFewColumns); many != 0; many &= many - 1) {
            const int who = __ffs(many) - 1, rb = t0 + warp * 32 + who;
            const int first = __shfl_sync(~0u, s.first, who), need = __shfl_sync(~0u, s.need, who), held = __shfl_sync(~0u, s.held, who);
            const int part_c = __shfl_sync(~0u, part, who);
            int done = __shfl_sync(~0u, k, who), f = -1, g = -1;
            for (int c0 = first; c0 < need; c0 += 32) {
                const int c = c0 + lane;
                int page = -1;
                const bool fresh = c < need && (c >= held || replaced(p, rb, c, &page));
                const unsigned all = __ballot_sync(~0u, fresh);
                if (fresh) give(rb, c, done + __popc(all & ((1u << lane) - 1u)), page, part_c, &f, &g);
                done += __popc(all);
            }
            f = __reduce_max_sync(~0u, f);
            g = __reduce_max_sync(~0u, g);
            if (lane == who) {
                from = f;
                to = g;
            }
        }
        if (b < b1) {
            if (goes && s.need > s.held) p.held[b] = s.need;
            p.src[b] = from;
            p.dst[b] = to;
            p.ok[b] = fits;
        }
        __syncthreads();  // the tile's rows and starts are there
        if (p.slots_here)
            for (int i = threadIdx.x; i < min(kThreads, b1 - t0) * p.width; i += kThreads) {
                const int r = i / p.width, w = i - r * p.width, rb = t0 + r;
                const bool there = starts[r] >= 0 && w < p.tokens[rb];
                p.slots[static_cast<int64_t>(rb) * p.width + w] = there ? slot_at(p, rb, static_cast<int64_t>(max(p.lengths[rb], 0)) + w) : -1;
            }
        __syncthreads();
    }
    if (wanted == 0) return;  // (no CTA waits for another, or writes to it, from here)
    // ---- their counts: nobody reads them any more
    served = __reduce_max_sync(~0u, served);
    __syncthreads();
    if (lane == 0) warp_sums[warp] = served;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) served = max(served, warp_sums[w]);
    if (ranks > 1) {
        if (static_cast<int>(threadIdx.x) < ranks) cluster.map_shared_rank(box[2], threadIdx.x)[me] = served;
        cluster.sync();
        for (int i = 0; i < ranks; ++i) served = max(served, box[2][i]);
    }
    for (int i = me * kThreads + threadIdx.x; i < served; i += ranks * kThreads) {
        p.refs[p.fresh[i]] = 1;
        const int old = p.old[i];
        if (old >= 0) atomicSub(p.refs + old, 1);
    }
}

// Slots of calls with many tokens a request, which one warp a request would take long for.
__global__ void __launch_bounds__(256) kvpage_slots_kernel(const PageParams p) {
    const int b = blockIdx.y, w = blockIdx.x * 256 + threadIdx.x;
    if (w >= p.width) return;
    const bool there = p.ok[b] != 0 && w < p.tokens[b];
    p.slots[static_cast<int64_t>(b) * p.width + w] = there ? slot_at(p, b, static_cast<int64_t>(max(p.lengths[b], 0)) + w) : -1;
}

// fork, first: what every changed request becomes is put aside, and its pages counted
__global__ void __launch_bounds__(256) kvpage_fork_read_kernel(const PageParams p, const int *parents, int *rows, int *count) {
    const int b = blockIdx.x, parent = parents[b];
    if (parent == b) return;
    const int n = static_cast<unsigned>(parent) < static_cast<unsigned>(p.requests) ? min(max(p.held[parent], 0), p.columns) : 0;
    for (int c = threadIdx.x; c < n; c += 256) {
        const int page = p.table[static_cast<int64_t>(parent) * p.columns + c];
        rows[static_cast<int64_t>(b) * p.columns + c] = page;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pages)) atomicAdd(p.refs + page, 1);
    }
    if (threadIdx.x == 0) count[b] = n;
}

// fork, second: the pages that it held go back, and the others take their place
__global__ void __launch_bounds__(256) kvpage_fork_write_kernel(const PageParams p, const int *parents, const int *rows, const int *count) {
    const int b = blockIdx.x;
    if (parents[b] == b) return;
    const int n = count[b], held = min(max(p.held[b], 0), p.columns);
    for (int c = threadIdx.x; c < max(n, held); c += 256) {
        int *at = p.table + static_cast<int64_t>(b) * p.columns + c;
        if (c < held) {
            const int page = *at;
            if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pages)) atomicSub(p.refs + page, 1);
        }
        *at = c < n ? rows[static_cast<int64_t>(b) * p.columns + c] : -1;
    }
    __syncthreads();  // everyone has read held
    if (threadIdx.x == 0) p.held[b] = n;
}

__global__ void __launch_bounds__(256) kvpage_free_kernel(const PageParams p) {
    const int b = blockIdx.x, held = min(max(p.held[b], 0), p.columns);
    const int64_t pages = (static_cast<int64_t>(max(p.lengths[b], 0)) + p.page_size - 1) / p.page_size;
    const int keep = static_cast<int>(min(pages, static_cast<int64_t>(held)));
    for (int c = keep + threadIdx.x; c < held; c += 256) {
        int *at = p.table + static_cast<int64_t>(b) * p.columns + c;
        const int page = *at;
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.pages)) atomicSub(p.refs + page, 1);
        *at = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) p.held[b] = keep;
}

// compact, first: who moves where (p.fresh: a page's new number, -1 for one past the dense part that nobody holds)
__global__ void __launch_bounds__(kThreads, 1) kvpage_compact_kernel(const PageParams p) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    __shared__ int warp_sums[kThreads / 32], box[3][kCluster];
    const int ranks = cluster.num_blocks(), me = cluster.block_rank();
    const int share = ((p.pages + ranks - 1) / ranks + kPer - 1) / kPer * kPer;
    const int p0 = static_cast<int>(min(static_cast<int64_t>(me) * share, static_cast<int64_t>(p.pages)));
    const int p1 = min(p0 + share, p.pages);
    int n = 0, r[kPer], total, dense, moves, holes;
    for (int t = p0 + threadIdx.x * kPer; t < p1; t += kTile) {
        load_refs(p.refs, t, p1, r);
#pragma unroll
        for (int i = 0; i < kPer; ++i) n += r[i] > 0;
    }
    scan(n, &total, warp_sums);
    cluster.barrier_wait();
    exchange(cluster, box[0], total, &dense);
    // holes below `dense`, and pages to move behind it
    n = 0;
    int m = 0;
    for (int t = p0 + threadIdx.x * kPer; t < p1; t += kTile) {
        load_refs(p.refs, t, p1, r);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n += t + i < dense && t + i < p1 && r[i] <= 0;
            m += t + i >= dense && r[i] > 0;
        }
    }
    scan(n, &total, warp_sums);
    int hole = exchange(cluster, box[1], total, &holes);
    scan(m, &total, warp_sums);
    int move = exchange(cluster, box[2], total, &moves);
    for (int t0 = p0; t0 < p1; t0 += kTile) {
        const int t = t0 + threadIdx.x * kPer;
        load_refs(p.refs, t, p1, r);
        n = m = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            n += t + i < dense && t + i < p1 && r[i] <= 0;
            m += t + i >= dense && r[i] > 0;
        }
        int kn = hole + scan(n, &total, warp_sums);
        hole += total;
        int km = move + scan(m, &total, warp_sums);
        move += total;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (t + i < p1) {
                if (t + i < dense && r[i] <= 0) p.dst[kn++] = t + i;
                if (t + i >= dense) {
                    if (r[i] > 0)
                        p.src[km++] = t + i;
                    else
                        p.fresh[t + i] = -1;
                }
            }
    }
    cluster.sync();  // the lists are there
    for (int i = me * kThreads + threadIdx.x; i < p.pages / 2; i += ranks * kThreads) {
        if (i < moves) {
            const int from = p.src[i], to = p.dst[i];
            p.refs[to] = p.refs[from];
            p.refs[from] = 0;
            p.fresh[from] = to;
        } else {
            p.src[i] = p.dst[i] = -1;
        }
    }
    if (me == 0 && threadIdx.x == 0) {
        p.count[0] = moves;
        p.dense[0] = dense;
    }
}

// compact, second: the tables follow
__global__ void __launch_bounds__(256) kvpage_follow_kernel(const PageParams p) {
    const int b = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= min(p.held[b], p.columns)) return;
    int *at = p.table + static_cast<int64_t>(b) * p.columns + c;
    const int page = *at;
    if (page >= p.dense[0] && page < p.pages) {
        const int now = p.fresh[page];
        if (now >= 0) *at = now;
    }
}

struct CopyParams {
    Cache c;
    const int *src, *dst, *count;
    int n;
    int rows;                      // of a page
    int code_pieces, scale_pieces; // of one array: of a page's memory (CONTIGUOUS) or of a row
    int wide;                      // scales move in 16 bytes, else in 4
    int chunks;                    // of a page
};

constexpr int kCopyThreads = 256, kCopyPieces = 4, kCopyBlocks = 152 * 8;

// Blocks take chunks of kCopyThreads * kCopyPieces pieces (16 KB) of pages in turn.
template <bool CONTIGUOUS>
__global__ void __launch_bounds__(kCopyThreads) kv_copy_pages_kernel(const CopyParams p) {
    const int pairs = p.count ? min(p.n, max(*p.count, 0)) : p.n;
    const int64_t total = static_cast<int64_t>(pairs) * p.chunks;
    const int per = 2 * (p.code_pieces + p.scale_pieces) * (CONTIGUOUS ? 1 : p.rows);
    for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const int pair = static_cast<int>(w / p.chunks), chunk = static_cast<int>(w - static_cast<int64_t>(pair) * p.chunks);
        const int from = __ldg(p.src + pair), to = __ldg(p.dst + pair);
        if (static_cast<unsigned>(from) >= static_cast<unsigned>(p.c.pages) || static_cast<unsigned>(to) >= static_cast<unsigned>(p.c.pages))
            continue;
        uint4 v[kCopyPieces];
        char *at[kCopyPieces];
        int size[kCopyPieces];  // 16, 4 or 0
#pragma unroll
        for (int j = 0; j < kCopyPieces; ++j) {
            const int i = (chunk * kCopyPieces + j) * kCopyThreads + threadIdx.x;
            size[j] = 0;
            if (i >= per) continue;
            int piece = i;
            // rows of the page before the piece's own, and their bytes in its array
            int64_t offset = 0;
            if (!CONTIGUOUS) {
                const int each = 2 * (p.code_pieces + p.scale_pieces), r = i / each, h = r / p.c.page_size;
                piece = i - r * each;
                offset = h * p.c.stride_head + (r - h * p.c.page_size) * p.c.stride_token;
            }
            const bool codes = piece < 2 * p.code_pieces;
            const int of = codes ? p.code_pieces : p.scale_pieces, k = codes ? piece : piece - 2 * p.code_pieces;
            const int in = k < of ? k : k - of;
            const int64_t pitch = codes ? p.c.dim : 4LL * p.c.blocks;
            char *base = codes ? reinterpret_cast<char *>(k < of ? p.c.k_codes : p.c.v_codes)
                               : reinterpret_cast<char *>(k < of ? p.c.k_scales : p.c.v_scales);
            size[j] = codes || p.wide ? 16 : 4;
            base += offset * pitch + static_cast<int64_t>(in) * size[j];
            at[j] = base + to * p.c.stride_page * pitch;
            const char *x = base + from * p.c.stride_page * pitch;
            if (size[j] == 16)
                v[j] = __ldcs(reinterpret_cast<const uint4 *>(x));
            else
                v[j].x = *reinterpret_cast<const uint32_t *>(x);
        }
#pragma unroll
        for (int j = 0; j < kCopyPieces; ++j) {
            if (size[j] == 16)
                *reinterpret_cast<uint4 *>(at[j]) = v[j];
            else if (size[j] == 4)
                *reinterpret_cast<uint32_t *>(at[j]) = v[j].x;
        }
    }
}

q8mv_status_t copy_pages(const Cache &c, int64_t n, const int32_t *src, const int32_t *dst, const int32_t *count,
                         cudaStream_t stream) {
    if (n < 0 || n >= (1LL << 31)) return Q8MV_ERR_INVALID_ARG;
    if (n == 0 || c.pages == 0) return Q8MV_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4)) return Q8MV_ERR_INVALID_ARG;
    CopyParams p = {};
    p.c = c;
    p.src = src;
    p.dst = dst;
    p.count = count;
    p.n = static_cast<int>(n);
    const int64_t rows = static_cast<int64_t>(c.heads) * c.page_size;
    // pieces of a page are numbered in 31 bits
    if (rows * (c.dim / 16 + c.blocks) * 2 + kCopyThreads * kCopyPieces >= (1LL << 31)) return Q8MV_ERR_INVALID_ARG;
    p.rows = static_cast<int>(rows);
    // an axis of one says nothing about its stride
    const bool by_head = (c.page_size == 1 || c.stride_token == 1) && (c.heads == 1 || c.stride_head == c.page_size);
    const bool by_token = (c.heads == 1 || c.stride_head == 1) && (c.page_size == 1 || c.stride_token == c.heads);
    const bool whole = by_head || by_token;
    if (whole) {
        p.code_pieces = static_cast<int>(rows * (c.dim / 16));
        p.wide = rows * c.blocks % 4 == 0 && c.stride_page % 4 * c.blocks % 4 == 0;
        p.scale_pieces = static_cast<int>(p.wide ? rows * c.blocks / 4 : rows * c.blocks);
    } else {
        p.code_pieces = c.dim / 16;
        p.wide = c.blocks % 4 == 0;
        p.scale_pieces = p.wide ? c.blocks / 4 : c.blocks;
    }
    const int64_t per = 2LL * (p.code_pieces + p.scale_pieces) * (whole ? 1 : rows);
    p.chunks = static_cast<int>(ceil_div(per, kCopyThreads * kCopyPieces));
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(kCopyBlocks, n * p.chunks));
    if (whole)
        kv_copy_pages_kernel<true><<<grid, kCopyThreads, 0, stream>>>(p);
    else
        kv_copy_pages_kernel<false><<<grid, kCopyThreads, 0, stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

// The state of a call; false if a pointer is missing or unaligned.
bool take(const kvpage_s *plan, const kvpage_state_t *s, PageParams *p) {
    if (plan == nullptr || s == nullptr) return false;
    for (const void *x : {static_cast<const void *>(s->refs), static_cast<const void *>(s->table), static_cast<const void *>(s->held)})
        if (x == nullptr || !aligned(x, 4)) return false;
    p->refs = s->refs;
    p->table = s->table;
    p->held = s->held;
    p->pages = plan->pages;
    p->page_size = plan->page_size;
    p->requests = plan->requests;
    p->columns = plan->columns;
    p->amount = plan->work;
    p->fresh = p->amount + plan->requests;
    p->old = p->fresh + plan->pages;
    p->dense = p->old + plan->pages;
    return true;
}

// One CTA for up to `pages` pages, whose work is a few round trips; a cluster, whose barriers are round trips of their own,
// for more (extend, 144 requests and 4096 pages: 11.0 us by a cluster, 6.8 by one; compact, 16384 pages: 8.4 and 16.8).
q8mv_status_t launch_cluster(void (*kernel)(PageParams), const PageParams &p, int pages, cudaStream_t stream) {
    const int ctas = p.pages > pages || p.requests > kThreads ? kCluster : 1;
    if (ctas == 1) {  // (a cluster of its own)
        kernel<<<1, kThreads, 0, stream>>>(p);
        return q8i::cuda_status(cudaGetLastError());
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    const cudaError_t last = cudaGetLastError();
    return q8i::cuda_status(e != cudaSuccess ? e : last);
}

}  // namespace

}  // namespace kv

extern "C" {

q8mv_status_t kvpage_plan(kvpage_plan_t *out, int64_t pages, int32_t page_size, int32_t requests, int32_t columns,
                          int device) {
    if (out == nullptr) return Q8MV_ERR_INVALID_ARG;
    *out = nullptr;
    if (pages < 1 || pages > (1LL << 28) || page_size < 1 || page_size > 65536 || requests < 1 || requests > 65535 ||
        columns < 1 || columns > (1 << 24) || static_cast<int64_t>(requests) * columns > (1LL << 28))
        return Q8MV_ERR_INVALID_ARG;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(device);
    if (st != Q8MV_OK) return st;
    kvpage_s *p = new (std::nothrow) kvpage_s();
    if (p == nullptr) return Q8MV_ERR_OUT_OF_MEMORY;
    p->device = scope.device();
    p->pages = static_cast<int>(pages);
    p->page_size = page_size;
    p->requests = requests;
    p->columns = columns;
    // amounts, two lists of pages, one number; fork: a table and its counts.  No call reads what another left.
    const size_t own = static_cast<size_t>(requests) + 2 * static_cast<size_t>(pages) + 1;
    const size_t fork = static_cast<size_t>(requests) * (static_cast<size_t>(columns) + 1);
    const cudaError_t e = cudaMalloc(&p->work, sizeof(int) * std::max(own, fork));
    if (e != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return q8i::cuda_status(e);
    }
    *out = p;
    return Q8MV_OK;
}

q8mv_status_t kvpage_extend(kvpage_plan_t plan, const kvpage_state_t *state, const int32_t *lengths,
                            const int32_t *tokens, int32_t width, int64_t *slots, int32_t *src, int32_t *dst,
                            int32_t *ok, cudaStream_t stream) {
    kv::PageParams p = {};
    if (!kv::take(plan, state, &p) || width < 0) return Q8MV_ERR_INVALID_ARG;
    if (!lengths || !tokens || !src || !dst || !ok || (width > 0 && !slots)) return Q8MV_ERR_INVALID_ARG;
    if (!kv::aligned(lengths, 4) || !kv::aligned(tokens, 4) || !kv::aligned(src, 4) || !kv::aligned(dst, 4) ||
        !kv::aligned(ok, 4) || !kv::aligned(slots, 8))
        return Q8MV_ERR_INVALID_ARG;
    p.lengths = lengths;
    p.tokens = tokens;
    p.width = width;
    p.slots = slots;
    p.src = src;
    p.dst = dst;
    p.ok = ok;
    p.slots_here = width <= 64;
    const q8mv_status_t st = kv::launch_cluster(kv::kvpage_extend_kernel, p, 16384, stream);
    if (st != Q8MV_OK || p.slots_here) return st;
    kv::kvpage_slots_kernel<<<dim3(static_cast<unsigned>(kv::ceil_div(width, 256)), static_cast<unsigned>(p.requests)), 256, 0,
                              stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t kvpage_fork(kvpage_plan_t plan, const kvpage_state_t *state, const int32_t *parents, cudaStream_t stream) {
    kv::PageParams p = {};
    if (!kv::take(plan, state, &p) || !parents || !kv::aligned(parents, 4)) return Q8MV_ERR_INVALID_ARG;
    int *count = plan->work, *rows = count + p.requests;
    kv::kvpage_fork_read_kernel<<<p.requests, 256, 0, stream>>>(p, parents, rows, count);
    kv::kvpage_fork_write_kernel<<<p.requests, 256, 0, stream>>>(p, parents, rows, count);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t kvpage_free(kvpage_plan_t plan, const kvpage_state_t *state, const int32_t *lengths, cudaStream_t stream) {
    kv::PageParams p = {};
    if (!kv::take(plan, state, &p) || !lengths || !kv::aligned(lengths, 4)) return Q8MV_ERR_INVALID_ARG;
    p.lengths = lengths;
    kv::kvpage_free_kernel<<<p.requests, 256, 0, stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t kvpage_compact(kvpage_plan_t plan, const kvpage_state_t *state, int32_t *src, int32_t *dst, int32_t *count,
                             cudaStream_t stream) {
    kv::PageParams p = {};
    if (!kv::take(plan, state, &p) || !count || !kv::aligned(count, 4)) return Q8MV_ERR_INVALID_ARG;
    if (p.pages >= 2 && (!src || !dst || !kv::aligned(src, 4) || !kv::aligned(dst, 4))) return Q8MV_ERR_INVALID_ARG;
    p.src = src;
    p.dst = dst;
    p.count = count;
    const q8mv_status_t st = kv::launch_cluster(kv::kvpage_compact_kernel, p, 4096, stream);
    if (st != Q8MV_OK) return st;
    kv::kvpage_follow_kernel<<<dim3(static_cast<unsigned>(kv::ceil_div(p.columns, 256)), static_cast<unsigned>(p.requests)), 256,
                               0, stream>>>(p);
    return q8i::cuda_status(cudaGetLastError());
}

q8mv_status_t kvpage_destroy(kvpage_plan_t p) {
    if (p == nullptr) return Q8MV_OK;
    kv::DeviceScope scope;
    q8mv_status_t st = scope.enter(p->device);
    if (st == Q8MV_OK) st = q8i::cuda_status(cudaDeviceSynchronize());
    if (p->work) cudaFree(p->work);
    delete p;
    return st;
}

q8mv_status_t kvpage_copy_q8(const q8kv_cache_t *cache, int64_t n, const int32_t *src, const int32_t *dst,
                             const int32_t *count, cudaStream_t stream) {
    kv::Cache c;
    if (!kv::make_cache(cache, &c)) return Q8MV_ERR_INVALID_ARG;
    return kv::copy_pages(c, n, src, dst, count, stream);
}

q8mv_status_t kvpage_copy_q4(const q4kv_cache_t *cache, int64_t n, const int32_t *src, const int32_t *dst,
                             const int32_t *count, cudaStream_t stream) {
    kv::Cache4 c = {};
    if (!kv::make_cache4(cache, &c)) return Q8MV_ERR_INVALID_ARG;
    return kv::copy_pages(c.rows, n, src, dst, count, stream);
}

}  // extern "C"
