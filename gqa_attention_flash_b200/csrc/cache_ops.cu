// cache_ops.cu -- operators on a paged KV cache: rows written to its pages and moved
// inside them, pages copied, and the tables' bookkeeping (fork, extend, free).
//
// The cache is the one attn_decode_paged reads: pools (num_blocks, block_size, Hkv, D)
// and tables int32 (R, max_blocks), row r of which names the pages of sequence r in
// order (-1: no page).  The bookkeeping's state is ref_counts int32 (num_blocks): how
// many table entries name a page.  A page is free when its count is 0, and the lowest
// free pages are handed out first, so every result is a function of the inputs alone.
//
// All kernels are launched with programmatic dependent launch and wait for their
// predecessor before the first global access.
#include <cuda_bf16.h>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace gqa {

namespace {

__device__ __forceinline__ void pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
attn_status_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess ? ATTN_OK
                                                                                      : ATTN_ERR_CUDA;
}

// Pool row of position `pos` of the sequence whose table row is `bt`, or -1 (no page,
// or a page outside the pool).
template <class Params>
__device__ __forceinline__ long long pool_row(const Params &q, const int32_t *bt, int pos) {
    const int shift = q.shift, num_blocks = q.num_blocks;
    // checked build: the entry lies in the sequence's table row
    if (!in_range(pos >= 0 && (pos >> shift) < q.max_blocks, q.status, nullptr)) return -1;
    const int p = bt[pos >> shift];
    return p >= 0 && p < num_blocks ? ((long long)p << shift) + (pos & ((1 << shift) - 1)) : -1;
}

// ---------------------------------------------------------------------------------
// append: row t of sequence b to position start[b] + t
// ---------------------------------------------------------------------------------
// A thread moves kAppendUnroll x 16 bytes of K and of V, all loads in flight at once.  The
// source's innermost axes are (t, d), so a warp reads consecutive bytes and writes whole
// rows of one head (2 D bytes each).
constexpr int kAppendThreads = 128;
constexpr int kAppendUnroll = 4;

struct AppendParams {
    uint4 *K, *V;
    const uint4 *Kn, *Vn;
    const int32_t *tables, *start, *n_new;
    int B, Hkv, T, vec, max_blocks, shift, num_blocks, chunks;  // vec: 16-byte words per head row
    long long capacity;
    int *status;
};

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
    pdl_wait();
    const int chunk = static_cast<int>(blockIdx.x % p.chunks);
    const long long bh = blockIdx.x / p.chunks;
    const int h = static_cast<int>(bh % p.Hkv), b = static_cast<int>(bh / p.Hkv);
    int n = p.T;
    if (p.n_new) {
        n = p.n_new[b];
        if (n > p.T) {
            record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            n = p.T;
        }
    }
    const long long start = p.start[b];
    const int32_t *bt = p.tables + (long long)b * p.max_blocks;
    uint4 k[kAppendUnroll], v[kAppendUnroll];
    long long dst[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
        const long long idx =
            ((long long)chunk * kAppendUnroll + u) * kAppendThreads + threadIdx.x;
        const int t = static_cast<int>(idx / p.vec), c = static_cast<int>(idx % p.vec);
        dst[u] = -1;
        if (t >= n) continue;
        const long long pos = start + t;
        long long row = -1;
        if (pos >= 0 && pos < p.capacity) row = pool_row(p, bt, static_cast<int>(pos));
        if (row < 0) {
            record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            continue;
        }
        const long long src = (bh * p.T + t) * p.vec + c, to = (row * p.Hkv + h) * p.vec + c;
        // checked build: both rows lie inside their tensors
        if (!in_range(t < p.T && src < (long long)p.B * p.Hkv * p.T * p.vec &&
                          to < ((long long)p.num_blocks << p.shift) * p.Hkv * p.vec,
                      p.status, nullptr))
            continue;
        k[u] = p.Kn[src];
        v[u] = p.Vn[src];
        dst[u] = to;
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u)
        if (dst[u] >= 0) {
            p.K[dst[u]] = k[u];
            p.V[dst[u]] = v[u];
        }
}

// ---------------------------------------------------------------------------------
// compact: position base[b] + k takes the row of position base[b] + keep[b][k]
// ---------------------------------------------------------------------------------
// In place.  keep is ascending, so keep[k] >= k: a row that step k writes is the source
// of no later step, and a block may move its slice of the columns in steps of kStep rows
// (read the step, wait for the block, write it), with nothing but its own order to keep; a
// step may even be read before the one before it is written.  So two steps are in flight,
// their rows looked up in shared memory (B4, half of 2048 to 4096 rows of 2 KB kept:
// 35 us with one step of 128 rows in flight and the lookups in its way, 17 us with two of
// 256, 12 us with two of 512).
constexpr int kCompactThreads = 256;
constexpr int kSliceVec = 4;                                  // 16-byte words of a row per block
constexpr int kStepRows = kCompactThreads / kSliceVec;        // rows per pass of the block
constexpr int kPasses = 8;
constexpr int kStep = kStepRows * kPasses;
constexpr int kCompactList = 2048;                            // rows looked up at a time

struct CompactParams {
    uint4 *K, *V;
    const int32_t *tables, *base, *keep, *n_keep;
    int A, row_vec, slices, max_blocks, shift, num_blocks;  // row_vec: 16-byte words per token
    long long capacity;
    int *status;
};

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p) {
    __shared__ int rows_from[kCompactList], rows_to[kCompactList];
    pdl_wait();
    const int slice = static_cast<int>(blockIdx.x % p.slices);
    const int b = static_cast<int>(blockIdx.x / p.slices);
    uint4 *pool = blockIdx.y ? p.V : p.K;
    const bool report = slice == 0 && blockIdx.y == 0 && threadIdx.x == 0;
    const int32_t *bt = p.tables + (long long)b * p.max_blocks;
    const int32_t *keep = p.keep + (long long)b * p.A;
    const long long base = p.base[b];
    int n = p.A;
    if (p.n_keep) {
        n = p.n_keep[b];
        if (n > p.A) {
            if (report) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            n = p.A;
        }
    }
    if (n <= 0) return;
    // The whole list is checked first: ascending, inside the table, on pages of the pool.
    // Four entries per thread and step, so that their lookups overlap.
    bool bad = base < 0;
    for (int k0 = threadIdx.x; k0 < n; k0 += 4 * kCompactThreads) {
        int x[4], before[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + i * kCompactThreads;
            x[i] = k < n ? keep[k] : 0;
            before[i] = k < n && k > 0 ? keep[k - 1] : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + i * kCompactThreads;
            if (k >= n) continue;
            // (an entry that passes has k <= x, so both positions lie in the table)
            const bool fits = base >= 0 && x[i] > before[i] && x[i] >= k && base + x[i] < p.capacity;
            const long long from =
                fits ? pool_row(p, bt, static_cast<int>(base + x[i])) : -1;
            const long long to = fits ? pool_row(p, bt, static_cast<int>(base + k)) : -1;
            bad = bad || from < 0 || to < 0;
            if (k < kCompactList) {
                rows_from[k] = static_cast<int>(from);
                rows_to[k] = static_cast<int>(to);
            }
        }
    }
    if (__syncthreads_or(bad)) {
        if (report) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    const int col = slice * kSliceVec + threadIdx.x % kSliceVec;
    const int r = threadIdx.x / kSliceVec;
    for (int l0 = 0; l0 < n; l0 += kCompactList) {
        const int m = min(n - l0, kCompactList);  // rows l0 .. l0 + m - 1 of the list
        if (l0 > 0) __syncthreads();  // the first rows are there from the check
        for (int k = threadIdx.x; k < m && l0 > 0; k += kCompactThreads) {
            rows_from[k] = static_cast<int>(pool_row(p, bt, static_cast<int>(base + keep[l0 + k])));
            rows_to[k] = static_cast<int>(pool_row(p, bt, static_cast<int>(base + l0 + k)));
        }
        if (l0 > 0) __syncthreads();
        uint4 v[2][kPasses];
        // checked build: row k of the list is one of the pool's
        auto ok = [&](const int *rows, int k) -> bool {
            return in_range(k < kCompactList && rows[k] >= 0 &&
                                rows[k] < ((long long)p.num_blocks << p.shift),
                            p.status, nullptr);
        };
        auto read = [&](uint4 (&x)[kPasses], int k0) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int k = k0 + i * kStepRows + r;
                if (k < m && col < p.row_vec && ok(rows_from, k)) x[i] = pool[(long long)rows_from[k] * p.row_vec + col];
            }
        };
        auto write = [&](const uint4 (&x)[kPasses], int k0) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int k = k0 + i * kStepRows + r;
                if (k < m && col < p.row_vec && ok(rows_to, k)) pool[(long long)rows_to[k] * p.row_vec + col] = x[i];
            }
        };
        read(v[0], 0);
        for (int k0 = 0; k0 < m; k0 += 2 * kStep) {
            read(v[1], k0 + kStep);
            __syncthreads();  // every read of step k0 is done
            write(v[0], k0);
            read(v[0], k0 + 2 * kStep);
            __syncthreads();
            write(v[1], k0 + kStep);
        }
    }
}

// ---------------------------------------------------------------------------------
// copy_blocks: page dst[i] takes the contents of page src[i]
// ---------------------------------------------------------------------------------
// Every block first looks through the list: a pair whose source is another pair's
// destination, or whose destination a later pair names too, is skipped and flagged, so
// the copies that run do not meet and the result does not depend on their order.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

__global__ void __launch_bounds__(kCopyThreads)
    copy_blocks_kernel(uint4 *K, uint4 *V, const int32_t *src, const int32_t *dst, int n, int num_blocks,
                       long long page_vec, int chunks, int *status) {
    pdl_wait();
    const int i = static_cast<int>(blockIdx.x / chunks), chunk = static_cast<int>(blockIdx.x % chunks);
    const int s = src[i], d = dst[i];
    if (s < 0 || d < 0) return;  // no pair
    bool bad = s >= num_blocks || d >= num_blocks;
    for (int j = threadIdx.x; j < n && !bad; j += kCopyThreads)
        if (j != i && src[j] >= 0) bad = dst[j] == s || (j > i && dst[j] == d);
    if (__syncthreads_or(bad)) {
        if (chunk == 0 && threadIdx.x == 0) record_status(status, ATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    if (s == d) return;
    // checked build: both are pages of the pool
    if (!in_range(i < n && s < num_blocks && d < num_blocks, status, nullptr)) return;
    const long long at = (long long)chunk * kCopyThreads * kCopyUnroll + threadIdx.x;
    uint4 k[kCopyUnroll], v[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const long long x = at + u * kCopyThreads;
        if (x < page_vec) {
            k[u] = K[s * page_vec + x];
            v[u] = V[s * page_vec + x];
        }
    }
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const long long x = at + u * kCopyThreads;
        if (x < page_vec) {
            K[d * page_vec + x] = k[u];
            V[d * page_vec + x] = v[u];
        }
    }
}

// ---------------------------------------------------------------------------------
// free: table entries [first, last) of the named rows
// ---------------------------------------------------------------------------------
constexpr int kTableThreads = 256;

__global__ void __launch_bounds__(kTableThreads)
    free_kernel(int32_t *tables, int32_t *refs, const int32_t *rows, const int32_t *first,
                const int32_t *last, int R, int max_blocks, int num_blocks, int chunks, int *status) {
    pdl_wait();
    const int n = static_cast<int>(blockIdx.x / chunks), chunk = static_cast<int>(blockIdx.x % chunks);
    const int row = rows[n];
    if (row < 0) return;
    if (row >= R) {
        if (chunk == 0 && threadIdx.x == 0) record_status(status, ATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    const int k = chunk * kTableThreads + threadIdx.x;
    if (k < first[n] || k >= last[n] || k >= max_blocks) return;
    // checked build: the entry is one of the table's
    if (!in_range(k >= 0 && row < R, status, nullptr)) return;
    // taken out of the table at once, so that an entry named twice is given back once
    const int page = atomicExch(&tables[(long long)row * max_blocks + k], -1);
    if (page < 0) return;
    if (page >= num_blocks) {
        record_status(status, ATTN_ERR_DEVICE_BOUNDS);
        return;
    }
    if (!in_range(page >= 0 && page < num_blocks, status, nullptr)) return;
    if (atomicSub(&refs[page], 1) <= 0) {  // not held: put the count back
        atomicAdd(&refs[page], 1);
        record_status(status, ATTN_ERR_DEVICE_BOUNDS);
    }
}

// ---------------------------------------------------------------------------------
// fork, first half: children's rows from their parents', shared pages counted
// ---------------------------------------------------------------------------------
// copy_src[n] is left at the parent's part-filled page (-1: none, or no such pair); the
// second half gives the child a page of its own for it.
struct ForkParams {
    int32_t *tables, *refs, *lens;
    const int32_t *parents, *children;
    int32_t *copy_src, *copy_dst;
    int N, R, max_blocks, num_blocks, shift, chunks;
    int *status;
};

__device__ __forceinline__ int fork_len(const ForkParams &p, int row, bool report) {
    const long long cap = (long long)p.max_blocks << p.shift;
    const int len = p.lens[row];
    if (len >= 0 && len <= cap) return len;
    if (report) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
    return len < 0 ? 0 : static_cast<int>(cap);
}

__global__ void __launch_bounds__(kTableThreads) fork_kernel(const ForkParams p) {
    pdl_wait();
    const int n = static_cast<int>(blockIdx.x / p.chunks), chunk = static_cast<int>(blockIdx.x % p.chunks);
    const bool report = chunk == 0 && threadIdx.x == 0;
    const int par = p.parents[n], chi = p.children[n];
    bool bad = par >= p.R || chi >= p.R || par == chi;
    const bool none = par < 0 || chi < 0;
    for (int j = threadIdx.x; j < p.N && !bad && !none; j += kTableThreads)
        if (p.parents[j] >= 0 && p.children[j] >= 0)
            bad = p.parents[j] == chi || (j < n && p.children[j] == chi);
    bad = __syncthreads_or(bad);
    if (none || bad) {
        if (report) {
            p.copy_src[n] = -1;
            if (!none) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        }
        return;
    }
    const int len = fork_len(p, par, report);
    const int full = len >> p.shift;
    const bool part = len & ((1 << p.shift) - 1);
    // checked build: both rows are the table's, and the part-filled page's entry is the row's
    if (!in_range(n < p.N && par >= 0 && par < p.R && chi >= 0 && chi < p.R && full <= p.max_blocks &&
                      (!part || full < p.max_blocks),
                  p.status, nullptr))
        return;
    const int32_t *from = p.tables + (long long)par * p.max_blocks;
    int32_t *to = p.tables + (long long)chi * p.max_blocks;
    const int k = chunk * kTableThreads + threadIdx.x;
    if (k < p.max_blocks) {
        int page = k < full ? from[k] : -1;
        if (page >= p.num_blocks) {
            record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            page = -1;
        }
        if (page >= 0 && in_range(page < p.num_blocks, p.status, nullptr)) atomicAdd(&p.refs[page], 1);
        to[k] = page;
    }
    if (report) {
        int page = part ? from[full] : -1;
        if (page >= p.num_blocks) {
            record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            page = -1;
        }
        p.copy_src[n] = page < 0 ? -1 : page;
        p.lens[chi] = len;
    }
}

// ---------------------------------------------------------------------------------
// Handing out pages: fork's second half and extend
// ---------------------------------------------------------------------------------
constexpr int kAllocThreads = 1024;

// No page left.  A length out of range that was recorded before (a clamp) does not hide it:
// the caller has to act on missing pages.
__device__ __forceinline__ void record_no_pages(int *status) {
    if (atomicCAS(status, 0, ATTN_ERR_NO_PAGES) == ATTN_ERR_DEVICE_BOUNDS)
        atomicCAS(status, ATTN_ERR_DEVICE_BOUNDS, ATTN_ERR_NO_PAGES);
}

// Exclusive sum over the block; `total` gets the whole sum.
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// The first `need` free pages, in increasing order, into `list`; returns how many there
// are (at most `need`).  Whole block.
// checked build: `room` is the length of `list`.
__device__ int free_pages(const int32_t *refs, int num_blocks, int need, int32_t *list, long long room,
                          int *warp_sums, int *status) {
    constexpr int kPer = 16;
    int found = 0;
    for (long long at = 0; at < num_blocks && found < need; at += kAllocThreads * kPer) {
        const long long first = at + threadIdx.x * kPer;
        uint32_t free_mask = 0;
#pragma unroll
        for (int q = 0; q < kPer / 4; ++q) {
            const long long x = first + 4 * q;
            if (x + 4 <= num_blocks) {
                const int4 r = *reinterpret_cast<const int4 *>(refs + x);
                free_mask |= ((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << (4 * q);
            } else {
                for (int e = 0; e < 4; ++e)
                    if (x + e < num_blocks && refs[x + e] == 0) free_mask |= 1u << (4 * q + e);
            }
        }
        int total;
        int rank = found + block_exclusive(__popc(free_mask), warp_sums, total);
        while (free_mask && rank < need && in_range(rank < room, status, nullptr)) {
            list[rank++] = static_cast<int32_t>(first) + __ffs(free_mask) - 1;
            free_mask &= free_mask - 1;
        }
        found += total;
    }
    __syncthreads();  // the list is complete, and refs[] may be written
    return min(found, need);
}

// fork, second half: the k-th pair with a part-filled page gets the k-th free page.
__global__ void __launch_bounds__(kAllocThreads) fork_alloc_kernel(const ForkParams p, int32_t *list) {
    __shared__ int warp_sums[32];
    pdl_wait();
    int need = 0;
    for (int n0 = 0; n0 < p.N; n0 += kAllocThreads) {
        const int n = n0 + threadIdx.x;
        int total;
        block_exclusive(n < p.N && p.copy_src[n] >= 0, warp_sums, total);
        need += total;
    }
    const int got = free_pages(p.refs, p.num_blocks, need, list, p.N, warp_sums, p.status);
    if (got < need && threadIdx.x == 0) record_no_pages(p.status);
    int before = 0;
    for (int n0 = 0; n0 < p.N; n0 += kAllocThreads) {
        const int n = n0 + threadIdx.x;
        const bool mine = n < p.N && p.copy_src[n] >= 0;
        int total;
        const int rank = before + block_exclusive(mine, warp_sums, total);
        before += total;
        if (n < p.N) {
            int page = -1;
            if (mine && rank < got) {
                page = list[rank];
                const int full = fork_len(p, p.parents[n], false) >> p.shift;
                // checked build: a page of the pool, an entry of the table
                if (!in_range(rank < p.N && page >= 0 && page < p.num_blocks && full < p.max_blocks &&
                                  p.children[n] >= 0 && p.children[n] < p.R,
                              p.status, nullptr))
                    continue;
                p.tables[(long long)p.children[n] * p.max_blocks + full] = page;
                p.refs[page] = 1;
            }
            p.copy_dst[n] = page;
            if (page < 0) p.copy_src[n] = -1;
        }
    }
}

// extend: every empty entry of row r from position from_lens[r]'s page to the last page
// that to_lens[r] tokens need gets a page, rows in order.
struct ExtendParams {
    int32_t *tables, *refs;
    const int32_t *from, *to;
    int32_t *offsets, *list;  // workspace: R + 1 and min(R * max_blocks, num_blocks)
    int R, max_blocks, num_blocks, shift;
    int *status;
    __device__ long long room() const { return min((long long)R * max_blocks, (long long)num_blocks); }
};

__device__ __forceinline__ void extend_range(const ExtendParams &p, int r, bool report, int &k0, int &k1) {
    const long long cap = (long long)p.max_blocks << p.shift;
    long long to = p.to[r];
    if (to > cap) {
        if (report) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        to = cap;
    }
    k0 = max(p.from[r], 0) >> p.shift;
    k1 = to > 0 ? static_cast<int>((to + (1 << p.shift) - 1) >> p.shift) : 0;
}

__global__ void __launch_bounds__(kAllocThreads) extend_kernel(const ExtendParams p) {
    __shared__ int warp_sums[32];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // empty entries of each row (a warp per row), then their exclusive sum over the rows
    for (int r = warp; r < p.R; r += kAllocThreads / 32) {
        int k0, k1, n = 0;
        extend_range(p, r, lane == 0, k0, k1);
        // checked build: the entries are the row's
        if (!in_range(k0 >= 0 && k1 <= p.max_blocks, p.status, nullptr)) k1 = k0;
        for (int k = k0 + lane; k < k1; k += 32) n += p.tables[(long long)r * p.max_blocks + k] < 0;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) p.offsets[r] = n;
    }
    __syncthreads();
    long long need_all = 0;
    for (int r0 = 0; r0 < p.R; r0 += kAllocThreads) {
        const int r = r0 + threadIdx.x;
        int total;
        const int off = block_exclusive(r < p.R ? p.offsets[r] : 0, warp_sums, total);
        if (r < p.R) p.offsets[r] = static_cast<int>(min(need_all + off, (long long)p.num_blocks));
        need_all += total;
    }
    const int need = static_cast<int>(min(need_all, (long long)p.num_blocks));
    if (need == 0) return;
    const int got = free_pages(p.refs, p.num_blocks, need, p.list, p.room(), warp_sums, p.status);
    if (got < need_all && threadIdx.x == 0) record_no_pages(p.status);
    for (int r = warp; r < p.R; r += kAllocThreads / 32) {
        int k0, k1;
        extend_range(p, r, false, k0, k1);
        if (!in_range(k0 >= 0 && k1 <= p.max_blocks, p.status, nullptr)) k1 = k0;
        int rank = p.offsets[r];
        for (int kb = k0; kb < k1; kb += 32) {
            const int k = kb + lane;
            int32_t *e = p.tables + (long long)r * p.max_blocks + k;
            const bool empty = k < k1 && *e < 0;
            const uint32_t vote = __ballot_sync(0xffffffffu, empty);
            const int mine = rank + __popc(vote & ((1u << lane) - 1u));
            if (empty && mine < got && in_range(mine < p.room(), p.status, nullptr)) {
                const int page = p.list[mine];
                if (in_range(page >= 0 && page < p.num_blocks, p.status, nullptr)) {
                    *e = page;
                    p.refs[page] = 1;
                }
            }
            rank += __popc(vote);
        }
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

}  // namespace

attn_status_t launch_cache_append(const CacheArgs &a, cudaStream_t stream) {
    AppendParams p;
    p.K = static_cast<uint4 *>(a.K);
    p.V = static_cast<uint4 *>(a.V);
    p.Kn = static_cast<const uint4 *>(a.K_new);
    p.Vn = static_cast<const uint4 *>(a.V_new);
    p.tables = a.block_tables;
    p.start = a.start;
    p.n_new = a.counts;
    p.B = a.B;
    p.Hkv = a.Hkv;
    p.T = a.T;
    p.vec = a.D / 8;
    p.max_blocks = a.max_blocks;
    p.shift = log2_of(a.block_size);
    p.num_blocks = a.num_blocks;
    p.capacity = (long long)a.max_blocks * a.block_size;
    p.status = device_status_word();
    if (!p.status) return ATTN_ERR_CUDA;
    constexpr int kPer = kAppendThreads * kAppendUnroll;
    const long long chunks = ((long long)a.T * p.vec + kPer - 1) / kPer;
    const long long grid = chunks * a.B * a.Hkv;
    if (grid > 0x7fffffffll) return ATTN_ERR_INVALID;
    p.chunks = static_cast<int>(chunks);
    return launch_pdl(append_kernel, dim3(static_cast<unsigned>(grid)), kAppendThreads, 0, stream, p);
}

attn_status_t launch_cache_compact(const CacheArgs &a, cudaStream_t stream) {
    CompactParams p;
    p.K = static_cast<uint4 *>(a.K);
    p.V = static_cast<uint4 *>(a.V);
    p.tables = a.block_tables;
    p.base = a.start;
    p.keep = a.keep;
    p.n_keep = a.counts;
    p.A = a.T;
    p.row_vec = a.Hkv * (a.D / 8);
    p.slices = (p.row_vec + kSliceVec - 1) / kSliceVec;
    p.max_blocks = a.max_blocks;
    p.shift = log2_of(a.block_size);
    p.num_blocks = a.num_blocks;
    p.capacity = (long long)a.max_blocks * a.block_size;
    p.status = device_status_word();
    if (!p.status) return ATTN_ERR_CUDA;
    const long long grid = (long long)p.slices * a.B;
    if (grid > 0x7fffffffll) return ATTN_ERR_INVALID;
    return launch_pdl(compact_kernel, dim3(static_cast<unsigned>(grid), 2), kCompactThreads, 0, stream, p);
}

attn_status_t launch_cache_copy(void *K, void *V, const int32_t *src, const int32_t *dst, int n,
                                int num_blocks, long long page_bytes, cudaStream_t stream) {
    int *status = device_status_word();
    if (!status) return ATTN_ERR_CUDA;
    const long long page_vec = page_bytes / 16;
    const long long chunks = (page_vec + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll);
    if (chunks * n > 0x7fffffffll) return ATTN_ERR_INVALID;
    return launch_pdl(copy_blocks_kernel, dim3(static_cast<unsigned>(chunks * n)), kCopyThreads, 0, stream,
                      static_cast<uint4 *>(K), static_cast<uint4 *>(V), src, dst, n, num_blocks, page_vec,
                      static_cast<int>(chunks), status);
}

attn_status_t launch_cache_free(int32_t *tables, int32_t *refs, const int32_t *rows, const int32_t *first,
                                const int32_t *last, int N, int R, int max_blocks, int num_blocks,
                                cudaStream_t stream) {
    int *status = device_status_word();
    if (!status) return ATTN_ERR_CUDA;
    const long long chunks = ((long long)max_blocks + kTableThreads - 1) / kTableThreads;
    if (chunks * N > 0x7fffffffll) return ATTN_ERR_INVALID;
    return launch_pdl(free_kernel, dim3(static_cast<unsigned>(chunks * N)), kTableThreads, 0, stream, tables,
                      refs, rows, first, last, R, max_blocks, num_blocks, static_cast<int>(chunks), status);
}

attn_status_t launch_cache_fork(const CacheForkArgs &a, cudaStream_t stream) {
    ForkParams p;
    p.tables = a.tables;
    p.refs = a.refs;
    p.lens = a.lens;
    p.parents = a.parents;
    p.children = a.children;
    p.copy_src = a.copy_src;
    p.copy_dst = a.copy_dst;
    p.N = a.N;
    p.R = a.R;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.shift = log2_of(a.block_size);
    p.status = device_status_word();
    if (!p.status) return ATTN_ERR_CUDA;
    const long long chunks = ((long long)a.max_blocks + kTableThreads - 1) / kTableThreads;
    if (chunks * a.N > 0x7fffffffll) return ATTN_ERR_INVALID;
    p.chunks = static_cast<int>(chunks);
    attn_status_t st = launch_pdl(fork_kernel, dim3(static_cast<unsigned>(chunks * a.N)), kTableThreads, 0,
                                  stream, p);
    if (st != ATTN_OK) return st;
    return launch_pdl(fork_alloc_kernel, dim3(1), kAllocThreads, 0, stream, p, a.workspace);
}

attn_status_t launch_cache_extend(const CacheExtendArgs &a, cudaStream_t stream) {
    ExtendParams p;
    p.tables = a.tables;
    p.refs = a.refs;
    p.from = a.from;
    p.to = a.to;
    p.offsets = a.workspace;
    p.list = a.workspace + a.R + 1;
    p.R = a.R;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.shift = log2_of(a.block_size);
    p.status = device_status_word();
    if (!p.status) return ATTN_ERR_CUDA;
    return launch_pdl(extend_kernel, dim3(1), kAllocThreads, 0, stream, p);
}

}  // namespace gqa
