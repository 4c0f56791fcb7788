// attn_tree.cu -- attention of a tree of drafted tokens over a paged KV cache (sm_100a).
//
// Speculative decoding checks T drafted tokens per sequence in one pass.  Their keys and
// values already stand in the sequence's pages behind its `ctx` committed tokens (draft i
// at position ctx + i).  Draft i continues draft parents[i] (< i) or, for -1, the context;
// it sees every key before ctx, itself and its ancestors:
//   O_i = softmax_j(<q_i, k_j> / sqrt(D)) V over j < ctx and j = ctx + a, a in anc(i).
//
// Rows.  The G T queries of a KV head (its G query heads, T drafts each) are consecutive
// rows of Q, so every K/V byte is read from HBM once for up to 256 of them.
// Up to 128 rows, one M = 128 tile (kTwo = false): the two softmax warpgroups take the even
// and the odd key tiles of the same rows and merge their states at the end, so that one's
// softmax overlaps the other's products.  Above, two tiles (kTwo) share every key tile, one
// warpgroup each; more rows take several passes.  Few rows leave most of the tile empty, but
// the time is HBM's: transposed products (keys as M, N = 64 rows) halve the tensor work of
// 64 rows and ran no faster (B64 x 16 drafts: 768 us against 732).
//
// Work.  The 128-key tiles of all (sequence, KV head, row pass) segments form a list that
// the CTAs share out in equal runs, so ragged lengths leave no SM idle and a single long
// sequence uses all of them.  A segment that ends up in several CTAs leaves partial states
// (max, sum, unnormalised O, fp32) in a workspace; tree_combine_kernel merges them.
// The (KV head, row pass) pairs run in lanes, one CTA each over the same runs: the heads'
// rows of a token are neighbours in HBM, and the passes' K / V are the same, so that what
// stands together is read together.
//
// 12 warps: 0-3 and 4-7 softmax (one row per thread = TMEM lane), 8 and 10 TMA producers,
// 9 MMA issuer, 11 idle; registers move from 8-11 to the softmax warps as in the forward.
// The producers gather K and V page by page into a ring of 128-row slots each; a lane per
// page copies min(block_size, 128) rows of one head in one 5-D TMA box whose shared-memory
// order is (8-row group, 64-column half, row, column): the 128-byte-swizzled operand layout
// with 8-row groups 1024 D / 64 bytes apart.
#include <cuda_bf16.h>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace gqa {

namespace {

constexpr int TM = 128;        // rows per tile (= TMEM lanes)
constexpr int TK = 128;        // keys per tile
constexpr int kTreeThreads = 384;
constexpr int kTreeRegs = 168;  // per thread at launch (checked on the host)
constexpr uint32_t kLoadRegs = 88, kSoftRegs = 208;
static_assert(128 * kLoadRegs + 256 * kSoftRegs <= kTreeThreads * kTreeRegs,
              "register split must use exactly the launch allocation");
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpLoadV = 10;
constexpr int kMaxDrafts = 256;

template <int D, bool kTwo>
struct TreeCfg {
    static constexpr int NQ = kTwo ? 2 : 1;          // resident row tiles
    static constexpr int RQ = TM;                    // rows of a Q tile
    static constexpr int NBOX = D / 64;
    static constexpr int TILE = TK * D * 2;          // one K, V or Q tile
    static constexpr int QTILE = RQ * D * 2;
    static constexpr int QBOX = RQ * 128;            // a Q tile's 64-column half
    static constexpr int GROUP = NBOX * 1024;        // 8 rows of a K or V tile
    // K and V slots, a ring each: every producer fills its own ring in order, so the parity
    // that it waits for is never ambiguous
    static constexpr int NS = (D == 128 ? 7 : 13) - NQ, NK = NS / 2, NV = NS - NK;
    static constexpr int ROWS = NQ * TM;             // rows of a segment
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = NQ * TILE;
    static constexpr int OFF_BAR = OFF_RING + NS * TILE;
    // full and empty: [NK] slots of K, then [NV] of V
    static constexpr int BAR_FULL = 0, BAR_EMPTY = NS, BAR_QFULL = 2 * NS, BAR_QFREE = 2 * NS + 1,
                         BAR_S = 2 * NS + 2, BAR_P = 2 * NS + 4, BAR_O = 2 * NS + 6,
                         N_BARS = 2 * NS + 8;
    static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;  // tmem, abort, first b, warp sums
    // exchange of the two halves' states, float [2][TM]; the run's start before that
    static constexpr int OFF_ML = OFF_MISC + 16;
    static constexpr int OFF_PAR = OFF_ML + (kTwo ? 128 : 2 * TM * 4);  // [2][kMaxDrafts] uint8
    static constexpr int SMEM = OFF_PAR + 2 * kMaxDrafts + 1024;
    static constexpr uint32_t TMEM_COLS = 512;
    __host__ __device__ static constexpr uint32_t s_col(int t) { return t * TK; }
    __host__ __device__ static constexpr uint32_t o_col(int t) { return 2 * TK + t * D; }
    // workspace floats of one partial: O, max, sum
    static constexpr int WS = ROWS * (D + 2);
};
static_assert(TreeCfg<128, false>::SMEM <= 232448 && TreeCfg<128, true>::SMEM <= 232448 &&
                  TreeCfg<64, false>::SMEM <= 232448 && TreeCfg<64, true>::SMEM <= 232448,
              "tree shared memory above 227 KB");

struct TreeParams {
    __nv_bfloat16 *O;
    float *ws;
    long long *before;  // workspace (B + 1): key tiles of one pair before each sequence, all of them
    const int32_t *tables, *ctx, *parents, *drafts;
    int B, Hq, Hkv, T, R, n_rt, max_blocks, num_blocks, shift, box_rows;
    // (KV head, row pass) pair q runs in lane q % lanes, as segment q / lanes of each
    // sequence; a lane's list of segs segments per sequence is cut into n_run runs, run k
    // of lane l being CTA k * lanes + l
    int lanes, segs, n_run;
    // checked build: the n-th partial is one of the workspace's; `row` is one of O's
    __device__ __forceinline__ bool slot_ok(long long n) const { return n >= 0 && n < 2ll * lanes * n_run; }
    __device__ __forceinline__ bool row_ok(long long row) const {
        return row >= 0 && row < (long long)B * Hq * T;
    }
    float scale_log2;
    uint64_t wait_limit_ns;
    int *status;
};

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, uint32_t bar, int x, int y,
                                            int z, int w, int v) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
        : "memory");
}

// Barrier 3 of the 256 softmax threads: true for all if `ok` is true for all.
__device__ __forceinline__ bool all_of_256(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 3, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(ok))
        : "memory");
    return r != 0;
}

// Lengths of sequence b, clamped to the table; key tiles it has (0 without a draft).
struct TreeLens {
    int ctx, drafts, nt;
};
__device__ __forceinline__ TreeLens tree_lens(const TreeParams &p, int b, bool report) {
    const long long cap = (long long)p.max_blocks << p.shift;
    long long ctx = p.ctx[b];
    long long d = p.drafts ? p.drafts[b] : p.T;
    if (ctx < 0 || d > p.T || ctx + d > cap) {
        if (report) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        ctx = max(0ll, min(ctx, cap));
        d = min(min(d, (long long)p.T), cap - ctx);
    }
    d = max(d, 0ll);
    TreeLens l;
    l.ctx = static_cast<int>(ctx);
    l.drafts = static_cast<int>(d);
    l.nt = d > 0 ? static_cast<int>((ctx + d + TK - 1) / TK) : 0;
    return l;
}

// Exclusive sum over a block's threads in thread order; `total` gets the whole sum.
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sums, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < n_warps; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    return before + x - v;
}

// One CTA's walk over its run [f, f_end) of the list of key tiles.
struct TreeWalk {
    long long f, f_end, f_first, pre;  // pre: tiles (of one head) of the sequences before b
    int b;
    TreeLens len;
    // current piece: tiles [t_a, t_b) of segment (b, hkv, rt)
    int hkv, rt, t_a, t_b;

    __device__ __forceinline__ bool next(const TreeParams &p) {
        if (f >= f_end) return false;
        const long long H = p.segs;
        while (f >= (pre + len.nt) * H) {
            pre += len.nt;
            len = tree_lens(p, ++b, false);
        }
        const long long rem = f - pre * H;
        const int seg = static_cast<int>(rem / len.nt);
        t_a = static_cast<int>(rem - (long long)seg * len.nt);
        const int q = seg * p.lanes + static_cast<int>(blockIdx.x % p.lanes);
        hkv = q / p.n_rt;
        rt = q - hkv * p.n_rt;
        t_b = static_cast<int>(min((long long)len.nt, t_a + f_end - f));
        f += t_b - t_a;
        return true;
    }
    __device__ __forceinline__ bool whole() const { return t_a == 0 && t_b == len.nt; }
    // partial slot: 2 c for the piece that opens the CTA's run, 2 c + 1 for one that closes it
    __device__ __forceinline__ int slot(int cta) const {
        return 2 * cta + (f - (t_b - t_a) == f_first ? 0 : 1);
    }
};

// Set-up shared by the kernels: barriers, this CTA's run of the list, TMEM.  False: the CTA
// has no work (nothing is allocated then).
template <class C>
__device__ __forceinline__ bool tree_setup(const TreeParams &p, uint8_t *smem, TreeWalk &w, uint32_t &tmem) {
    const uint32_t sbase = smem_u32(smem);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    int *abort_flag = reinterpret_cast<int *>(smem + C::OFF_MISC + 4);
    int *first_b = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);
    long long *first_pre = reinterpret_cast<long long *>(smem + C::OFF_ML);  // before the first piece
    long long *warp_sums = first_pre + 1;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::N_BARS; ++i)
            mbar_init(sbase + C::OFF_BAR + 8 * i, i == C::BAR_P || i == C::BAR_P + 1 ? TM : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int per = (p.B + kTreeThreads - 1) / kTreeThreads;
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
    long long mine = 0, total;
    for (int b = b0; b < b1; ++b) mine += tree_lens(p, b, blockIdx.x == 0).nt;
    const long long before = block_scan(mine, warp_sums, total);
    if (blockIdx.x == 0) {  // for the combine
        long long pre = before;
        for (int b = b0; b < b1; ++b) {
            p.before[b] = pre;
            pre += tree_lens(p, b, false).nt;
        }
        if (threadIdx.x == 0) p.before[p.B] = total;
    }
    const long long H = p.segs;
    const long long share = (total * H + p.n_run - 1) / p.n_run;
    w.f_first = w.f = blockIdx.x / p.lanes * share;
    w.f_end = min(total * H, w.f + share);
    if (w.f >= w.f_end) return false;
    if (before * H <= w.f && w.f < (before + mine) * H) {
        long long pre = before;
        int b = b0;
        for (;; ++b) {
            const int nt = tree_lens(p, b, false).nt;
            if (w.f < (pre + nt) * H) break;
            pre += nt;
        }
        *first_b = b;
        *first_pre = pre;
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *tmem_slot;
    w.b = *first_b;
    w.pre = *first_pre;
    w.len = tree_lens(p, w.b, false);
    __syncthreads();  // the exchange area is reused from here on
    return true;
}

template <class C>
__device__ __forceinline__ void tree_teardown(uint8_t *smem, uint32_t tmem) {
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    if (*abort_flag) drain_delay(2000000);  // let copies and MMAs in flight land
    tc_fence_before();
    __syncthreads();
    if ((threadIdx.x >> 5) == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Rows of tile t of the segment that exist.
template <class C>
__device__ __forceinline__ int tree_rows(const TreeParams &p, int rt, int t) {
    return min(C::RQ, p.R - (rt * C::NQ + t) * C::RQ);
}

// TMA producers: warp 8 copies the pieces' Q tiles and K, warp 10 V, page by page.  A box
// takes its warp about 28 ns to issue (the copy wants its operands in uniform registers, so
// the lanes take turns): with 16-token pages one warp for both would need 0.45 us for a
// 128-key tile, a third of the time its 64 KB take from HBM.
template <int D, class C>
__device__ __forceinline__ void tree_produce(const TreeParams &p, uint8_t *smem, TreeWalk &w,
                                             bool is_v, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                                             const CUtensorMap *tmV) {
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8 * i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        prefetch_tensormap(tmQ);
        prefetch_tensormap(tmK);
        prefetch_tensormap(tmV);
    }
    uint32_t g0 = 0;  // key tiles of the pieces before
    bool ok = true;
    for (int piece = 0; ok && w.next(p); ++piece) {
        const int32_t *bt = p.tables + (long long)w.b * p.max_blocks;
        const int n_keys = w.len.ctx + w.len.drafts;
        // page of this lane's chunk, read one tile ahead
        auto page_of = [&](int tile) -> int {
            const long long j = (long long)tile * TK + lane * p.box_rows;
            // checked build: the entry is one of the sequence's
            return lane * p.box_rows < TK && j < n_keys &&
                           in_range((j >> p.shift) < p.max_blocks, p.status, abort_flag)
                       ? bt[j >> p.shift]
                       : -1;
        };
        const int n = w.t_b - w.t_a;
        int page = page_of(w.t_a);
        for (int g = 0; ok && g < n; ++g) {
            const int tile = w.t_a + g;
            const uint32_t G = g0 + g;
            const int j = tile * TK + lane * p.box_rows;
            const bool mine = lane * p.box_rows < TK && j < n_keys;
            const int n_chunks = (min(TK, n_keys - tile * TK) + p.box_rows - 1) / p.box_rows;
            // a page outside the pool reads as zeros (a group past the tensor map)
            int group = p.num_blocks << (p.shift - 3);
            if (mine) {
                if (page >= 0 && page < p.num_blocks)
                    group = (page << (p.shift - 3)) + ((j & ((1 << p.shift) - 1)) >> 3);
                else
                    record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            }
            if (g + 1 < n) page = page_of(tile + 1);
            const uint32_t st = is_v ? C::NK + G % C::NV : G % C::NK, use = is_v ? G / C::NV : G / C::NK;
            if (use > 0)
                ok = warp_wait(bar(C::BAR_EMPTY + st), (use - 1) & 1, abort_flag, p.wait_limit_ns, p.status);
            // checked build: the chunks stay inside the slot and the head inside the pool
            ok = ok && in_range(n_chunks * p.box_rows <= TK && w.hkv < p.Hkv && w.b < p.B &&
                                    tile >= w.t_a && tile < w.t_b,
                                p.status, abort_flag);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(C::BAR_FULL + st), n_chunks * p.box_rows * D * 2);
            __syncwarp();
            if (mine)
                tma_load_5d(sbase + C::OFF_RING + st * C::TILE + lane * (p.box_rows >> 3) * C::GROUP,
                            is_v ? tmV : tmK, bar(C::BAR_FULL + st), 0, 0, 0, group, w.hkv);
            // Q after the piece's first K, which need not wait for its slot
            if (g == 0 && !is_v && lane == 0) {
                if (piece > 0 && !mbar_wait(bar(C::BAR_QFREE), (piece - 1) & 1, abort_flag, p.wait_limit_ns,
                                            p.status)) {
                    ok = false;
                } else if (!in_range(box_ok(0, w.rt * C::ROWS, w.b * p.Hkv + w.hkv, D, p.R,
                                            (long long)p.B * p.Hkv, C::RQ) &&
                                         w.rt * C::ROWS < p.R,
                                     p.status, abort_flag)) {
                    ok = false;  // checked build: the head's rows are not Q's
                } else {
                    const int n_q = C::NQ == 2 && tree_rows<C>(p, w.rt, 1) > 0 ? 2 : 1;
                    mbar_arrive_expect_tx(bar(C::BAR_QFULL), n_q * C::QTILE);
                    for (int t = 0; t < n_q; ++t)
                        for (int c = 0; c < C::NBOX; ++c)
                            tma_load_3d(sbase + C::OFF_Q + t * C::QTILE + c * C::QBOX, tmQ,
                                        bar(C::BAR_QFULL), c * 64, w.rt * C::ROWS + t * C::RQ,
                                        w.b * p.Hkv + w.hkv);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
        }
        g0 += n;
    }
}

template <int D, bool kTwo>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
    using C = TreeCfg<D, kTwo>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8 * i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TreeWalk w;
    uint32_t tmem;
    if (!tree_setup<C>(p, smem, w, tmem)) return;
    auto slot_addr = [&](uint32_t st) -> uint32_t { return sbase + C::OFF_RING + st * C::TILE; };
    auto rows_of = [&](int rt, int t) -> int { return tree_rows<C>(p, rt, t); };

    if (warp >= kWarpLoad) regs_dec<kLoadRegs>();
    if (warp == kWarpLoad || warp == kWarpLoadV) {
        tree_produce<D, C>(p, smem, w, warp == kWarpLoadV, &tmQ, &tmK, &tmV);
    } else if (warp == kWarpMma) {
        // ===================== MMA issuer =====================
        if (lane == 0) {
            constexpr uint32_t idS = idesc_bf16_f32(TM, TK, 0, 0);
            constexpr uint32_t idO = idesc_bf16_f32(TM, D, 0, 1);
            uint32_t g0 = 0, np0 = 0, np1 = 0;
            bool ok = true;
            for (int piece = 0; ok && w.next(p); ++piece) {
                const int n = w.t_b - w.t_a;
                const bool two = kTwo && rows_of(w.rt, 1) > 0;
                auto full = [&](uint32_t st, uint32_t use) -> bool {
                    return mbar_wait(bar(C::BAR_FULL + st), use & 1, abort_flag, p.wait_limit_ns, p.status);
                };
                // S = Q K^T of key tile g into buffer t, from row tile q
                auto issue_s = [&](int g, int t, int q, bool last_use) -> bool {
                    const uint32_t st = (g0 + g) % C::NK;
                    if (!full(st, (g0 + g) / C::NK)) return false;
                    tc_fence_after();
                    const uint32_t qa = sbase + C::OFF_Q + q * C::TILE, ka = slot_addr(st);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tmem + C::s_col(t),
                               smem_desc_sw128(qa + (kk >> 2) * C::QBOX + (kk & 3) * 32, 16, 1024),
                               smem_desc_sw128(ka + (kk >> 2) * 1024 + (kk & 3) * 32, 16, C::GROUP), idS,
                               kk > 0 ? 1u : 0u);
                    mma_commit(bar(C::BAR_S + t));
                    if (last_use) mma_commit(bar(C::BAR_EMPTY + st));
                    if (last_use && g == n - 1) mma_commit(bar(C::BAR_QFREE));
                    return true;
                };
                // O_t += P_t V of key tile g; `first` opens the accumulator, `last` closes it
                auto issue_pv = [&](int g, int t, bool first, bool last, bool last_use) -> bool {
                    const uint32_t st = C::NK + (g0 + g) % C::NV;
                    const uint32_t np = t ? np1++ : np0++;
                    if (!mbar_wait(bar(C::BAR_P + t), np & 1, abort_flag, p.wait_limit_ns, p.status) ||
                        !full(st, (g0 + g) / C::NV))
                        return false;
                    tc_fence_after();
                    const uint32_t va = slot_addr(st);
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk)
                        mma_ts(tmem + C::o_col(t), tmem + C::s_col(t) + kk * 8,
                               smem_desc_sw128(va + kk * 2 * C::GROUP, 1024, C::GROUP), idO,
                               !first || kk > 0 ? 1u : 0u);
                    if (last) mma_commit(bar(C::BAR_O + t));
                    if (last_use) mma_commit(bar(C::BAR_EMPTY + st));
                    return true;
                };
                ok = mbar_wait(bar(C::BAR_QFULL), piece & 1, abort_flag, p.wait_limit_ns, p.status);
                if constexpr (!kTwo) {
                    ok = ok && issue_s(0, 0, 0, true) && (n < 2 || issue_s(1, 1, 0, true));
                    for (int g = 0; ok && g < n; ++g) {
                        ok = issue_pv(g, g & 1, g < 2, g + 2 >= n, true);
                        if (ok && g + 2 < n) ok = issue_s(g + 2, g & 1, 0, true);
                    }
                } else {
                    ok = ok && issue_s(0, 0, 0, !two) && (!two || issue_s(0, 1, 1, true));
                    for (int g = 0; ok && g < n; ++g) {
                        const bool last = g == n - 1;
                        ok = issue_pv(g, 0, g == 0, last, !two) && (last || issue_s(g + 1, 0, 0, !two));
                        if (two)
                            ok = ok && issue_pv(g, 1, g == 0, last, true) &&
                                 (last || issue_s(g + 1, 1, 1, true));
                    }
                }
                g0 += n;
            }
        }
    } else if (warp < kWarpLoad) {
        // ===================== softmax and epilogue =====================
        regs_inc<kSoftRegs>();
        const int t = warp >> 2, r = threadIdx.x & (TM - 1);
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_addr = trow + (t ? C::s_col(1) : C::s_col(0));
        const uint32_t o_addr = trow + (t ? C::o_col(1) : C::o_col(0));
        float *ml = reinterpret_cast<float *>(smem + C::OFF_ML);
        uint8_t *par = smem + C::OFF_PAR + t * kMaxDrafts;
        uint32_t n_s = 0, n_o = 0, g0 = 0;  // S tiles, accumulators and key tiles so far
        bool ok = true;
        while (ok && w.next(p)) {
            const int ctx = w.len.ctx, n_keys = ctx + w.len.drafts;
            const int row0 = (w.rt * C::NQ + (kTwo ? t : 0)) * TM;  // of the segment's R rows
            const int row = row0 + r;
            const int draft = row % p.T;
            const bool have_rows = row0 + (warp & 3) * 32 < p.R;  // this warp
            const bool two = kTwo && rows_of(w.rt, 1) > 0;
            const int n = w.t_b - w.t_a;
            // key tiles of this warpgroup: t_a + first, step apart
            const int first = kTwo ? 0 : t, step = kTwo ? 1 : 2;
            const int n_iter = kTwo ? (t == 0 || two ? n : 0) : (n - t + 1) / 2;
            if (n_iter > 0 && (long long)w.t_b * TK > ctx) {
                // the tree: a parent per draft, 255 = the context
                for (int i = r; i < w.len.drafts; i += TM) {
                    // checked build: the parent is one of the sequence's
                    if (!in_range(w.b < p.B && i < p.T, p.status, abort_flag)) break;
                    const int up = p.parents[(long long)w.b * p.T + i];
                    const bool good = up >= -1 && up < i;
                    if (!good) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
                    par[i] = static_cast<uint8_t>(good && up >= 0 ? up : 255);
                }
                if (t == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
                else asm volatile("bar.sync 2, 128;" ::: "memory");
            }
            float m_used = ninf(), l = 0.f;
            for (int i = 0; i < n_iter; ++i) {
                const int g = first + i * step;
                const int kv0 = (w.t_a + g) * TK;
                if (!warp_wait(bar(C::BAR_S + t), (n_s + i) & 1, abort_flag, p.wait_limit_ns, p.status)) {
                    ok = false;
                    break;
                }
                // V rows past the keys may hold anything; their weights are 0, but 0 * NaN is
                // NaN, so this tile's (first) warpgroup zeroes them
                if (kv0 + TK > n_keys && (!kTwo || t == 0)) {
                    const uint32_t st = C::NK + (g0 + g) % C::NV;
                    if (!warp_wait(bar(C::BAR_FULL + st), ((g0 + g) / C::NV) & 1, abort_flag,
                                   p.wait_limit_ns, p.status)) {
                        ok = false;
                        break;
                    }
                    if (kv0 + r >= n_keys) {
                        uint8_t *v = smem + C::OFF_RING + st * C::TILE + (r >> 3) * C::GROUP +
                                     (r & 7) * 128;
#pragma unroll
                        for (int c = 0; c < C::NBOX; ++c)
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                reinterpret_cast<uint4 *>(v + c * 1024)[k] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (have_rows) {
                    tc_fence_after();
                    uint32_t sr[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, sr[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 4; ++c) reg_fence32(sr[c]);
                    float *s = reinterpret_cast<float *>(&sr[0][0]);
                    if (kv0 + TK > ctx) {
                        // one bit per key: the context, then this draft and its ancestors
                        const int c0 = ctx - kv0;  // column of draft 0
                        uint32_t vm[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int below = min(max(c0 - 32 * q, 0), 32);
                            vm[q] = below >= 32 ? 0xffffffffu : (1u << below) - 1u;
                        }
                        for (int a = draft < w.len.drafts ? draft : -1; a >= 0 && a + c0 >= 0;) {
                            const int c = a + c0;
                            const uint32_t bit = 1u << (c & 31);
#pragma unroll
                            for (int q = 0; q < 4; ++q) vm[q] |= (c >> 5) == q ? bit : 0u;
                            a = par[a] == 255 ? -1 : par[a];
                        }
#pragma unroll
                        for (int c = 0; c < TK; ++c)
                            s[c] = ((vm[c >> 5] >> (c & 31)) & 1u) ? s[c] : ninf();
                    }
                    // online softmax in the exp2 domain, O rescaled only when the max grew by
                    // more than 2^8 (fp32 sums and bf16 weights relative to the kept max)
                    float mx0 = s[0], mx1 = s[1];
#pragma unroll
                    for (int c = 2; c < TK; c += 2) {
                        mx0 = fmaxf(mx0, s[c]);
                        mx1 = fmaxf(mx1, s[c + 1]);
                    }
                    const float m_new = fmaxf(mx0, mx1) * p.scale_log2;
                    float alpha = 1.f;
                    bool resc = false;
                    if (m_new > m_used + 8.f) {
                        alpha = fast_exp2(m_used - m_new);
                        m_used = m_new;
                        resc = true;
                    }
                    const float neg_m = m_used == ninf() ? 0.f : -m_used;
                    const uint64_t sl2 = f2_pack(p.scale_log2, p.scale_log2), nm2 = f2_pack(neg_m, neg_m);
                    uint64_t sum2 = f2_pack(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float x0, x1;
                            f2_unpack(f2_fma(f2_pack(s[c * 32 + 2 * k], s[c * 32 + 2 * k + 1]), sl2, nm2),
                                      x0, x1);
                            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                            sum2 = f2_add(sum2, f2_pack(p0, p1));
                            pk[k] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(s_addr + c * 16, pk);
                    }
                    float sum0, sum1;
                    f2_unpack(sum2, sum0, sum1);
                    l = l * alpha + (sum0 + sum1);
                    // S of this tile being complete, so is the P V before it: O is quiet
                    if (i > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t v[32];
                            tmem_ld32(o_addr + c * 32, v);
                            tmem_wait_ld();
                            reg_fence32(v);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
                            tmem_st32(o_addr + c * 32, v);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                mbar_arrive(bar(C::BAR_P + t));
            }
            // ---- the piece's rows: O_t of this warpgroup, or both halves merged ----
            if (ok && n_iter > 0) {
                ok = warp_wait(bar(C::BAR_O + t), n_o & 1, abort_flag, p.wait_limit_ns, p.status);
                ++n_o;
            }
            n_s += n_iter;
            g0 += n;
            float a0 = 1.f, a1 = 0.f, m = m_used;  // factors of O_0 and O_1 for this row
            int c_lo = 0, c_hi = D / 32;            // 32-column chunks this warpgroup writes
            const bool whole = w.whole();
            if constexpr (!kTwo) {
                // warpgroup 1 hands over its max and sum, warpgroup 0 hands back the factors
                if (t == 1) {
                    ml[r] = m_used;
                    ml[TM + r] = l;
                }
                tc_fence_before();
                asm volatile("bar.sync 3, 256;" ::: "memory");
                if (t == 0) {
                    const float m1 = ml[r];
                    m = fmaxf(m_used, m1);
                    const float base = m == ninf() ? 0.f : m;
                    a0 = fast_exp2(m_used - base);
                    a1 = fast_exp2(m1 - base);
                    l = a0 * l + a1 * ml[TM + r];
                }
            }
            // a whole segment's factors carry 1 / sum; -1 marks a row that is zero (a sum that
            // is NaN reaches the row)
            if (whole && (kTwo || t == 0)) {
                const bool some = l != 0.f && draft < w.len.drafts;
                a0 = some ? a0 / l : -1.f;
                a1 = some ? a1 / l : -1.f;
            }
            if constexpr (!kTwo) {
                if (t == 0) {
                    ml[r] = a0;
                    ml[TM + r] = a1;
                }
                asm volatile("bar.sync 3, 256;" ::: "memory");
                a0 = ml[r];
                a1 = ml[TM + r];
                c_lo = t * (D / 64);
                c_hi = c_lo + D / 64;
            }
            bool write = row < p.R && (!kTwo || n_iter > 0);
            const bool use1 = !kTwo && n > 1, zero = a0 < 0.f;
            const long long orow = (long long)(w.b * p.Hq + w.hkv * (p.Hq / p.Hkv)) * p.T + row;
            float *part = p.ws + (long long)w.slot(blockIdx.x) * C::WS;
            const int prow = (kTwo ? t * TM : 0) + r;
            // checked build: the row is one of O's, the partial one of the workspace's
            if (write)
                write = in_range(whole ? p.row_ok(orow) : p.slot_ok(w.slot(blockIdx.x)) && prow < C::ROWS,
                                 p.status, abort_flag);
            tc_fence_after();
            if (have_rows && (!kTwo || n_iter > 0)) {
                for (int c = c_lo; c < c_hi; ++c) {
                    float acc[32];
                    uint32_t v[32];
                    tmem_ld32(kTwo ? o_addr + c * 32 : trow + C::o_col(0) + c * 32, v);
                    tmem_wait_ld();
                    reg_fence32(v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) acc[k] = a0 * __uint_as_float(v[k]);
                    if constexpr (!kTwo) {
                        if (use1) {
                            tmem_ld32(trow + C::o_col(1) + c * 32, v);
                            tmem_wait_ld();
                            reg_fence32(v);
#pragma unroll
                            for (int k = 0; k < 32; ++k) acc[k] = fmaf(a1, __uint_as_float(v[k]), acc[k]);
                        }
                    }
                    if (write && ok) {
                        if (whole) {
                            uint4 *dst = reinterpret_cast<uint4 *>(p.O + orow * D + c * 32);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t o[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    o[x] = zero ? 0u : pack_bf16x2(acc[8 * k + 2 * x],
                                                                   acc[8 * k + 2 * x + 1]);
                                dst[k] = make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        } else {
                            float4 *dst = reinterpret_cast<float4 *>(part + prow * D + c * 32);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                dst[k] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2],
                                                     acc[4 * k + 3]);
                        }
                    }
                }
            }
            if (!whole && write && (kTwo || t == 0)) {
                // a piece whose bounded wait ran out weighs nothing
                part[C::ROWS * D + prow] = ok ? m : ninf();
                part[C::ROWS * (D + 1) + prow] = ok ? l : 0.f;
            }
            tc_fence_before();
            // Both halves are read before either accumulator is opened again; and after a
            // wait that ran out all softmax warps leave together, so that none is missing
            // at a later barrier.
            ok = all_of_256(ok);
        }
    }
    tree_teardown<C>(smem, tmem);
}

// Rows of the segments that several CTAs worked on, from their partial states; rows of
// sequences without a draft are zeroed here too.  One warp per row: a lane per piece for the
// weights, then D / 32 columns per lane over all pieces, whose loads do not depend on one
// another (8 pieces a row: 28 -> 5 us for one sequence of 8 drafts against a loop that read
// a piece's max before its row).
constexpr int kCombineThreads = 256;

template <int D, class C>
__global__ void __launch_bounds__(kCombineThreads)
    tree_combine_kernel(const TreeParams p, int row_blocks, int rows_per_block) {
    constexpr int PER = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int rb = static_cast<int>(blockIdx.x % row_blocks);
    const int bh = static_cast<int>(blockIdx.x / row_blocks);
    const int hkv = bh % p.Hkv, b = bh / p.Hkv;
    const long long found = p.before[b], total = p.before[p.B];
    const long long H = p.segs;
    const long long share = (total * H + p.n_run - 1) / p.n_run;
    const TreeLens len = tree_lens(p, b, false);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = warp; k < rows_per_block; k += kCombineThreads / 32) {
        const int row = rb * rows_per_block + k;
        if (row >= p.R) break;
        // checked build: the row is one of O's
        if (!in_range(b < p.B && p.row_ok((long long)(b * p.Hq + hkv * (p.Hq / p.Hkv)) * p.T + row), p.status,
                      nullptr))
            break;
        __nv_bfloat16 *out = p.O + ((long long)(b * p.Hq + hkv * (p.Hq / p.Hkv)) * p.T + row) * D + lane * PER;
        float acc[PER] = {};
        float inv = 0.f;
        if (len.nt > 0) {
            const int rt = row / C::ROWS, prow = row - rt * C::ROWS;
            const int q = hkv * p.n_rt + rt, lane_q = q % p.lanes;
            const long long f0 = found * H + (long long)(q / p.lanes) * len.nt, f1 = f0 + len.nt;
            const int c0 = static_cast<int>(f0 / share), n = static_cast<int>((f1 - 1) / share) - c0 + 1;
            if (n == 1) continue;  // one CTA wrote the row
            // piece i of the segment, in run c0 + i of its lane: the first slot of that CTA, or
            // the second where the piece closes run c0
            const int odd = f0 > c0 * share ? 1 : 0;
            auto piece = [&](int i) -> const float * {
                return p.ws + (2 * ((long long)(c0 + i) * p.lanes + lane_q) + (i == 0 ? odd : 0)) * C::WS;
            };
            // checked build: all pieces stand in the workspace
            if (!in_range(p.slot_ok(2 * ((long long)c0 * p.lanes + lane_q) + odd) &&
                              p.slot_ok(2 * ((long long)(c0 + n - 1) * p.lanes + lane_q)) && prow < C::ROWS,
                          p.status, nullptr))
                continue;
            float M = ninf(), lsum = 0.f;
            for (int i0 = 0; i0 < n; i0 += 32) {
                const bool has = i0 + lane < n;
                const float *s = piece(has ? i0 + lane : 0) + C::ROWS * D + prow;
                const float m = has ? s[0] : ninf(), l = has ? s[C::ROWS] : 0.f;
                float top = m;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float grown = fmaxf(M, top);
                if (grown == ninf()) {  // no key seen so far, or NaN scores alone
                    lsum += l;
                    continue;
                }
                const float old = fast_exp2(M - grown);  // 0 for the first batch
                M = grown;
                const float wt = fast_exp2(m - M);
                lsum = lsum * old + wt * l;
#pragma unroll
                for (int x = 0; x < PER; ++x) acc[x] *= old;
                const int cnt = min(32, n - i0);
#pragma unroll 8
                for (int i = 0; i < cnt; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, wt, i);
                    const float *src = piece(i0 + i) + prow * D + lane * PER;
                    float v[PER];
                    if constexpr (PER == 4) *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(src);
                    else *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(src);
                    // a piece that saw no key of this row holds nothing to weigh
#pragma unroll
                    for (int x = 0; x < PER; ++x) acc[x] = wi > 0.f ? fmaf(wi, v[x], acc[x]) : acc[x];
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
            if (lsum != 0.f && row % p.T < len.drafts) inv = 1.f / lsum;
        }
#pragma unroll
        for (int x = 0; x < PER; x += 2)
            *reinterpret_cast<uint32_t *>(out + x) =
                inv != 0.f ? pack_bf16x2(acc[x] * inv, acc[x + 1] * inv) : 0u;
    }
}

template <int D, class C>
attn_status_t launch_tree_d(const TreeArgs &a, cudaStream_t stream,
                            void (*kernel)(CUtensorMap, CUtensorMap, CUtensorMap, TreeParams)) {
    TreeParams p;
    p.O = static_cast<__nv_bfloat16 *>(a.O);
    p.tables = a.block_tables;
    p.ctx = a.context_lens;
    p.parents = a.parents;
    p.drafts = a.draft_lens;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.T = a.T;
    p.R = a.Hq / a.Hkv * a.T;
    p.n_rt = (p.R + C::ROWS - 1) / C::ROWS;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.shift = 0;
    while ((1 << p.shift) < a.block_size) ++p.shift;
    p.box_rows = a.block_size < TK ? a.block_size : TK;
    p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
    p.wait_limit_ns = wait_limit_ns();
    p.status = device_status_word();
    if (!p.status) return ATTN_ERR_CUDA;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm < 1)
        return ATTN_ERR_CUDA;
    // As many lanes as divide the pairs evenly and leave at most a tenth of the SMs without
    // a CTA (8 KV heads: 144 CTAs of 148 SMs).
    const int q = a.Hkv * p.n_rt;
    p.lanes = 1;
    for (int l = 2; l <= q && l <= n_sm; ++l)
        if (q % l == 0 && n_sm / l * l * 10 >= n_sm * 9) p.lanes = l;
    p.segs = q / p.lanes;
    p.n_run = n_sm / p.lanes;
    const int n_cta = p.lanes * p.n_run;
    CUtensorMap tq, tk, tv;
    attn_status_t st;
    const uint64_t rows = (uint64_t)a.num_blocks * a.block_size;
    if ((st = make_tmap_bf16_3d(&tq, a.Q, D, p.R, (uint64_t)a.B * a.Hkv, C::RQ)) != ATTN_OK ||
        (st = make_tmap_bf16_paged_groups(&tk, a.K, D, a.Hkv, rows, p.box_rows)) != ATTN_OK ||
        (st = make_tmap_bf16_paged_groups(&tv, a.V, D, a.Hkv, rows, p.box_rows)) != ATTN_OK)
        return st;
    if (kernel_setup(reinterpret_cast<const void *>(kernel), C::SMEM, kTreeRegs) != cudaSuccess)
        return ATTN_ERR_CUDA;
    void *ws = nullptr;
    const size_t partials = (size_t)2 * n_cta * C::WS * sizeof(float);  // a multiple of 8
    if (workspace_alloc(&ws, partials + ((size_t)a.B + 1) * sizeof(long long), stream) != cudaSuccess)
        return ATTN_ERR_CUDA;
    p.ws = static_cast<float *>(ws);
    p.before = reinterpret_cast<long long *>(static_cast<char *>(ws) + partials);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_cta), 1, 1);
    cfg.blockDim = dim3(kTreeThreads, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    st = cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    // a row per warp while the blocks fit on the SMs at once, four where that leaves more
    // blocks that only find their segment whole
    const long long fine = ((long long)p.R + 7) / 8 * a.B * a.Hkv;
    const int rows_per_block = fine <= 8ll * n_cta ? 8 : 32;
    const int row_blocks = (p.R + rows_per_block - 1) / rows_per_block;
    if (st == ATTN_OK) {
        cfg.gridDim = dim3(static_cast<unsigned>(row_blocks) * a.B * a.Hkv, 1, 1);
        cfg.blockDim = dim3(kCombineThreads, 1, 1);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, C>, p, row_blocks, rows_per_block) != cudaSuccess)
            st = ATTN_ERR_CUDA;
    }
    if (workspace_free(ws, stream) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return st;
}

}  // namespace

attn_status_t launch_tree(const TreeArgs &a, cudaStream_t stream) {
    const int R = a.Hq / a.Hkv * a.T;
    if ((long long)a.B * a.Hq * a.T > 0x7fffffffll - 2 * TM ||
        (long long)a.B * a.Hkv * ((R + 31) / 32) > 0x7fffffffll)
        return ATTN_ERR_INVALID;
#define GQA_LAUNCH(DD)                                                                              \
    do {                                                                                            \
        if (R <= TM)                                                                                \
            return launch_tree_d<DD, TreeCfg<DD, false>>(a, stream, tree_kernel<DD, false>);        \
        return launch_tree_d<DD, TreeCfg<DD, true>>(a, stream, tree_kernel<DD, true>);              \
    } while (0)
    if (a.D == 128) GQA_LAUNCH(128);
    GQA_LAUNCH(64);
#undef GQA_LAUNCH
}

}  // namespace gqa
