// internal.h -- declarations shared by the library's translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "gqa_attn.h"

namespace gqa {

// Encode a 3-D bf16 tensor map over a row-major (outer, rows, D) tensor with
// a (64, box_rows, 1) box and 128-byte swizzle; out-of-range rows read as 0.
attn_status_t make_tmap_bf16_3d(CUtensorMap *map, const void *base, uint64_t D, uint64_t rows,
                                uint64_t outer, uint32_t box_rows);

// Encode a 3-D bf16 tensor map over a paged cache viewed as (rows, heads, D)
// row-major, with a (64, 1, box_rows) box and 128-byte swizzle: one box is
// box_rows consecutive cache rows of one head, 64 columns wide.
attn_status_t make_tmap_bf16_paged(CUtensorMap *map, const void *base, uint64_t D, uint64_t heads,
                                   uint64_t rows, uint32_t box_rows);

// The same cache with D = 128 viewed as (rows, heads, 2, 64): one (64, 2, 1, box_rows) box
// copies both 64-column halves of box_rows rows, stored row by row (half 0, half 1).
attn_status_t make_tmap_bf16_paged_wide(CUtensorMap *map, const void *base, uint64_t heads,
                                        uint64_t rows, uint32_t box_rows);

// The same cache (D = 64 or 128) viewed as 8-row groups: one box copies box_rows (a
// multiple of 8) consecutive rows of one head, stored as (group, 64-column half, 8 rows,
// 64 columns), each 8 x 128-byte block 128-byte swizzled.  Coordinates (0, 0, 0, group, head).
attn_status_t make_tmap_bf16_paged_groups(CUtensorMap *map, const void *base, uint64_t D, uint64_t heads,
                                          uint64_t rows, uint32_t box_rows);

// Stream-ordered workspace from the library's pool on the current device, and its end on the
// same stream.
cudaError_t workspace_alloc(void **ptr, size_t bytes, cudaStream_t stream);
cudaError_t workspace_free(void *ptr, cudaStream_t stream);

// What an entry point answers.  A CUDA call that failed also leaves its error with the
// runtime, where the process's next check of it, in whatever code, would take it for its
// own; the answer reports it, so it is cleared.
inline attn_status_t answer(attn_status_t st) {
    if (st == ATTN_ERR_CUDA) (void)cudaGetLastError();
    return st;
}

// Launch without attributes.  The launch's own result counts, not an error that was there
// before it.
template <typename... KArgs, typename... Args>
attn_status_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                            Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess ? ATTN_OK
                                                                                      : ATTN_ERR_CUDA;
}

struct FwdArgs {
    void *O;
    const void *Q, *K, *V;
    float *LSE;
    const int32_t *k_lengths, *q_lengths;
    int B, Hq, Hkv, Sq, Sk, D;
    float scale;
    int causal, window, input_pos;
    // first keys that stay visible outside the window (attn_fwd_sinks); needs
    // causal and window > 0, and excludes the flex extras
    int sinks = 0;
    // flex_attention! extras; flex = 0 selects the plain kernel
    int flex = 0;
    float softcap = 0.f;
    const float *alibi_slopes = nullptr;
    const int32_t *doc_q = nullptr, *doc_kv = nullptr;
    const uint8_t *block_mask = nullptr;
    int block_mask_per_head = 0;  // block_mask is (B, Hq, nqb, nkb) instead of (nqb, nkb)
};

// Longest KV sequence the flex kernel takes, in 128-key tiles (its per-CTA list
// of visited tiles lives in shared memory).
constexpr int kFlexMaxKvTiles = 1024;

// Block-sparse prefill kernel (BlockMask alone, no score mod, no DocumentMask,
// not causal, no lengths): longest key sequence it takes, in 64-key blocks (its
// per-CTA list of visited blocks lives in shared memory).  Other flex calls, and
// longer sequences, run on the flex kernel's list path.
constexpr int kBsparseMaxKvBlocks = 1024;
bool bsparse_eligible(const FwdArgs &a);
attn_status_t launch_fwd_bsparse(const FwdArgs &a, cudaStream_t stream);

struct DecodeArgs {
    void *O;
    const void *Q, *K, *V;
    const int32_t *lengths;
    int n_splits;
    int B, Hq, Hkv, S_cap, D;
    float *workspace;  // B * Hq * n_splits * (D + 4) floats
    // paged KV cache (block_tables != nullptr): K/V are (num_blocks, block_size,
    // Hkv, D) and S_cap = max_blocks * block_size
    const int32_t *block_tables = nullptr;
    int num_blocks = 0, block_size = 0, max_blocks = 0;
    // sliding window with sinks (attn_decode_sinks): window > 0 keeps the last
    // `window` keys and the first `sinks`; 0 = every key
    int window = 0, sinks = 0;
};

// Whether attn_decode_sinks with that many slices runs as one cluster per (KV head,
// sequence), which takes no workspace.
bool decode_sinks_in_cluster(int n_splits);

// Backward of the forward (Tylo.jl `∇attention!`).
struct BwdArgs {
    void *dQ, *dK, *dV;
    const void *dO, *Q, *K, *V, *O;
    const float *LSE;
    const int32_t *k_lengths, *q_lengths;
    int B, Hq, Hkv, Sq, Sk, D;
    float scale;
    int causal, window, input_pos;
    float *delta;  // workspace (B, Hq, Sq)
    int sinks = 0;  // first keys that stay visible outside the window
};

attn_status_t launch_bwd(const BwdArgs &a, cudaStream_t stream);
// dK / dV and dQ on tcgen05 (after the delta workspace is written).
attn_status_t launch_bwd_tc(const BwdArgs &a, cudaStream_t stream);

// Block scores + block mask of block-sparse prefill (RBS page of mlx-arsenal).
struct RbsArgs {
    const void *Q, *K;
    int B, Hq, Hkv, Sq, Sk, D;
    float alpha_base, alpha_rescue;
    int diagonal;
    uint8_t *mask;                     // (B, Hq, nqb, nkb) BlockMask states 2 / 0
    float *base_scores, *rescue_scores;  // (B, Hq, nqb, nkb) or nullptr
    float *cent, *rad, *beta;          // workspace: (B, Hkv, nkb, D), (B, Hkv, nkb) x 2
};

attn_status_t launch_rbs(const RbsArgs &a, cudaStream_t stream);

// Attention of T drafted tokens per sequence over a paged cache.
struct TreeArgs {
    void *O;
    const void *Q, *K, *V;
    const int32_t *block_tables, *context_lens, *parents, *draft_lens;
    int B, Hq, Hkv, T, D;
    int num_blocks, block_size, max_blocks;
};
attn_status_t launch_tree(const TreeArgs &a, cudaStream_t stream);

// Operators on a paged cache (cache_ops.cu).
struct CacheArgs {  // append and compact
    void *K, *V;
    const void *K_new = nullptr, *V_new = nullptr;
    const int32_t *block_tables, *start, *counts, *keep = nullptr;
    int B, Hkv, T, D;  // T: rows of K_new per sequence, or entries of keep
    int num_blocks, block_size, max_blocks;
};
attn_status_t launch_cache_append(const CacheArgs &a, cudaStream_t stream);
attn_status_t launch_cache_compact(const CacheArgs &a, cudaStream_t stream);
attn_status_t launch_cache_copy(void *K, void *V, const int32_t *src, const int32_t *dst, int n,
                                int num_blocks, long long page_bytes, cudaStream_t stream);

struct CacheForkArgs {
    int32_t *tables, *refs, *lens;
    const int32_t *parents, *children;
    int32_t *copy_src, *copy_dst;
    int N, R, num_blocks, block_size, max_blocks;
    int32_t *workspace;  // N ints
};
attn_status_t launch_cache_fork(const CacheForkArgs &a, cudaStream_t stream);

struct CacheExtendArgs {
    int32_t *tables, *refs;
    const int32_t *from, *to;
    int R, num_blocks, block_size, max_blocks;
    int32_t *workspace;  // R + 1 + min(R * max_blocks, num_blocks) ints
};
attn_status_t launch_cache_extend(const CacheExtendArgs &a, cudaStream_t stream);

attn_status_t launch_cache_free(int32_t *tables, int32_t *refs, const int32_t *rows, const int32_t *first,
                                const int32_t *last, int N, int R, int max_blocks, int num_blocks,
                                cudaStream_t stream);

// Device address of the status word on the current device (looked up once per
// device), or nullptr if the lookup failed.
int *device_status_word();

attn_status_t launch_fwd(const FwdArgs &a, cudaStream_t stream);
attn_status_t launch_decode(const DecodeArgs &a, cudaStream_t stream);
attn_status_t launch_wait_probe(int limit_us, cudaStream_t stream);

// Once per (device, kernel), thread-safe: check that the kernel was built with
// `required_regs` registers per thread (skipped when negative), raise its
// dynamic shared-memory limit to `smem_bytes` on the current device and, with
// max_smem_carveout, ask for the largest shared-memory carveout (kernels that
// run several CTAs per SM, each with a large dynamic allocation).
cudaError_t kernel_setup(const void *func, int smem_bytes, int required_regs = -1,
                         bool max_smem_carveout = false);

// Bounded-wait limit used by the attention kernels (nanoseconds of global time).
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// The limit of the next launches: kWaitLimitNs.  The checked build's tests set another with
// attn_debug_wait_limit; with 0 every wait gives up at once, which shows what a kernel
// leaves behind then.
#ifdef GQA_ATTN_DEBUG
uint64_t wait_limit_ns();
#else
constexpr uint64_t wait_limit_ns() { return kWaitLimitNs; }
#endif

}  // namespace gqa
