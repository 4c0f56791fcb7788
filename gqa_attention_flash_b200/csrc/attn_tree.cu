// attn_tree.cu -- attention of a tree of drafted tokens over a paged KV cache.
//
// Speculative decoding checks T drafted tokens per sequence in one pass.  Their keys and
// values already stand in the sequence's pages behind its `ctx` committed tokens (draft i
// at position ctx + i).  Draft i continues draft parents[i] (< i) or, for -1, the context;
// it sees every key before ctx, itself and its ancestors:
//   O_i = softmax_j(<q_i, k_j> / sqrt(D)) V over j < ctx and j = ctx + a, a in anc(i).
//
// One block of D threads per (draft, query head, sequence); keys in chunks of D: one
// score per thread, then one output column per thread.
#include <cuda_bf16.h>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace gqa {

namespace {

struct TreeParams {
    __nv_bfloat16 *O;
    const __nv_bfloat16 *Q, *K, *V;
    const int32_t *tables, *ctx, *parents, *drafts;
    int B, Hq, Hkv, T, max_blocks, num_blocks, shift;
    float scale_log2;
    int *status;
};

template <int D>
__global__ void __launch_bounds__(D) tree_kernel(const TreeParams p) {
    __shared__ float q[D], w[D], red[D / 32];
    __shared__ long long rows[D];
    const int i = blockIdx.x % p.T;
    const long long bh = blockIdx.x / p.T;
    const int h = static_cast<int>(bh % p.Hq), b = static_cast<int>(bh / p.Hq);
    const int hkv = h / (p.Hq / p.Hkv), tid = threadIdx.x;
    const long long cap = (long long)p.max_blocks << p.shift;
    long long ctx = p.ctx[b];
    int drafts = p.drafts ? p.drafts[b] : p.T;
    if (ctx < 0 || drafts > p.T || ctx + drafts > cap) {
        if (tid == 0) record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
        ctx = max(0ll, min(ctx, cap));
        drafts = static_cast<int>(min((long long)min(drafts, p.T), cap - ctx));
    }
    const long long out = (bh * p.T + i) * D;
    if (i >= drafts) {
        p.O[out + tid] = __float2bfloat16_rn(0.f);
        return;
    }
    q[tid] = __bfloat162float(p.Q[out + tid]);
    const int32_t *par = p.parents + (long long)b * p.T;
    float m = __int_as_float(0xff800000), l = 0.f, o = 0.f;
    const long long n = ctx + i + 1;
    for (long long k0 = 0; k0 < n; k0 += D) {
        __syncthreads();
        const long long j = k0 + tid;
        bool vis = j < ctx;
        if (!vis && j < n) {
            int a = i;
            while (a > j - ctx) {
                int up = par[a];
                if (up >= a || up < -1) {
                    record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
                    up = -1;
                }
                a = up;
            }
            vis = a == j - ctx;
        }
        float s = __int_as_float(0xff800000);
        rows[tid] = -1;
        if (vis) {
            const int page = p.tables[(long long)b * p.max_blocks + (j >> p.shift)];
            s = 0.f;
            if (page < 0 || page >= p.num_blocks) {
                record_status(p.status, ATTN_ERR_DEVICE_BOUNDS);
            } else {
                const long long row = (((long long)page << p.shift) + (j & ((1 << p.shift) - 1))) * p.Hkv + hkv;
                rows[tid] = row;
                for (int d = 0; d < D; ++d) s = fmaf(q[d], __bfloat162float(p.K[row * D + d]), s);
            }
            s *= p.scale_log2;
        }
        float mx = s;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        float m_new = m;
        for (int x = 0; x < D / 32; ++x) m_new = fmaxf(m_new, red[x]);
        const float base = m_new == __int_as_float(0xff800000) ? 0.f : m_new;
        w[tid] = exp2f(s - base);
        const float alpha = exp2f(m - base);
        m = m_new;
        l *= alpha;
        o *= alpha;
        __syncthreads();
        for (int x = 0; x < D; ++x) {
            if (w[x] == 0.f) continue;
            l += w[x];
            if (rows[x] >= 0) o = fmaf(w[x], __bfloat162float(p.V[rows[x] * D + tid]), o);
        }
    }
    p.O[out + tid] = __float2bfloat16_rn(o / l);
}

}  // namespace

attn_status_t launch_tree(const TreeArgs &a, cudaStream_t stream) {
    TreeParams p;
    p.O = static_cast<__nv_bfloat16 *>(a.O);
    p.Q = static_cast<const __nv_bfloat16 *>(a.Q);
    p.K = static_cast<const __nv_bfloat16 *>(a.K);
    p.V = static_cast<const __nv_bfloat16 *>(a.V);
    p.tables = a.block_tables;
    p.ctx = a.context_lens;
    p.parents = a.parents;
    p.drafts = a.draft_lens;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.T = a.T;
    p.max_blocks = a.max_blocks;
    p.num_blocks = a.num_blocks;
    p.shift = 0;
    while ((1 << p.shift) < a.block_size) ++p.shift;
    p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(a.D));
    p.status = device_status_word();
    if (!p.status) return ATTN_ERR_CUDA;
    const long long grid = (long long)a.B * a.Hq * a.T;
    if (grid > 0x7fffffffll) return ATTN_ERR_INVALID;
    if (a.D == 128) tree_kernel<128><<<static_cast<unsigned>(grid), 128, 0, stream>>>(p);
    else tree_kernel<64><<<static_cast<unsigned>(grid), 64, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace gqa
