// attn_api.cu -- the library's C ABI (declared in include/gqa_attn.h):
// host-side argument validation, TMA descriptor encoding, the per-device status
// word, and the workspaces (from a per-device pool the library owns).
#include <nvtx3/nvToolsExt.h>
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <set>
#include <utility>

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace gqa {

__device__ int g_status = 0;

namespace {
std::mutex g_status_mutex;
int *g_status_ptr[64] = {};
}  // namespace

int *device_status_word() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(g_status_mutex);
    if (g_status_ptr[dev] == nullptr) {
        void *ptr = nullptr;
        if (cudaGetSymbolAddress(&ptr, g_status) != cudaSuccess) return nullptr;
        g_status_ptr[dev] = static_cast<int *>(ptr);
    }
    return g_status_ptr[dev];
}

size_t decode_workspace_floats(int B, int Hq, int n_splits, int D);

namespace {
std::mutex g_setup_mutex;
std::set<std::pair<int, const void *>> g_setup_done;
}  // namespace

cudaError_t kernel_setup(const void *func, int smem_bytes, int required_regs, bool max_smem_carveout) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_setup_mutex);
    if (g_setup_done.count({dev, func})) return cudaSuccess;
    if (required_regs >= 0) {
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, func)) != cudaSuccess) return e;
        if (fa.numRegs != required_regs) return cudaErrorInvalidValue;
    }
    if ((e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes)) !=
        cudaSuccess)
        return e;
    if (max_smem_carveout &&
        (e = cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout,
                                  cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
        return e;
    g_setup_done.insert({dev, func});
    return cudaSuccess;
}

namespace {
// While a stream is captured in the global mode (or by this thread), the runtime refuses
// allocations on other streams and spoils the capture, since an allocation may synchronise.
// Stream-ordered ones do not: for their time the thread has the relaxed mode.
struct AnyCaptureMode {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    AnyCaptureMode() { (void)cudaThreadExchangeStreamCaptureMode(&mode); }
    ~AnyCaptureMode() { (void)cudaThreadExchangeStreamCaptureMode(&mode); }
    AnyCaptureMode(const AnyCaptureMode &) = delete;
    AnyCaptureMode &operator=(const AnyCaptureMode &) = delete;
};

std::mutex g_pool_mutex;
cudaMemPool_t g_pool[64] = {};
bool g_pool_made[64] = {};
}  // namespace

// Stream-ordered workspace from a memory pool the library owns on each device
// (made on first use).  Its release threshold is the maximum, so memory freed
// back to it stays reserved for the next call instead of returning to the driver
// at every synchronisation; the default pool, which other code in the process may
// use, keeps its own settings.
cudaError_t workspace_alloc(void **ptr, size_t bytes, cudaStream_t stream) {
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaMemPool_t pool;
    {
        std::lock_guard<std::mutex> lock(g_pool_mutex);
        if (!g_pool_made[dev]) {
            cudaMemPoolProps props = {};
            props.allocType = cudaMemAllocationTypePinned;
            props.handleTypes = cudaMemHandleTypeNone;
            props.location.type = cudaMemLocationTypeDevice;
            props.location.id = dev;
            if ((e = cudaMemPoolCreate(&g_pool[dev], &props)) != cudaSuccess) return e;
            uint64_t keep = UINT64_MAX;
            if ((e = cudaMemPoolSetAttribute(g_pool[dev], cudaMemPoolAttrReleaseThreshold, &keep)) !=
                cudaSuccess)
                return e;
            g_pool_made[dev] = true;
        }
        pool = g_pool[dev];
    }
    AnyCaptureMode any;
    return cudaMallocFromPoolAsync(ptr, bytes, pool, stream);
}

cudaError_t workspace_free(void *ptr, cudaStream_t stream) {
    AnyCaptureMode any;
    return cudaFreeAsync(ptr, stream);
}

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    return fn;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

attn_status_t make_tmap_bf16_3d(CUtensorMap *map, const void *base, uint64_t D, uint64_t rows,
                                uint64_t outer, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return ATTN_ERR_CUDA;
    const cuuint64_t dims[3] = {D, rows > 0 ? rows : 1, outer > 0 ? outer : 1};
    const cuuint64_t strides[2] = {D * 2, D * 2 * (rows > 0 ? rows : 1)};
    const cuuint32_t box[3] = {64, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_INVALID;
}

attn_status_t make_tmap_bf16_paged(CUtensorMap *map, const void *base, uint64_t D, uint64_t heads,
                                   uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return ATTN_ERR_CUDA;
    const cuuint64_t dims[3] = {D, heads, rows > 0 ? rows : 1};
    const cuuint64_t strides[2] = {D * 2, D * 2 * heads};
    const cuuint32_t box[3] = {64, 1, box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_INVALID;
}

attn_status_t make_tmap_bf16_paged_wide(CUtensorMap *map, const void *base, uint64_t heads,
                                        uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return ATTN_ERR_CUDA;
    const cuuint64_t dims[4] = {64, 2, heads, rows > 0 ? rows : 1};
    const cuuint64_t strides[3] = {128, 256, 256 * heads};
    const cuuint32_t box[4] = {64, 2, 1, box_rows};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_INVALID;
}

attn_status_t make_tmap_bf16_paged_groups(CUtensorMap *map, const void *base, uint64_t D, uint64_t heads,
                                          uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return ATTN_ERR_CUDA;
    const cuuint64_t row = D * 2 * heads;  // bytes
    const cuuint64_t dims[5] = {64, 8, D / 64, rows / 8, heads};
    const cuuint64_t strides[4] = {row, 128, 8 * row, D * 2};
    const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), box_rows / 8, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_INVALID;
}

namespace {

__global__ void wait_probe_kernel(uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    // Nobody arrives on `bar`: the bounded wait must give up and record the status.
    warp_wait(b, 0, &abort_flag, limit_ns, &g_status);
    __syncthreads();
}

}  // namespace

#ifdef GQA_ATTN_DEBUG
namespace {
std::atomic<uint64_t> g_wait_limit_ns{kWaitLimitNs};
}  // namespace

uint64_t wait_limit_ns() { return g_wait_limit_ns.load(); }

// Checked build only: the bounded waits' limit in the launches that follow; negative: the
// usual one again.
extern "C" void attn_debug_wait_limit(long long ns) {
    g_wait_limit_ns = ns < 0 ? kWaitLimitNs : static_cast<uint64_t>(ns);
}
#endif

attn_status_t launch_wait_probe(int limit_us, cudaStream_t stream) {
    return launch_kernel(wait_probe_kernel, dim3(1), 32, 0, stream,
                         static_cast<uint64_t>(limit_us) * 1000ull);
}

}  // namespace gqa

using namespace gqa;

namespace {
// NVTX range around an ABI call (host side: the enqueue of its kernels), so that
// a profiler's timeline names the calls; no cost without a tool attached.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};
}  // namespace

namespace {

attn_status_t validate_fwd(void *O, const void *Q, const void *K, const void *V, float *LSE, int B,
                           int Hq, int Hkv, int Sq, int Sk, int D, float scale, int causal,
                           int window, int input_pos) {
    if (B < 0 || Sq < 0 || Sk < 0 || Hq < 1 || Hkv < 1 || input_pos < 0 || window < 0)
        return ATTN_ERR_INVALID;
    if (Hq % Hkv != 0) return ATTN_ERR_INVALID;
    if (causal != 0 && causal != 1) return ATTN_ERR_INVALID;
    if (window > 0 && !causal) return ATTN_ERR_INVALID;
    if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    const long long rows_q = (long long)B * Hq * Sq, rows_k = (long long)B * Hkv * Sk;
    if (rows_q > 0 && (!O || !Q)) return ATTN_ERR_NULL;
    if (rows_q > 0 && Sk > 0 && (!K || !V)) return ATTN_ERR_NULL;
    if (!aligned16(O) || !aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(LSE))
        return ATTN_ERR_INVALID;
    // TMA coordinates are 32-bit and each dimension must stay below 2^32 elements.
    if ((long long)B * Hq > 0x7fffffffll || (long long)B * Hkv > 0x7fffffffll)
        return ATTN_ERR_INVALID;
    (void)rows_k;
    (void)LSE;
    return ATTN_OK;
}

}  // namespace

extern "C" {

attn_status_t attn_fwd_varlen(void *O, const void *Q, const void *K, const void *V, float *LSE,
                              int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                              int causal, int window, int input_pos, const int32_t *k_lengths,
                              const int32_t *q_lengths, void *stream) {
    NvtxRange nvtx_range("attn_fwd_varlen");
    attn_status_t st =
        validate_fwd(O, Q, K, V, LSE, B, Hq, Hkv, Sq, Sk, D, scale, causal, window, input_pos);
    if (st != ATTN_OK) return st;
    if ((long long)B * Hq * Sq == 0) return ATTN_OK;
    FwdArgs a;
    a.O = O;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.LSE = LSE;
    a.k_lengths = k_lengths;
    a.q_lengths = q_lengths;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Sq = Sq;
    a.Sk = Sk;
    a.D = D;
    a.scale = scale;
    a.causal = causal;
    a.window = window;
    a.input_pos = input_pos;
    if (Sk == 0) {
        // No key at all: every row is empty.  The kernel handles k_end = 0 but
        // needs a valid K/V tensor map; use the query tensor as a stand-in.
        a.K = Q;
        a.V = Q;
        a.Sk = 0;
    }
    return answer(launch_fwd(a, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_fwd(void *O, const void *Q, const void *K, const void *V, float *LSE, int B,
                       int Hq, int Hkv, int Sq, int Sk, int D, float scale, int causal, int window,
                       int input_pos, const int32_t *k_lengths, void *stream) {
    NvtxRange nvtx_range("attn_fwd");
    return attn_fwd_varlen(O, Q, K, V, LSE, B, Hq, Hkv, Sq, Sk, D, scale, causal, window,
                           input_pos, k_lengths, nullptr, stream);
}

attn_status_t attn_fwd_flex(void *O, const void *Q, const void *K, const void *V, float *LSE,
                            int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale,
                            int causal, int window, int input_pos,
                            const int32_t *k_lengths, const int32_t *q_lengths,
                            float softcap, const float *alibi_slopes,
                            const int32_t *doc_q, const int32_t *doc_kv,
                            const uint8_t *block_mask, int block_mask_per_head, void *stream) {
    NvtxRange nvtx_range("attn_fwd_flex");
    attn_status_t st =
        validate_fwd(O, Q, K, V, LSE, B, Hq, Hkv, Sq, Sk, D, scale, causal, window, input_pos);
    if (st != ATTN_OK) return st;
    if (!(softcap >= 0.f) || !std::isfinite(softcap)) return ATTN_ERR_INVALID;
    if (softcap > 0.f && alibi_slopes) return ATTN_ERR_INVALID;
    if ((doc_q == nullptr) != (doc_kv == nullptr)) return ATTN_ERR_INVALID;
    if (block_mask_per_head != 0 && block_mask_per_head != 1) return ATTN_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(alibi_slopes) | reinterpret_cast<uintptr_t>(doc_q) |
         reinterpret_cast<uintptr_t>(doc_kv)) & 3u)
        return ATTN_ERR_INVALID;
    if ((long long)Sk > (long long)gqa::kFlexMaxKvTiles * 128) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * Hq * Sq == 0) return ATTN_OK;
    FwdArgs a;
    a.O = O;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.LSE = LSE;
    a.k_lengths = k_lengths;
    a.q_lengths = q_lengths;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Sq = Sq;
    a.Sk = Sk;
    a.D = D;
    a.scale = scale;
    a.causal = causal;
    a.window = window;
    a.input_pos = input_pos;
    a.flex = 1;
    a.softcap = softcap;
    a.alibi_slopes = alibi_slopes;
    a.doc_q = doc_q;
    a.doc_kv = doc_kv;
    a.block_mask = block_mask;
    a.block_mask_per_head = block_mask_per_head;
    if (Sk == 0) {
        a.K = Q;  // stand-in tensor map; no key is visible
        a.V = Q;
        a.doc_kv = nullptr;
        a.doc_q = nullptr;
        a.block_mask = nullptr;
    }
    if (gqa::bsparse_eligible(a))
        return answer(gqa::launch_fwd_bsparse(a, static_cast<cudaStream_t>(stream)));
    return answer(launch_fwd(a, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_fwd_sinks(void *O, const void *Q, const void *K, const void *V, float *LSE,
                             int B, int Hq, int Hkv, int Sq, int Sk, int D, float scale, int window,
                             int sinks, int input_pos, const int32_t *k_lengths,
                             const int32_t *q_lengths, void *stream) {
    NvtxRange nvtx_range("attn_fwd_sinks");
    attn_status_t st =
        validate_fwd(O, Q, K, V, LSE, B, Hq, Hkv, Sq, Sk, D, scale, 1, window, input_pos);
    if (st != ATTN_OK) return st;
    if (window < 1 || sinks < 0) return ATTN_ERR_INVALID;
    if ((long long)B * Hq * Sq == 0) return ATTN_OK;
    FwdArgs a;
    a.O = O;
    a.Q = Q;
    a.K = Sk > 0 ? K : Q;  // stand-in tensor map without a key
    a.V = Sk > 0 ? V : Q;
    a.LSE = LSE;
    a.k_lengths = k_lengths;
    a.q_lengths = q_lengths;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Sq = Sq;
    a.Sk = Sk;
    a.D = D;
    a.scale = scale;
    a.causal = 1;
    a.window = window;
    a.sinks = sinks;
    a.input_pos = input_pos;
    return answer(launch_fwd(a, static_cast<cudaStream_t>(stream)));
}

namespace {

// Most positions of a cache that the windowed decode and the tree accept: their kernels
// add tile and slice offsets to positions in 32 bits.
constexpr long long kMaxPositions = 1ll << 30;

// Slices per (sequence, KV head) when the caller leaves them to the library: enough for
// two blocks per SM, and at most one per 64-key tile that can hold a visible key.  Up to 8
// slices need no workspace and no second kernel, so more are made only where 8 would be
// left with more than 32 tiles each.  0: the device cannot be asked for its SMs.
int sink_splits(int B, int Hkv, long long S_cap, int window, int sinks) {
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n_sm < 1)
        return 0;
    const long long tiles = std::min((std::min<long long>(window, S_cap) + 62) / 64 + 1 +
                                         (std::min<long long>(sinks, S_cap) + 63) / 64,
                                     (S_cap + 63) / 64);
    const long long pairs = std::max(1ll, (long long)B * Hkv);
    const long long n = std::max(1ll, std::min({(2ll * n_sm + pairs - 1) / pairs, tiles, 64ll}));
    return static_cast<int>(n > 8 && tiles <= 8 * 32 ? 8 : n);
}

// attn_decode (window = 0) and attn_decode_sinks (where n_splits may be 0).
attn_status_t decode_contiguous(void *O, const void *Q, const void *K, const void *V,
                                const int32_t *lengths, int window, int sinks, int n_splits,
                                void *stream, int B, int Hq, int Hkv, int S_cap, int D) {
    if (B < 0 || Hq < 1 || Hkv < 1 || S_cap < 0 || n_splits < (window > 0 ? 0 : 1) || n_splits > 64)
        return ATTN_ERR_INVALID;
    if (Hq % Hkv != 0 || Hq / Hkv > 16 || Hkv > 65535) return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (B == 0) return ATTN_OK;
    if (!O || !Q || !lengths) return ATTN_ERR_NULL;
    if (S_cap > 0 && (!K || !V)) return ATTN_ERR_NULL;
    if (!aligned16(O) || !aligned16(Q) || !aligned16(K) || !aligned16(V) ||
        (reinterpret_cast<uintptr_t>(lengths) & 3u))
        return ATTN_ERR_INVALID;
    if ((long long)B * Hkv > 0x7fffffffll) return ATTN_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_splits == 0 && (n_splits = sink_splits(B, Hkv, S_cap, window, sinks)) == 0)
        return answer(ATTN_ERR_CUDA);
    const size_t bytes = decode_workspace_floats(B, Hq, n_splits, D) * sizeof(float);
    const bool needs_ws = window == 0 || !decode_sinks_in_cluster(n_splits);
    void *ws = nullptr;
    if (needs_ws && workspace_alloc(&ws, bytes, s) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    DecodeArgs a;
    a.O = O;
    a.Q = Q;
    a.K = S_cap > 0 ? K : Q;
    a.V = S_cap > 0 ? V : Q;
    a.lengths = lengths;
    a.n_splits = n_splits;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.S_cap = S_cap;
    a.D = D;
    a.workspace = static_cast<float *>(ws);
    a.window = window;
    a.sinks = sinks;
    attn_status_t st = launch_decode(a, s);
    if (needs_ws && workspace_free(ws, s) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return answer(st);
}

}  // namespace

attn_status_t attn_decode(void *O, const void *Q, const void *K, const void *V,
                          const int32_t *lengths, int n_splits, void *stream, int B, int Hq,
                          int Hkv, int S_cap, int D) {
    NvtxRange nvtx_range("attn_decode");
    return decode_contiguous(O, Q, K, V, lengths, 0, 0, n_splits, stream, B, Hq, Hkv, S_cap, D);
}

attn_status_t attn_decode_sinks(void *O, const void *Q, const void *K, const void *V,
                                const int32_t *lengths, int window, int sinks, int n_splits,
                                void *stream, int B, int Hq, int Hkv, int S_cap, int D) {
    NvtxRange nvtx_range("attn_decode_sinks");
    if (window < 1 || sinks < 0 || S_cap > kMaxPositions) return ATTN_ERR_INVALID;
    return decode_contiguous(O, Q, K, V, lengths, window, sinks, n_splits, stream, B, Hq, Hkv, S_cap,
                             D);
}

namespace {

// attn_bwd (sinks = 0) and attn_bwd_sinks.
attn_status_t backward(void *dQ, void *dK, void *dV, const void *dO, const void *Q, const void *K,
                       const void *V, const void *O, const float *LSE, int B, int Hq, int Hkv,
                       int Sq, int Sk, int D, float scale, int causal, int window, int sinks,
                       int input_pos, const int32_t *k_lengths, const int32_t *q_lengths,
                       void *stream) {
    attn_status_t st =
        validate_fwd(const_cast<void *>(O), Q, K, V, nullptr, B, Hq, Hkv, Sq, Sk, D, scale, causal,
                     window, input_pos);
    if (st != ATTN_OK) return st;
    const long long rows_q = (long long)B * Hq * Sq, rows_k = (long long)B * Hkv * Sk;
    if (rows_q > 0 && (!dQ || !dO || !LSE)) return ATTN_ERR_NULL;
    if (rows_k > 0 && (!dK || !dV)) return ATTN_ERR_NULL;
    if (!aligned16(dQ) || !aligned16(dK) || !aligned16(dV) || !aligned16(dO) ||
        (reinterpret_cast<uintptr_t>(LSE) & 3u))
        return ATTN_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows_q == 0) {  // no query: dK = dV = 0
        if (rows_k > 0) {
            const size_t bytes = (size_t)rows_k * D * 2;
            if (cudaMemsetAsync(dK, 0, bytes, s) != cudaSuccess ||
                cudaMemsetAsync(dV, 0, bytes, s) != cudaSuccess)
                return answer(ATTN_ERR_CUDA);
        }
        return ATTN_OK;
    }
    void *ws = nullptr;
    if (workspace_alloc(&ws, (size_t)rows_q * sizeof(float), s) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    BwdArgs a;
    a.dQ = dQ;
    a.dK = dK;
    a.dV = dV;
    a.dO = dO;
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.O = O;
    a.LSE = LSE;
    a.k_lengths = k_lengths;
    a.q_lengths = q_lengths;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Sq = Sq;
    a.Sk = Sk;
    a.D = D;
    a.scale = scale;
    a.causal = causal;
    a.window = window;
    a.input_pos = input_pos;
    a.sinks = sinks;
    a.delta = static_cast<float *>(ws);
    st = launch_bwd(a, s);
    if (workspace_free(ws, s) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return answer(st);
}

}  // namespace

attn_status_t attn_bwd(void *dQ, void *dK, void *dV, const void *dO, const void *Q, const void *K,
                       const void *V, const void *O, const float *LSE, int B, int Hq, int Hkv,
                       int Sq, int Sk, int D, float scale, int causal, int window, int input_pos,
                       const int32_t *k_lengths, const int32_t *q_lengths, void *stream) {
    NvtxRange nvtx_range("attn_bwd");
    return backward(dQ, dK, dV, dO, Q, K, V, O, LSE, B, Hq, Hkv, Sq, Sk, D, scale, causal, window, 0,
                    input_pos, k_lengths, q_lengths, stream);
}

attn_status_t attn_bwd_sinks(void *dQ, void *dK, void *dV, const void *dO, const void *Q,
                             const void *K, const void *V, const void *O, const float *LSE, int B,
                             int Hq, int Hkv, int Sq, int Sk, int D, float scale, int window,
                             int sinks, int input_pos, const int32_t *k_lengths,
                             const int32_t *q_lengths, void *stream) {
    NvtxRange nvtx_range("attn_bwd_sinks");
    if (window < 1 || sinks < 0) return ATTN_ERR_INVALID;
    return backward(dQ, dK, dV, dO, Q, K, V, O, LSE, B, Hq, Hkv, Sq, Sk, D, scale, 1, window, sinks,
                    input_pos, k_lengths, q_lengths, stream);
}

attn_status_t attn_rbs_block_mask(uint8_t *block_mask, float *base_scores, float *rescue_scores,
                                  const void *Q, const void *K, int B, int Hq, int Hkv, int Sq,
                                  int Sk, int D, float alpha_base, float alpha_rescue,
                                  int diagonal, void *stream) {
    NvtxRange nvtx_range("attn_rbs_block_mask");
    if (B < 0 || Hq < 1 || Hkv < 1 || Sq < 0 || Sk < 0 || diagonal < 0) return ATTN_ERR_INVALID;
    if (Hq % Hkv != 0) return ATTN_ERR_INVALID;
    if (!(alpha_base > 0.f) || !(alpha_rescue > 0.f) || !std::isfinite(alpha_base) ||
        !std::isfinite(alpha_rescue))
        return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if ((long long)Sk > 131072) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * Hq * Sq == 0 || Sk == 0) return ATTN_OK;
    if (!block_mask || !Q || !K) return ATTN_ERR_NULL;
    if (!aligned16(Q) || !aligned16(K) ||
        ((reinterpret_cast<uintptr_t>(base_scores) | reinterpret_cast<uintptr_t>(rescue_scores)) & 3u))
        return ATTN_ERR_INVALID;
    const long long nkb = (Sk + 63) / 64;
    const size_t ws_floats = (size_t)B * Hkv * nkb * (D + 2);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if (workspace_alloc(&ws, ws_floats * sizeof(float), s) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    RbsArgs a;
    a.Q = Q;
    a.K = K;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Sq = Sq;
    a.Sk = Sk;
    a.D = D;
    a.alpha_base = alpha_base;
    a.alpha_rescue = alpha_rescue;
    a.diagonal = diagonal;
    a.mask = block_mask;
    a.base_scores = base_scores;
    a.rescue_scores = rescue_scores;
    a.cent = static_cast<float *>(ws);
    a.rad = a.cent + (size_t)B * Hkv * nkb * D;
    a.beta = a.rad + (size_t)B * Hkv * nkb;
    attn_status_t st = launch_rbs(a, s);
    if (workspace_free(ws, s) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return answer(st);
}

namespace {

// attn_decode_paged (window = 0) and attn_decode_paged_sinks (where n_splits may be 0).
attn_status_t decode_paged(void *O, const void *Q, const void *K_cache, const void *V_cache,
                           const int32_t *block_tables, const int32_t *seq_lens, int window,
                           int sinks, int n_splits, void *stream, int B, int Hq, int Hkv,
                           int num_blocks, int block_size, int max_blocks_per_seq, int D) {
    if (B < 0 || Hq < 1 || Hkv < 1 || num_blocks < 1 || max_blocks_per_seq < 0 ||
        n_splits < (window > 0 ? 0 : 1) || n_splits > 64)
        return ATTN_ERR_INVALID;
    if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1)) != 0)
        return ATTN_ERR_INVALID;
    if (Hq % Hkv != 0 || Hq / Hkv > 16 || Hkv > 65535) return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if ((long long)num_blocks * block_size > 0x7fffffffll ||
        (long long)max_blocks_per_seq * block_size > 0x7fffffffll)
        return ATTN_ERR_INVALID;
    if (B == 0) return ATTN_OK;
    if (!O || !Q || !K_cache || !V_cache || !seq_lens || (max_blocks_per_seq > 0 && !block_tables))
        return ATTN_ERR_NULL;
    if (!aligned16(O) || !aligned16(Q) || !aligned16(K_cache) || !aligned16(V_cache) ||
        ((reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(block_tables)) & 3u))
        return ATTN_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_splits == 0 &&
        (n_splits = sink_splits(B, Hkv, (long long)max_blocks_per_seq * block_size, window, sinks)) == 0)
        return answer(ATTN_ERR_CUDA);
    const size_t bytes = decode_workspace_floats(B, Hq, n_splits, D) * sizeof(float);
    const bool needs_ws = window == 0 || !decode_sinks_in_cluster(n_splits);
    void *ws = nullptr;
    if (needs_ws && workspace_alloc(&ws, bytes, s) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    DecodeArgs a;
    a.O = O;
    a.Q = Q;
    a.K = K_cache;
    a.V = V_cache;
    a.lengths = seq_lens;
    a.n_splits = n_splits;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.S_cap = max_blocks_per_seq * block_size;
    a.D = D;
    a.workspace = static_cast<float *>(ws);
    a.block_tables = block_tables;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.window = window;
    a.sinks = sinks;
    attn_status_t st = launch_decode(a, s);
    if (needs_ws && workspace_free(ws, s) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return answer(st);
}

// Sizes of a paged cache that every operator on it checks.
attn_status_t validate_pool(int num_blocks, int block_size, int max_blocks) {
    if (num_blocks < 1 || max_blocks < 1) return ATTN_ERR_INVALID;
    if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1)) != 0)
        return ATTN_ERR_INVALID;
    if ((long long)num_blocks * block_size > 0x7fffffffll ||
        (long long)max_blocks * block_size > 0x7fffffffll)
        return ATTN_ERR_INVALID;
    return ATTN_OK;
}

// Alignment of int32 arrays (ref_counts, which fork and extend read in 16-byte vectors, is
// checked with aligned16 there).
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

attn_status_t attn_decode_paged(void *O, const void *Q, const void *K_cache, const void *V_cache,
                                const int32_t *block_tables, const int32_t *seq_lens, int n_splits,
                                void *stream, int B, int Hq, int Hkv, int num_blocks,
                                int block_size, int max_blocks_per_seq, int D) {
    NvtxRange nvtx_range("attn_decode_paged");
    return decode_paged(O, Q, K_cache, V_cache, block_tables, seq_lens, 0, 0, n_splits, stream, B, Hq,
                        Hkv, num_blocks, block_size, max_blocks_per_seq, D);
}

attn_status_t attn_decode_paged_sinks(void *O, const void *Q, const void *K_cache,
                                      const void *V_cache, const int32_t *block_tables,
                                      const int32_t *seq_lens, int window, int sinks, int n_splits,
                                      void *stream, int B, int Hq, int Hkv, int num_blocks,
                                      int block_size, int max_blocks_per_seq, int D) {
    NvtxRange nvtx_range("attn_decode_paged_sinks");
    if (window < 1 || sinks < 0) return ATTN_ERR_INVALID;
    if ((long long)max_blocks_per_seq * block_size > kMaxPositions) return ATTN_ERR_INVALID;
    return decode_paged(O, Q, K_cache, V_cache, block_tables, seq_lens, window, sinks, n_splits, stream,
                        B, Hq, Hkv, num_blocks, block_size, max_blocks_per_seq, D);
}

attn_status_t attn_tree_paged(void *O, const void *Q, const void *K_cache, const void *V_cache,
                              const int32_t *block_tables, const int32_t *context_lens,
                              const int32_t *parents, const int32_t *draft_lens, void *stream,
                              int B, int Hq, int Hkv, int T, int num_blocks, int block_size,
                              int max_blocks_per_seq, int D) {
    NvtxRange nvtx_range("attn_tree_paged");
    if (B < 0 || Hq < 1 || Hkv < 1 || T < 0 || T > 256) return ATTN_ERR_INVALID;
    attn_status_t st = validate_pool(num_blocks, block_size, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    if ((long long)max_blocks_per_seq * block_size > kMaxPositions) return ATTN_ERR_INVALID;
    if (Hq % Hkv != 0 || Hq / Hkv > 16) return ATTN_ERR_INVALID;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if ((long long)B * Hkv > 0x7fffffffll) return ATTN_ERR_INVALID;
    if (B == 0 || T == 0) return ATTN_OK;
    if (!O || !Q || !K_cache || !V_cache || !block_tables || !context_lens || !parents)
        return ATTN_ERR_NULL;
    if (!aligned16(O) || !aligned16(Q) || !aligned16(K_cache) || !aligned16(V_cache) ||
        !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(parents) ||
        !aligned4(draft_lens))
        return ATTN_ERR_INVALID;
    TreeArgs a;
    a.O = O;
    a.Q = Q;
    a.K = K_cache;
    a.V = V_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.parents = parents;
    a.draft_lens = draft_lens;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.T = T;
    a.D = D;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    return answer(launch_tree(a, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_cache_append(void *K_cache, void *V_cache, const void *K_new, const void *V_new,
                                const int32_t *block_tables, const int32_t *start,
                                const int32_t *n_new, void *stream, int B, int Hkv, int T,
                                int num_blocks, int block_size, int max_blocks_per_seq, int D) {
    NvtxRange nvtx_range("attn_cache_append");
    if (B < 0 || Hkv < 1 || T < 0) return ATTN_ERR_INVALID;
    attn_status_t st = validate_pool(num_blocks, block_size, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return ATTN_OK;
    if (!K_cache || !V_cache || !K_new || !V_new || !block_tables || !start) return ATTN_ERR_NULL;
    if (!aligned16(K_cache) || !aligned16(V_cache) || !aligned16(K_new) || !aligned16(V_new) ||
        !aligned4(block_tables) || !aligned4(start) || !aligned4(n_new))
        return ATTN_ERR_INVALID;
    CacheArgs a;
    a.K = K_cache;
    a.V = V_cache;
    a.K_new = K_new;
    a.V_new = V_new;
    a.block_tables = block_tables;
    a.start = start;
    a.counts = n_new;
    a.B = B;
    a.Hkv = Hkv;
    a.T = T;
    a.D = D;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    return answer(launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_cache_compact(void *K_cache, void *V_cache, const int32_t *block_tables,
                                 const int32_t *base, const int32_t *keep, const int32_t *n_keep,
                                 void *stream, int B, int Hkv, int A, int num_blocks,
                                 int block_size, int max_blocks_per_seq, int D) {
    NvtxRange nvtx_range("attn_cache_compact");
    if (B < 0 || Hkv < 1 || Hkv > (1 << 24) || A < 0) return ATTN_ERR_INVALID;
    attn_status_t st = validate_pool(num_blocks, block_size, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (B == 0 || A == 0) return ATTN_OK;
    if (!K_cache || !V_cache || !block_tables || !base || !keep) return ATTN_ERR_NULL;
    if (!aligned16(K_cache) || !aligned16(V_cache) || !aligned4(block_tables) || !aligned4(base) ||
        !aligned4(keep) || !aligned4(n_keep))
        return ATTN_ERR_INVALID;
    CacheArgs a;
    a.K = K_cache;
    a.V = V_cache;
    a.block_tables = block_tables;
    a.start = base;
    a.keep = keep;
    a.counts = n_keep;
    a.B = B;
    a.Hkv = Hkv;
    a.T = A;
    a.D = D;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    return answer(launch_cache_compact(a, static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_cache_copy_blocks(void *K_cache, void *V_cache, const int32_t *src,
                                     const int32_t *dst, void *stream, int N, int num_blocks,
                                     int block_size, int Hkv, int D) {
    NvtxRange nvtx_range("attn_cache_copy_blocks");
    if (N < 0 || N > 65536 || Hkv < 1) return ATTN_ERR_INVALID;
    attn_status_t st = validate_pool(num_blocks, block_size, 1);
    if (st != ATTN_OK) return st;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (N == 0) return ATTN_OK;
    if (!K_cache || !V_cache || !src || !dst) return ATTN_ERR_NULL;
    if (!aligned16(K_cache) || !aligned16(V_cache) || !aligned4(src) || !aligned4(dst))
        return ATTN_ERR_INVALID;
    return answer(launch_cache_copy(K_cache, V_cache, src, dst, N, num_blocks,
                                    (long long)block_size * Hkv * D * 2,
                                    static_cast<cudaStream_t>(stream)));
}

attn_status_t attn_cache_fork(int32_t *block_tables, int32_t *ref_counts, int32_t *seq_lens,
                              const int32_t *parents, const int32_t *children, int32_t *copy_src,
                              int32_t *copy_dst, void *stream, int N, int R, int num_blocks,
                              int block_size, int max_blocks_per_seq) {
    NvtxRange nvtx_range("attn_cache_fork");
    if (N < 0 || N > 65536 || R < 0) return ATTN_ERR_INVALID;
    attn_status_t st = validate_pool(num_blocks, block_size, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    if (N == 0) return ATTN_OK;
    if (!block_tables || !ref_counts || !seq_lens || !parents || !children || !copy_src || !copy_dst)
        return ATTN_ERR_NULL;
    if (!aligned4(block_tables) || !aligned16(ref_counts) || !aligned4(seq_lens) ||
        !aligned4(parents) || !aligned4(children) || !aligned4(copy_src) || !aligned4(copy_dst))
        return ATTN_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if (workspace_alloc(&ws, (size_t)N * sizeof(int32_t), s) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    CacheForkArgs a;
    a.tables = block_tables;
    a.refs = ref_counts;
    a.lens = seq_lens;
    a.parents = parents;
    a.children = children;
    a.copy_src = copy_src;
    a.copy_dst = copy_dst;
    a.N = N;
    a.R = R;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.workspace = static_cast<int32_t *>(ws);
    st = launch_cache_fork(a, s);
    if (workspace_free(ws, s) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return answer(st);
}

attn_status_t attn_cache_extend(int32_t *block_tables, int32_t *ref_counts, const int32_t *from_lens,
                                const int32_t *to_lens, void *stream, int R, int num_blocks,
                                int block_size, int max_blocks_per_seq) {
    NvtxRange nvtx_range("attn_cache_extend");
    if (R < 0) return ATTN_ERR_INVALID;
    attn_status_t st = validate_pool(num_blocks, block_size, max_blocks_per_seq);
    if (st != ATTN_OK) return st;
    // the kernel counts and ranks empty entries in 32 bits
    if ((long long)R * max_blocks_per_seq > 0x7fffffffll) return ATTN_ERR_INVALID;
    if (R == 0) return ATTN_OK;
    if (!block_tables || !ref_counts || !from_lens || !to_lens) return ATTN_ERR_NULL;
    if (!aligned4(block_tables) || !aligned16(ref_counts) || !aligned4(from_lens) ||
        !aligned4(to_lens))
        return ATTN_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const long long ints = R + 1ll + std::min((long long)R * max_blocks_per_seq, (long long)num_blocks);
    void *ws = nullptr;
    if (workspace_alloc(&ws, (size_t)ints * sizeof(int32_t), s) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    CacheExtendArgs a;
    a.tables = block_tables;
    a.refs = ref_counts;
    a.from = from_lens;
    a.to = to_lens;
    a.R = R;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.workspace = static_cast<int32_t *>(ws);
    st = launch_cache_extend(a, s);
    if (workspace_free(ws, s) != cudaSuccess && st == ATTN_OK) st = ATTN_ERR_CUDA;
    return answer(st);
}

attn_status_t attn_cache_free(int32_t *block_tables, int32_t *ref_counts, const int32_t *rows,
                              const int32_t *first, const int32_t *last, void *stream, int N, int R,
                              int num_blocks, int max_blocks_per_seq) {
    NvtxRange nvtx_range("attn_cache_free");
    if (N < 0 || R < 0 || num_blocks < 1 || max_blocks_per_seq < 1) return ATTN_ERR_INVALID;
    if (N == 0) return ATTN_OK;
    if (!block_tables || !ref_counts || !rows || !first || !last) return ATTN_ERR_NULL;
    if (!aligned4(block_tables) || !aligned4(ref_counts) || !aligned4(rows) || !aligned4(first) ||
        !aligned4(last))
        return ATTN_ERR_INVALID;
    return answer(launch_cache_free(block_tables, ref_counts, rows, first, last, N, R, max_blocks_per_seq,
                                    num_blocks, static_cast<cudaStream_t>(stream)));
}

const char *attn_status_string(attn_status_t status) {
    switch (status) {
        case ATTN_OK: return "ATTN_OK";
        case ATTN_ERR_NULL: return "ATTN_ERR_NULL: a required pointer is NULL";
        case ATTN_ERR_INVALID: return "ATTN_ERR_INVALID: inconsistent sizes, flags or alignment";
        case ATTN_ERR_UNSUPPORTED: return "ATTN_ERR_UNSUPPORTED: head size not built (64, 128)";
        case ATTN_ERR_CUDA: return "ATTN_ERR_CUDA: a CUDA call failed";
        case ATTN_ERR_TIMEOUT: return "ATTN_ERR_TIMEOUT: a bounded device wait ran out";
        case ATTN_ERR_DEVICE_BOUNDS: return "ATTN_ERR_DEVICE_BOUNDS: a length exceeded its tensor";
        case ATTN_ERR_SCRATCH_LIMIT:
            return "ATTN_ERR_SCRATCH_LIMIT: workspace exceeds the 16 MiB fixed array of "
                   "attn_decode_noalloc";
        case ATTN_ERR_NO_PAGES: return "ATTN_ERR_NO_PAGES: no free page left in the cache's pool";
    }
    return "unknown attn_status_t";
}

attn_status_t attn_last_device_status(void *stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return answer(ATTN_ERR_CUDA);
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) != cudaSuccess) return answer(ATTN_ERR_CUDA);
    return static_cast<attn_status_t>(v);
}

attn_status_t attn_check_bounded_wait(int limit_us, void *stream) {
    if (limit_us < 1 || limit_us > 2000000) return ATTN_ERR_INVALID;
    return answer(launch_wait_probe(limit_us, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
