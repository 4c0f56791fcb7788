// A stand-in for the CUDA runtime, for tests of the library's host code without a GPU: it
// keeps a log of the calls, launches nothing, and lets one chosen call fail.
#include <cuda.h>
#include <cuda_runtime.h>

#include <vector>

namespace {
enum Kind { kAlloc, kFree, kLaunch, kRecord, kWait, kSync, kOther };
struct Entry {
    int kind;
    const void *stream, *what;
};
std::vector<Entry> g_log;
int g_calls = 0, g_fail_at = -1, g_sms = 148, g_grid_x = 0;
long long g_next = 0;

cudaError_t g_last = cudaSuccess;  // what cudaGetLastError answers

// One of the calls that can fail: true where this one does.
bool fails(cudaError_t e = cudaErrorUnknown) {
    if (g_calls++ != g_fail_at) return false;
    g_last = e;
    return true;
}
void note(int kind, const void *stream, const void *what) { g_log.push_back({kind, stream, what}); }
void *handle() { return reinterpret_cast<void *>(0x100000 + 0x1000 * ++g_next); }

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
}  // namespace

extern "C" {

void fake_reset(int fail_at) {
    g_log.clear();
    g_calls = 0;
    g_last = cudaSuccess;
    g_fail_at = fail_at;
}
void fake_set_last_error(int e) { g_last = static_cast<cudaError_t>(e); }
int fake_last_error() { return static_cast<int>(g_last); }
void fake_set_sms(int n) { g_sms = n; }
int fake_last_grid_x() { return g_grid_x; }
int fake_calls() { return g_calls; }
int fake_log_size() { return static_cast<int>(g_log.size()); }
void fake_log(int i, int *kind, const void **stream, const void **what) {
    *kind = g_log[i].kind;
    *stream = g_log[i].stream;
    *what = g_log[i].what;
}

void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
char __cudaInitModule(void **) { return 1; }
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *,
                            int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, struct CUstream_st *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }

cudaError_t cudaGetDevice(int *d) {
    *d = 0;
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) {
    *v = g_sms;
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *, int, size_t, unsigned) {
    *n = 1;
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes *a, const void *) {
    *a = cudaFuncAttributes();
    a->numRegs = 168;
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) {
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **p, const void *) {
    *p = handle();
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaGetDriverEntryPoint(const char *, void **p, unsigned long long,
                                    cudaDriverEntryPointQueryResult *q) {
    *p = reinterpret_cast<void *>(encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaMemPoolCreate(cudaMemPool_t *p, const cudaMemPoolProps *) {
    *p = static_cast<cudaMemPool_t>(handle());
    return cudaSuccess;
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void *) { return cudaSuccess; }
cudaError_t cudaMallocFromPoolAsync(void **p, size_t, cudaMemPool_t, cudaStream_t s) {
    if (fails(cudaErrorMemoryAllocation)) return cudaErrorMemoryAllocation;
    note(kAlloc, s, *p = handle());
    return cudaSuccess;
}
cudaError_t cudaFreeAsync(void *p, cudaStream_t s) {
    note(kFree, s, p);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
    if (fails()) return cudaErrorUnknown;
    g_grid_x = static_cast<int>(c->gridDim.x);
    note(kLaunch, c->stream, f);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void *f, dim3, dim3, void **, size_t, cudaStream_t s) {
    if (fails()) return cudaErrorUnknown;
    note(kLaunch, s, f);
    return cudaSuccess;
}
cudaError_t cudaGetLastError() {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t *s, unsigned) {
    *s = static_cast<cudaStream_t>(handle());
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaEventCreateWithFlags(cudaEvent_t *e, unsigned) {
    *e = static_cast<cudaEvent_t>(handle());
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaStreamGetCaptureInfo_v2(cudaStream_t, cudaStreamCaptureStatus *st, unsigned long long *,
                                        cudaGraph_t *, const cudaGraphNode_t **, size_t *) {
    *st = cudaStreamCaptureStatusNone;
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaThreadExchangeStreamCaptureMode(cudaStreamCaptureMode *) { return cudaSuccess; }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t e, cudaStream_t s) {
    if (fails()) return cudaErrorUnknown;
    note(kRecord, s, e);
    return cudaSuccess;
}
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t e, unsigned) {
    if (fails()) return cudaErrorUnknown;
    note(kWait, s, e);
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) {
    note(kSync, s, nullptr);
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *p, int, size_t, cudaStream_t s) {
    note(kOther, s, p);
    return fails() ? cudaErrorUnknown : cudaSuccess;
}
cudaError_t cudaMemcpyFromSymbol(void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }

}  // extern "C"
