// Host build of the library's C entry points (csrc/moe_cache.cu) over a stand-in
// for the CUDA runtime, for the CPU test suite: "device" memory is host memory,
// copies and sets take effect at once, kernel launches only write a line, and
// every call that belongs to a stream is logged with that stream.  What a test
// reads from the log is what the library asks of the runtime: which stream an
// upload, a kernel or a set went to, in which order, what a launch was given.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <string>

template <class T>
static inline T __ldcs(const T *p) { return *p; }
template <class T>
static inline T __ldg(const T *p) { return *p; }
static inline int __dp4a(int, int, int) { abort(); }
static inline unsigned __float_as_uint(float f) {
    unsigned u;
    memcpy(&u, &f, 4);
    return u;
}
static inline float __uint_as_float(unsigned u) {
    float f;
    memcpy(&f, &u, 4);
    return f;
}
template <class T>
static inline T __shfl_xor_sync(unsigned, T, int) { abort(); }
static inline unsigned __reduce_max_sync(unsigned, unsigned) { abort(); }
static inline int __reduce_add_sync(unsigned, int) { abort(); }
static inline unsigned atomicOr(unsigned *, unsigned) { abort(); }
template <class T>
static inline T atomicAdd(T *, T) { abort(); }

#include "moe_cache.cu"

namespace {
std::string g_log, g_fail_launch;
cudaError_t g_last = cudaSuccess;
constexpr size_t kDeviceMemory = (size_t)1 << 30;  // one allocation's limit

void note(const char *what, const void *stream, const void *a = nullptr, const void *b = nullptr, long long n = 0) {
    char s[200];
    snprintf(s, sizeof s, "%s %llx %llx %llx %lld\n", what, (unsigned long long)(uintptr_t)stream,
             (unsigned long long)(uintptr_t)a, (unsigned long long)(uintptr_t)b, n);
    g_log += s;
}
cudaError_t error(cudaError_t e) { return g_last = e; }
int launch(const char *what, const void *stream, const void *a = nullptr, const void *b = nullptr, long long n = 0) {
    note(what, stream, a, b, n);
    return g_fail_launch == what ? (int)error(cudaErrorLaunchOutOfResources) : 0;
}
CUresult CUDAAPI encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                        const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                        CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    return CUDA_SUCCESS;
}
}  // namespace

extern "C" {
// ---- what a test asks for
const char *host_log() { return g_log.c_str(); }
void host_clear() { g_log.clear(); }
void host_fail_launch(const char *what) { g_fail_launch = what; }
int host_last_error() { return (int)cudaGetLastError(); }

// ---- the runtime's stand-in
cudaError_t cudaGetLastError() {
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
const char *cudaGetErrorString(cudaError_t e) { return e == cudaSuccess ? "no error" : "error"; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return note("sync_device", nullptr), cudaSuccess; }
cudaError_t cudaMalloc(void **p, size_t n) {
    if (n > kDeviceMemory) return error(cudaErrorMemoryAllocation);
    *p = aligned_alloc(256, (n + 255) / 256 * 256 + 256);
    return cudaSuccess;
}
cudaError_t cudaFree(void *p) { return free(p), cudaSuccess; }
cudaError_t cudaHostAlloc(void **p, size_t n, unsigned) { return cudaMalloc(p, n); }
cudaError_t cudaFreeHost(void *p) { return cudaFree(p); }
cudaError_t cudaHostGetDevicePointer(void **d, void *h, unsigned) { return *d = h, cudaSuccess; }
cudaError_t cudaMemcpy(void *d, const void *s, size_t n, cudaMemcpyKind) {
    note("copy", nullptr, d, s, (long long)n);
    return memcpy(d, s, n), cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void *d, const void *s, size_t n, cudaMemcpyKind, cudaStream_t st) {
    note("copy", st, d, s, (long long)n);
    return memcpy(d, s, n), cudaSuccess;
}
cudaError_t cudaMemset(void *d, int v, size_t n) {
    note("set", nullptr, d, nullptr, (long long)n);
    return memset(d, v, n), cudaSuccess;
}
cudaError_t cudaMemsetAsync(void *d, int v, size_t n, cudaStream_t st) {
    note("set", st, d, nullptr, (long long)n);
    return memset(d, v, n), cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t *s, unsigned) { return *s = (cudaStream_t)(uintptr_t)0x55, cudaSuccess; }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t st) { return note("sync", st), cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) {
    return *s = cudaStreamCaptureStatusNone, cudaSuccess;
}
cudaError_t cudaEventCreate(cudaEvent_t *e) { return *e = (cudaEvent_t)(uintptr_t)0x66, cudaSuccess; }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t *e, unsigned) { return cudaEventCreate(e); }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float *ms, cudaEvent_t, cudaEvent_t) { return *ms = 0, cudaSuccess; }
cudaError_t cudaEventQuery(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes *, const void *) { return error(cudaErrorInvalidValue); }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
    *fn = (void *)encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}

// ---- the kernels' launchers
namespace moe {
int launch_rms_norm(const NormParams &p, cudaStream_t st) { return launch("rms_norm", st, p.x, p.y, p.n_tokens); }
int launch_router_loss(const RouterParams &p, int, cudaStream_t st) {
    return launch("router_loss", st, p.logits, p.ws_count, p.T);
}
size_t linear_weight_bytes(int fmt, int rows, int cols) {
    return (size_t)((rows + 15) / 16) * 16 * (cols / 32) * (fmt == kFmtQ4K ? 20 : 18);
}
int launch_linear_repack(const uint8_t *src, uint8_t *dst, int, int, int, int, cudaStream_t st) {
    return launch("linear_repack", st, src, dst);
}
int launch_linear_max(uint8_t *w, int, int, int, unsigned *out, int, cudaStream_t st) {
    return launch("linear_max", st, w, out);
}
int launch_linear(const LinearParams &p, int, cudaStream_t st) { return launch("linear", st, p.x, p.y, p.n_tokens); }
int linear_gemm_box() { return 32; }
int linear_gemm_configure() { return 0; }
int launch_linear_gemm(const LinearGemm &g, int, cudaStream_t st) {
    return launch("linear_gemm", st, g.p.x, g.p.y, g.p.n_tokens);
}
int launch_topk(const float *, int, int, int, int, int32_t *, float *, cudaStream_t st) { return launch("topk", st); }
int launch_quantize(const float *, int, int8_t *, BlockScale *, int, cudaStream_t st) { return launch("quantize", st); }
int launch_plan(const PlanParams &, cudaStream_t st) { return launch("plan", st); }
int launch_gemv(const GemvParams &, int, int, cudaStream_t st, cudaEvent_t const *) { return launch("gemv", st); }
int down_rows_per_item(int) { return 32; }
int launch_block_dots(const uint8_t *, int, int, int, int, int, const int8_t *, int32_t *, cudaStream_t st) {
    return launch("block_dots", st);
}
int launch_stream_read(const void *, size_t, uint32_t *, int, cudaStream_t st) { return launch("stream_read", st); }
size_t fused_smem_bytes(int, int) { return 1024; }
int fused_configure(int, size_t, int *b) { return *b = 0; }
int fused_rb_rows(int, int, int, int, int) { return 0; }
size_t fused_rb_smem(int, int, int, int, int, int, int *) { return 0; }
bool fused_t1_ok(int, int) { return false; }
int fused_configure_rb(int, size_t, int *b) { return *b = 0; }
int fused_configure_t1_fmt(int, int, size_t, int *b) { return *b = 0; }
int launch_fused(const FusedParams &, int, size_t, cudaStream_t st, cudaEvent_t const *) { return launch("fused", st); }
int launch_prefill(const PrefillLaunch &, cudaStream_t st, cudaEvent_t const *) { return launch("prefill", st); }
int launch_stage(const StageParams &, size_t, int, cudaStream_t st) { return launch("stage", st); }
int launch_prefetch_table(const uint64_t *, const int32_t *, const void *, int, size_t, int, uint64_t *,
                          cudaStream_t st) {
    return launch("prefetch_table", st);
}
int gemm_configure() { return 0; }
int gemm_bn(bool) { return 64; }
int gemm_rows_per_tile(bool) { return 64; }
int launch_step_finish(const Update *, int, uint64_t *, int32_t *, uint32_t *, uint32_t *, uint32_t, uint32_t *, int,
                       uint32_t *, int, cudaStream_t st) {
    return launch("step_finish", st);
}
int launch_count_assign(const int32_t *, int, int, int, uint32_t *, cudaStream_t st) { return launch("count", st); }
int launch_busy(unsigned long long, cudaStream_t st) { return launch("busy", st); }
int launch_shared_assign(const int32_t *, const float *, int, int, int, int32_t *, float *, int *, cudaStream_t st) {
    return launch("shared_assign", st);
}
}  // namespace moe
