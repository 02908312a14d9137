// host.cuh - host-side helpers shared by the translation units of libcolimoe:
// the thread's error message, launch checks, the shared-memory opt-in, launches
// as programmatic dependents and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <mutex>
#include <utility>

#include "coli_moe.h"

namespace coli {

// message of the last failure on this thread (a plain buffer: no allocation,
// so that no exception can cross the C boundary)
inline thread_local char g_err[512] = "";

inline int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return code;
}

// every address a multiple of its elements' size (a kernel would fault on others)
inline int elements_ok(const char* what, std::initializer_list<std::pair<const void*, int>> buffers) {
    for (const auto& b : buffers)
        if (reinterpret_cast<uintptr_t>(b.first) % b.second)
            return fail(COLI_E_INVAL, "%s: a buffer's address is no multiple of its elements' %d bytes", what, b.second);
    return COLI_OK;
}

inline int check_launch(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(COLI_E_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return COLI_OK;
}

inline cudaStream_t S(coli_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Raise a kernel's dynamic shared-memory limit to `bytes` (static + dynamic
// above 48 KB needs the opt-in).  The largest value set per (device, kernel) is
// remembered so that a forward normally makes no attribute call.
inline int set_smem(const void* fn, int bytes) {
    struct Entry { int dev; const void* fn; int bytes; };
    constexpr int kEntries = 256;  // past these the attribute is set at every call
    static std::mutex mu;
    static Entry done[kEntries];
    static int n = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(COLI_E_CUDA, "smem attribute: no device");
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < n; ++i)
        if (done[i].dev == dev && done[i].fn == fn && done[i].bytes >= bytes) return COLI_OK;
    const cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return fail(COLI_E_CUDA, "smem attribute: %s", cudaGetErrorString(e));
    for (int i = 0; i < n; ++i)
        if (done[i].dev == dev && done[i].fn == fn) { done[i].bytes = bytes; return COLI_OK; }
    if (n < kEntries) done[n++] = {dev, fn, bytes};
    return COLI_OK;
}

// Launch as a programmatic dependent of the previous kernel in the stream: the
// kernel may start while that one finishes and waits (griddepcontrol.wait)
// before it reads what that one wrote.
template <typename... Args>
inline int launch_pdl(void (*kern)(Args...), dim3 grid, dim3 threads, int smem, cudaStream_t st,
               const char* what, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return fail(COLI_E_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return check_launch(what);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

}  // namespace coli
