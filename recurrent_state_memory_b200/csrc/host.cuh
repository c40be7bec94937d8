// host.cuh -- host-side helpers shared by the library's translation units: the error detail of
// the calling thread, argument predicates, the SM count, and the device status words.
#pragma once

#include <cstdint>
#include <cstdio>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "gdr.h"

namespace gdr {

inline thread_local char t_detail[256] = "";

inline gdr_status fail(gdr_status s, const char* fmt, const char* what = "") {
    snprintf(t_detail, sizeof(t_detail), fmt, what);
    return s;
}

inline gdr_status cuda_fail(cudaError_t e, const char* where) {
    snprintf(t_detail, sizeof(t_detail), "%s: %s", where, cudaGetErrorString(e));
    return GDR_ERR_CUDA;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool dtype_ok(gdr_dtype t) { return t == GDR_F32 || t == GDR_BF16; }
inline size_t dtype_bytes(gdr_dtype t) { return t == GDR_BF16 ? 2 : 4; }

inline bool aligned_to(const void* p, gdr_dtype t) { return reinterpret_cast<uintptr_t>(p) % dtype_bytes(t) == 0; }

inline int device_sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) { cudaGetLastError(); return 148; }
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) { cudaGetLastError(); return 148; }
    return n;
}

// cuTensorMapEncodeTiled is a driver call; it is looked up through the runtime so that the
// library does not link libcuda itself.  Unlike the runtime's calls it needs a current context, which
// a host thread whose first CUDA call this is does not have yet: it gets its device's primary one.
typedef CUresult (*CtxGetCurrentFn)(CUcontext*);
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline gdr_status driver_fn(const char* name, void** fn) {
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    const cudaError_t e = cudaGetDriverEntryPoint(name, fn, cudaEnableDefault, &q);
    if (e != cudaSuccess) return cuda_fail(e, name);
    return q == cudaDriverEntryPointSuccess && *fn ? GDR_OK : fail(GDR_ERR_CUDA, "the driver has no %s", name);
}

inline gdr_status encode_fn(EncodeTiledFn* out) {
    static std::mutex mu;
    static void *encode = nullptr, *current = nullptr;
    CUcontext context = nullptr;
    {
        std::lock_guard<std::mutex> lock(mu);
        gdr_status s = encode ? GDR_OK : driver_fn("cuTensorMapEncodeTiled", &encode);
        if (s == GDR_OK && !current) s = driver_fn("cuCtxGetCurrent", &current);
        if (s != GDR_OK) return s;
        *out = reinterpret_cast<EncodeTiledFn>(encode);
    }
    if (reinterpret_cast<CtxGetCurrentFn>(current)(&context) == CUDA_SUCCESS && !context) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaSetDevice(dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
    }
    return GDR_OK;
}

// Every translation unit has a status word and a bounds site of its own (common.cuh): the ones of the
// files named.
struct StatusWords;
cudaError_t scan_status(StatusWords* w);
cudaError_t norm_status(StatusWords* w);
cudaError_t beam_status(StatusWords* w);

}  // namespace gdr
