// Host helpers shared by the library's translation units: the thread-local
// error text, checks of pointers, extents and dtypes, the device guard, cached
// device attributes, the tensor-map encoder and dependent launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include "fused_logp.h"

// Reads and clears the error word of the orthogonalisation's bounded waits on
// the current device (orthogonalize.cu).
cudaError_t flp_take_orthogonalize_error(int* code);

namespace flp_host {

inline thread_local char g_msg[512] = "";

inline flp_status fail(flp_status st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return st;
}

inline flp_status ok() {
    g_msg[0] = '\0';
    return FLP_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int elem_bytes(int dtype) { return dtype == FLP_DTYPE_F32 ? 4 : 2; }

// Bytes spanned by an [n, ld] matrix whose rows use the first `v` columns.
inline bool span_bytes(int64_t n, int64_t v, int64_t ld, int64_t elem, int64_t* out) {
    int64_t a, b;
    if (__builtin_mul_overflow(n - 1, ld, &a)) return false;
    if (__builtin_add_overflow(a, v, &b)) return false;
    if (__builtin_mul_overflow(b, elem, out)) return false;
    return true;
}

// Device that holds `p`; FLP_EINVAL if `p` is not device-accessible memory.
inline flp_status device_of(const void* p, const char* name, int* dev) {
    if (p == nullptr) return fail(FLP_EINVAL, "%s is a null pointer", name);
    cudaPointerAttributes a;
    const cudaError_t e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return fail(FLP_EINVAL, "%s: cudaPointerGetAttributes failed (%s)", name, cudaGetErrorString(e));
    }
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
        return fail(FLP_EINVAL, "%s must point to device memory", name);
    *dev = a.device;
    return FLP_OK;
}

// Every required pointer, and every optional one that is not null, must be
// device memory of one device; returns that device.
inline flp_status common_device(int count, const void* const* ptrs, const char* const* names,
                         const bool* optional, int* dev) {
    int d0 = -1;
    const char* first = nullptr;
    for (int i = 0; i < count; ++i)   // before the first CUDA call
        if (ptrs[i] == nullptr && !(optional && optional[i])) return fail(FLP_EINVAL, "%s is a null pointer", names[i]);
    for (int i = 0; i < count; ++i) {
        if (optional && optional[i] && ptrs[i] == nullptr) continue;
        int d;
        const flp_status st = device_of(ptrs[i], names[i], &d);
        if (st != FLP_OK) return st;
        if (!first) {
            d0 = d;
            first = names[i];
        } else if (d != d0) {
            return fail(FLP_EINVAL, "%s is on device %d but %s is on device %d", names[i], d, first, d0);
        }
    }
    *dev = d0;
    return FLP_OK;
}

// Makes `dev` current for the call and restores the caller's device after.
struct DeviceGuard {
    int prev = -1;
    bool switched = false;
    flp_status enter(int dev) {
        cudaError_t e = cudaGetDevice(&prev);
        if (e != cudaSuccess) return fail(FLP_ECUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
        if (prev != dev) {
            e = cudaSetDevice(dev);
            if (e != cudaSuccess) return fail(FLP_ECUDA, "cudaSetDevice: %s", cudaGetErrorString(e));
            switched = true;
        }
        return FLP_OK;
    }
    ~DeviceGuard() {
        if (switched) (void)cudaSetDevice(prev);
    }
};

inline flp_status check_launch(const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FLP_ECUDA, "%s launch failed: %s", what, cudaGetErrorString(e));
    return ok();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows start on 16-byte boundaries: base aligned and the byte stride a
// multiple of 16.
inline bool rows_aligned16(const void* p, int64_t ld, int dtype) {
    return aligned16(p) && (ld * elem_bytes(dtype)) % 16 == 0;
}

constexpr int64_t kMaxGrid = 2147483647;
constexpr int kMaxDevices = 64;

inline int grid_for(int64_t items) { return (int)(items < kMaxGrid ? items : kMaxGrid); }

inline flp_status check_dtype(int dtype) {
    if (dtype != FLP_DTYPE_BF16 && dtype != FLP_DTYPE_F16 && dtype != FLP_DTYPE_F32)
        return fail(FLP_EINVAL, "dtype must be FLP_DTYPE_BF16, FLP_DTYPE_F16 or FLP_DTYPE_F32 (got %d)", dtype);
    return FLP_OK;
}

// Per-device caches below are atomics: host threads may call in
// concurrently; every writer stores the same value, so the first one wins.
inline int sm_count(int dev) {
    static std::atomic<int> count[kMaxDevices];
    int c = count[dev].load(std::memory_order_acquire);
    if (c == 0) {
        if (cudaDeviceGetAttribute(&c, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        count[dev].store(c, std::memory_order_release);
    }
    return c;
}

// cuTensorMapEncodeTiled from the driver, found once through the runtime (no
// link against the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return (EncodeTiledFn) nullptr;
        }
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// Launches kern<<<grid, block, smem, s>>>(args...) with programmatic stream
// serialization: the kernel may start while the previous work on s runs and
// waits for it with griddepcontrol.wait.
template <class... Args>
inline flp_status launch_dependent(const char* what, void (*kern)(Args...), dim3 grid, int block, size_t smem,
                                   cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "%s launch: %s", what, cudaGetErrorString(e));
    return ok();
}

}  // namespace flp_host
