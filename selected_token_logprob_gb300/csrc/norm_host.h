// Host-side helpers of the norm's forward and backward.
#pragma once

#include "host_common.h"
#include "norm_kernels.cuh"

namespace flp_host {

constexpr int64_t kNormMaxDim = ((int64_t)1 << 31) - 1;

inline flp_status check_norm_shape(int64_t n, int64_t d, int dtype) {
    flp_status st;
    if ((st = check_dtype(dtype)) != FLP_OK) return st;
    if (n < 0) return fail(FLP_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (d < 1) return fail(FLP_EINVAL, "d must be >= 1 (got %lld)", (long long)d);
    if (d > kNormMaxDim) return fail(FLP_EUNSUPPORTED, "d must be below 2^31 (got %lld)", (long long)d);
    return FLP_OK;
}

// A vector's or gradient's dtype: the rows' own or FP32.
inline flp_status check_side_dtype(const char* name, int side, int dtype) {
    if (side != dtype && side != FLP_DTYPE_F32)
        return fail(FLP_EINVAL, "%s dtype must be x's (%d) or FLP_DTYPE_F32 (got %d)", name, dtype, side);
    return FLP_OK;
}

struct Extent {
    const char* name;
    const void* p;
    int64_t bytes;
};

// The output `o` must not share bytes with the input `i`, unless it lies on
// it exactly and `same` allows that.
inline flp_status check_apart(const Extent& o, const Extent& i, bool same) {
    if (o.p == nullptr || i.p == nullptr || (same && o.p == i.p)) return FLP_OK;
    const uintptr_t a = reinterpret_cast<uintptr_t>(o.p), b = reinterpret_cast<uintptr_t>(i.p);
    if (a < b + (uintptr_t)i.bytes && b < a + (uintptr_t)o.bytes)
        return fail(FLP_EINVAL, "%s overlaps %s", o.name, i.name);
    return FLP_OK;
}

// Allows a kernel its ring of shared memory, once per device.
template <class K>
flp_status norm_setup(K kern, int dev, std::atomic<bool>* ready) {
    if (ready[dev].load(std::memory_order_acquire)) return FLP_OK;
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, kern);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448 - (int)f.sharedSizeBytes);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "norm setup: %s", cudaGetErrorString(e));
    ready[dev].store(true, std::memory_order_release);
    return FLP_OK;
}

// SMs that the persistent grids are sized for: a constant, so that the order
// of the weight's gradient depends on the problem alone.
constexpr int kNormSms = 152;

inline int row_ctas(int64_t n, int rows, int most) {
    const int64_t c = ceil_div(n, rows);
    return (int)(c < most ? c : most);
}

constexpr size_t kNormMaxSmem = 232448 - 2048;   // of a CTA with a row, beside the static arrays

}  // namespace flp_host
