// The norm in front of the LM head: layer norm, or RMS norm (no centring).
//
// Forward, per row x of width d:
//   mu = mean(x) (0 without centring), var = mean((x - mu)^2),
//   rstd = (var + eps)^(-1/2), xh = (x - mu) rstd, y = xh w + b.
// Backward, with g = dy w:
//   dx = rstd (g - mean(g) - xh mean(g xh))      (no mean(g) without centring)
//   dw = sum over rows of dy xh, db = sum over rows of dy.
// All sums are FP32; y and dx are rounded once to x's type.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace flp {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A weight or bias vector: absent, of x's 16-bit type, or FP32.
struct NormVec {
    const void* p;
    int dtype;   // FLP_DTYPE_*
};
__device__ __forceinline__ float norm_vec_at(const NormVec& v, int64_t i, float absent) {
    if (v.p == nullptr) return absent;
    if (v.dtype == 0) return to_f32(static_cast<const __nv_bfloat16*>(v.p)[i]);
    if (v.dtype == 1) return to_f32(static_cast<const __half*>(v.p)[i]);
    return static_cast<const float*>(v.p)[i];
}

struct NormFwdArgs {
    const void* x;
    int64_t n, d, ld_x;
    NormVec w, b;
    float eps, inv_d;
    void* y;
    int64_t ld_y;
    float *mean, *rstd;   // nullable
};

struct NormBwdArgs {
    const void* dy;
    int64_t ld_dy;
    const void* x;
    int64_t n, d, ld_x;
    NormVec w;
    const float *mean, *rstd;   // mean null without centring
    float inv_d;
    void* dx;
    int64_t ld_dx;
    float* part_w;   // [kNormParts, d] partial sums of dy xh, or null
    float* part_b;   // [kNormParts, d] partial sums of dy, or null
};

// Rows of partial weight gradients: a constant, so that the order of the sum
// over the batch depends on the problem alone.
constexpr int kNormParts = 304;
constexpr int kNormAnyThreads = 256;

// Sum of v over a block of kThreads, the same value in every thread.
template <int kThreads>
__device__ __forceinline__ float norm_block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();   // the last sum's readers are done with red
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) s += red[k];
    return s;
}

// ---------------------------------------------------------------- any width

// One CTA per row, the row read once per sum: for widths that no register
// tile holds.
template <class T, bool kCenter>
__global__ void __launch_bounds__(kNormAnyThreads)
k_norm_fwd_any(NormFwdArgs a) {
    __shared__ float red[kNormAnyThreads / 32];
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
        T* y = static_cast<T*>(a.y) + r * a.ld_y;
        float mu = 0.f;
        if (kCenter) {
            float s = 0.f;
            for (int64_t i = threadIdx.x; i < a.d; i += kNormAnyThreads) s += to_f32(x[i]);
            mu = norm_block_sum<kNormAnyThreads>(s, red) * a.inv_d;
        }
        float q = 0.f;
        for (int64_t i = threadIdx.x; i < a.d; i += kNormAnyThreads) {
            const float c = to_f32(x[i]) - mu;
            q += c * c;
        }
        const float rstd = __frsqrt_rn(norm_block_sum<kNormAnyThreads>(q, red) * a.inv_d + a.eps);
        for (int64_t i = threadIdx.x; i < a.d; i += kNormAnyThreads)
            y[i] = from_f32<T>((to_f32(x[i]) - mu) * rstd * norm_vec_at(a.w, i, 1.f) + norm_vec_at(a.b, i, 0.f));
        if (threadIdx.x == 0) {
            if (kCenter && a.mean) a.mean[r] = mu;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <class T, class G, bool kCenter>
__global__ void __launch_bounds__(kNormAnyThreads)
k_norm_dx_any(NormBwdArgs a) {
    __shared__ float red[kNormAnyThreads / 32];
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ld_x;
        const G* dy = static_cast<const G*>(a.dy) + r * a.ld_dy;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
        const float mu = kCenter ? a.mean[r] : 0.f, rstd = a.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        for (int64_t i = threadIdx.x; i < a.d; i += kNormAnyThreads) {
            const float g = to_f32(dy[i]) * norm_vec_at(a.w, i, 1.f);
            if (kCenter) s1 += g;
            s2 += g * ((to_f32(x[i]) - mu) * rstd);
        }
        const float c1 = kCenter ? norm_block_sum<kNormAnyThreads>(s1, red) * a.inv_d : 0.f;
        const float c2 = norm_block_sum<kNormAnyThreads>(s2, red) * a.inv_d;
        for (int64_t i = threadIdx.x; i < a.d; i += kNormAnyThreads) {
            const float g = to_f32(dy[i]) * norm_vec_at(a.w, i, 1.f);
            const float xh = (to_f32(x[i]) - mu) * rstd;
            dx[i] = from_f32<T>((g - c1 - xh * c2) * rstd);
        }
    }
}

// Partial sums over the rows p, p + kNormParts, ... of one column per thread.
template <class T, class G, bool kCenter>
__global__ void __launch_bounds__(kNormAnyThreads)
k_norm_dw_any(NormBwdArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kNormAnyThreads + threadIdx.x;
    if (c >= a.d) return;
    const int p = blockIdx.y;
    float sw = 0.f, sb = 0.f;
    for (int64_t r = p; r < a.n; r += kNormParts) {
        const float g = to_f32(static_cast<const G*>(a.dy)[r * a.ld_dy + c]);
        const float mu = kCenter ? a.mean[r] : 0.f;
        const float xh = (to_f32(static_cast<const T*>(a.x)[r * a.ld_x + c]) - mu) * a.rstd[r];
        sw += g * xh;
        sb += g;
    }
    if (a.part_w) a.part_w[(int64_t)p * a.d + c] = sw;
    if (a.part_b) a.part_b[(int64_t)p * a.d + c] = sb;
}

// ---------------------------------------------------------------- partial rows

constexpr int kNormFoldCols = 32, kNormFoldRows = 16;

// out[c] (+)= sum over the partial rows in a fixed order: kNormFoldRows
// threads share a column, each taking every kNormFoldRows-th row.
__global__ void __launch_bounds__(kNormFoldCols * kNormFoldRows)
k_norm_fold(const float* __restrict__ part, int rows, int64_t d, float* __restrict__ out, int accumulate) {
    __shared__ float red[kNormFoldRows][kNormFoldCols + 1];
    const int tx = threadIdx.x % kNormFoldCols, ty = threadIdx.x / kNormFoldCols;
    const int64_t c = (int64_t)blockIdx.x * kNormFoldCols + tx;
    float s = 0.f;
    if (c < d)
        for (int r = ty; r < rows; r += kNormFoldRows) s += part[(int64_t)r * d + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < d) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kNormFoldRows; ++k) t += red[k][tx];
        out[c] = accumulate ? out[c] + t : t;
    }
}

}  // namespace flp
