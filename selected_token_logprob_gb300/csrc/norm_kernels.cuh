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
constexpr int kNormParts = 608;
constexpr int kNormAnyThreads = 256;
constexpr int kNormAnyParts = 304;

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

// Partial sums over the rows p, p + kNormAnyParts, ... of one column per thread.
template <class T, class G, bool kCenter>
__global__ void __launch_bounds__(kNormAnyThreads)
k_norm_dw_any(NormBwdArgs a) {
    const int64_t c = (int64_t)blockIdx.x * kNormAnyThreads + threadIdx.x;
    if (c >= a.d) return;
    const int p = blockIdx.y;
    float sw = 0.f, sb = 0.f;
    for (int64_t r = p; r < a.n; r += kNormAnyParts) {
        const float g = to_f32(static_cast<const G*>(a.dy)[r * a.ld_dy + c]);
        const float mu = kCenter ? a.mean[r] : 0.f;
        const float xh = (to_f32(static_cast<const T*>(a.x)[r * a.ld_x + c]) - mu) * a.rstd[r];
        sw += g * xh;
        sb += g;
    }
    if (a.part_w) a.part_w[(int64_t)p * a.d + c] = sw;
    if (a.part_b) a.part_b[(int64_t)p * a.d + c] = sb;
}

// ---------------------------------------------------------------- rows in registers

// A row is held by kTpr threads, kNormElems elements each: kTpr = 32 (a warp
// per row, four rows a CTA, no block-wide sums) up to 512 columns, then one
// CTA per row.  Persistent CTAs step through the rows.
//
// V > 1: rows of 16-byte vectors.  Each thread copies the vectors of its next
// rows into shared memory with cp.async and reads back only its own, so the
// ring of kStages rows needs no barrier and the loads of several rows are in
// flight while one is reduced and written.  V = 1 (any alignment, stride and
// width): element loads straight to registers.
constexpr int kNormElems = 16;
template <int kTpr>
constexpr int kNormThreads = kTpr < 128 ? 128 : kTpr;
// CTAs per SM that the registers (forward 64, backward 128 a thread) and the rings allow
template <int kTpr>
constexpr int kNormFwdCtas = 1024 / kNormThreads<kTpr>;
template <int kTpr>
constexpr int kNormBwdCtas = 512 / kNormThreads<kTpr>;
template <class T>
constexpr int kNormFwdStages = sizeof(T) == 2 ? 5 : 3;                           // 160 .. 192 KB of rings per SM
template <class T, class G>
constexpr int kNormBwdStages = 24 / (int)(sizeof(T) + sizeof(G));                // 192 KB of rings per SM

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 norm_lds(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a)
                 : "memory");
    return r;
}

// The values of one 16-byte vector.
__device__ __forceinline__ void norm_unpack(const uint4& q, float (&v)[4], float) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void norm_unpack(const uint4& q, float (&v)[8], __nv_bfloat16) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ void norm_unpack(const uint4& q, float (&v)[8], __half) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 norm_pack(const float (&v)[4], float) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 norm_pack(const float (&v)[8], __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 norm_pack(const float (&v)[8], __half) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements [i, i + V) of a weight or bias vector.
template <int V>
__device__ __forceinline__ void norm_vec_load(const NormVec& v, int i, float absent, float (&o)[V]) {
    if constexpr (V == 1) {
        o[0] = norm_vec_at(v, i, absent);
    } else {
        if (v.p == nullptr) {
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = absent;
        } else if (v.dtype == 2) {
#pragma unroll
            for (int h = 0; h < V / 4; ++h) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(v.p) + i) + h);
                o[4 * h] = f.x;
                o[4 * h + 1] = f.y;
                o[4 * h + 2] = f.z;
                o[4 * h + 3] = f.w;
            }
        } else if constexpr (V == 8) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const unsigned short*>(v.p) + i));
            if (v.dtype == 0) norm_unpack(q, o, __nv_bfloat16());
            else norm_unpack(q, o, __half());
        }
    }
}

// Sums of kCount values over the threads of a row, the same in each of them.
// `red` holds two buffers of 32 x kCount floats used in turn (`turn`), so one
// barrier per sum is enough.
template <int kTpr, int kCount>
__device__ __forceinline__ void norm_row_sum(float (&v)[kCount], float* red, int& turn) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
    if constexpr (kTpr > 32) {
        constexpr int kWarps = kTpr / 32;
        float* buf = red + turn * 64;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int c = 0; c < kCount; ++c) buf[c * 32 + (threadIdx.x >> 5)] = v[c];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kCount; ++c) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += buf[c * 32 + k];
            v[c] = s;
        }
    }
}

// The vectors of row `p` that this thread owns, into its ring slots at `dst`.
template <class T, int V, int kTpr>
__device__ __forceinline__ void norm_issue(const T* p, int t, int nvec, uint32_t dst) {
    constexpr int NV = kNormElems / V, kPer = V * (int)sizeof(T) / 16;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = k * kTpr + t;
        if (v < nvec) {
#pragma unroll
            for (int h = 0; h < kPer; ++h)
                cp_async16(dst + (k * kPer + h) * kNormThreads<kTpr> * 16, reinterpret_cast<const char*>(p + v * V) + 16 * h);
        }
    }
}
// Values of slot k (vector k kTpr + t of the row) as FP32.
template <class T, int V, int kTpr>
__device__ __forceinline__ void norm_slot(uint32_t src, int k, float (&o)[V]) {
    constexpr int kPer = V * (int)sizeof(T) / 16;
    if constexpr (kPer == 1) {
        norm_unpack(norm_lds(src + k * kNormThreads<kTpr> * 16), o, T());
    } else {   // FP32 values beside 16-bit ones: two vectors
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            float q[4];
            norm_unpack(norm_lds(src + (k * kPer + h) * kNormThreads<kTpr> * 16), q, 0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[4 * h + j] = q[j];
        }
    }
}

template <class T, int V, int kTpr, bool kCenter>
__global__ void __launch_bounds__(kNormThreads<kTpr>, kNormFwdCtas<kTpr>)
k_norm_fwd(NormFwdArgs a) {
    constexpr int NV = kNormElems / V, kThreads = kNormThreads<kTpr>, kRows = kThreads / kTpr;
    constexpr int kStages = kNormFwdStages<T>;
    constexpr uint32_t kStageBytes = kThreads * kNormElems * sizeof(T);
    extern __shared__ __align__(16) unsigned char norm_smem[];
    __shared__ float red[2 * 64];
    int turn = 0;
    const int t = threadIdx.x % kTpr, nvec = (int)a.d / V;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / kTpr;
    const uint32_t ring = V > 1 ? (uint32_t)__cvta_generic_to_shared(norm_smem) + threadIdx.x * 16 : 0;
    const T* x = static_cast<const T*>(a.x);
    if constexpr (V > 1) {
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) {
            if (r + k * step < a.n) norm_issue<T, V, kTpr>(x + (r + k * step) * a.ld_x, t, nvec, ring + k * kStageBytes);
            cp_async_commit();
        }
    }
    int stage = 0;
    for (; r < a.n; r += step) {
        float v[NV][V];
        if constexpr (V > 1) {
            const int64_t ahead = r + (kStages - 1) * step;
            const int into = stage == 0 ? kStages - 1 : stage - 1;
            if (ahead < a.n) norm_issue<T, V, kTpr>(x + ahead * a.ld_x, t, nvec, ring + into * kStageBytes);
            cp_async_commit();
            cp_async_wait<kStages - 1>();
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k * kTpr + t < nvec) norm_slot<T, V, kTpr>(ring + stage * kStageBytes, k, v[k]);
                else
#pragma unroll
                    for (int j = 0; j < V; ++j) v[k][j] = 0.f;
            }
            stage = stage == kStages - 1 ? 0 : stage + 1;
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) v[k][0] = k * kTpr + t < nvec ? to_f32(x[r * a.ld_x + k * kTpr + t]) : 0.f;
        }
        float mu = 0.f;
        if (kCenter) {
            float s[1] = {0.f};
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] += v[k][j];
            norm_row_sum<kTpr, 1>(s, red, turn);
            mu = s[0] * a.inv_d;
        }
        float q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (!kCenter || k * kTpr + t < nvec)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float c = v[k][j] - mu;
                    q[0] += c * c;
                }
        }
        norm_row_sum<kTpr, 1>(q, red, turn);
        const float rstd = __frsqrt_rn(q[0] * a.inv_d + a.eps);
        T* y = static_cast<T*>(a.y) + r * a.ld_y;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec) {
                float w[V], b[V];
                norm_vec_load<V>(a.w, i * V, 1.f, w);
                norm_vec_load<V>(a.b, i * V, 0.f, b);
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = (v[k][j] - mu) * rstd * w[j] + b[j];
                if constexpr (V > 1) *reinterpret_cast<uint4*>(y + i * V) = norm_pack(v[k], T());
                else y[i] = from_f32<T>(v[k][0]);
            }
        }
        if (t == 0) {
            if (kCenter && a.mean) a.mean[r] = mu;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dx and this CTA's partial row of dw (and db).  kFull: with centring (unless
// a.mean is null) and db; else RMS norm without db.
template <class T, class G, int V, int kTpr, bool kFull>
__global__ void __launch_bounds__(kNormThreads<kTpr>, kNormBwdCtas<kTpr>)
k_norm_bwd(NormBwdArgs a) {
    constexpr int NV = kNormElems / V, kThreads = kNormThreads<kTpr>, kRows = kThreads / kTpr;
    constexpr int kStages = kNormBwdStages<T, G>;
    constexpr uint32_t kXBytes = kThreads * kNormElems * sizeof(T);
    constexpr uint32_t kStageBytes = kXBytes + kThreads * kNormElems * sizeof(G);
    extern __shared__ __align__(16) unsigned char norm_smem[];
    __shared__ float red[2 * 64];
    int turn = 0;
    const int t = threadIdx.x % kTpr, nvec = (int)a.d / V;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / kTpr;
    const uint32_t ring = V > 1 ? (uint32_t)__cvta_generic_to_shared(norm_smem) + threadIdx.x * 16 : 0;
    const T* x = static_cast<const T*>(a.x);
    const G* dy = static_cast<const G*>(a.dy);
    const bool center = kFull && a.mean != nullptr;

    float w[NV][V], dw[NV][V], db[kFull ? NV : 1][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = k * kTpr + t;
        if (i < nvec) norm_vec_load<V>(a.w, i * V, 1.f, w[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (i >= nvec) w[k][j] = 0.f;
            dw[k][j] = 0.f;
            if (kFull) db[k][j] = 0.f;
        }
    }
    if constexpr (V > 1) {
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) {
            const int64_t q = r + k * step;
            if (q < a.n) {
                norm_issue<T, V, kTpr>(x + q * a.ld_x, t, nvec, ring + k * kStageBytes);
                norm_issue<G, V, kTpr>(dy + q * a.ld_dy, t, nvec, ring + k * kStageBytes + kXBytes);
            }
            cp_async_commit();
        }
    }
    float mu_next = 0.f, rstd_next = 0.f;
    if (r < a.n) {
        mu_next = center ? __ldg(a.mean + r) : 0.f;
        rstd_next = __ldg(a.rstd + r);
    }
    int stage = 0;
    for (; r < a.n; r += step) {
        const float mu = mu_next, rstd = rstd_next;
        if (r + step < a.n) {
            mu_next = center ? __ldg(a.mean + r + step) : 0.f;
            rstd_next = __ldg(a.rstd + r + step);
        }
        float xh[NV][V], g[NV][V];   // xh, then dx; dy, then dy w
        if constexpr (V > 1) {
            const int64_t ahead = r + (kStages - 1) * step;
            const int into = stage == 0 ? kStages - 1 : stage - 1;
            if (ahead < a.n) {
                norm_issue<T, V, kTpr>(x + ahead * a.ld_x, t, nvec, ring + into * kStageBytes);
                norm_issue<G, V, kTpr>(dy + ahead * a.ld_dy, t, nvec, ring + into * kStageBytes + kXBytes);
            }
            cp_async_commit();
            cp_async_wait<kStages - 1>();
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec) {
                if constexpr (V > 1) {
                    norm_slot<T, V, kTpr>(ring + stage * kStageBytes, k, xh[k]);
                    norm_slot<G, V, kTpr>(ring + stage * kStageBytes + kXBytes, k, g[k]);
                } else {
                    xh[k][0] = to_f32(x[r * a.ld_x + i]);
                    g[k][0] = to_f32(dy[r * a.ld_dy + i]);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xh[k][j] = (xh[k][j] - mu) * rstd;
                    dw[k][j] += g[k][j] * xh[k][j];
                    if (kFull) db[k][j] += g[k][j];
                    g[k][j] *= w[k][j];
                    s[0] += g[k][j] * xh[k][j];
                    if (kFull) s[1] += g[k][j];
                }
            }
        }
        if constexpr (V > 1) stage = stage == kStages - 1 ? 0 : stage + 1;
        if constexpr (kFull) {
            norm_row_sum<kTpr, 2>(s, red, turn);
        } else {
            float s0[1] = {s[0]};
            norm_row_sum<kTpr, 1>(s0, red, turn);
            s[0] = s0[0];
        }
        const float c2 = s[0] * a.inv_d, c1 = center ? s[1] * a.inv_d : 0.f;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec) {
#pragma unroll
                for (int j = 0; j < V; ++j) xh[k][j] = (g[k][j] - c1 - xh[k][j] * c2) * rstd;
                if constexpr (V > 1) *reinterpret_cast<uint4*>(dx + i * V) = norm_pack(xh[k], T());
                else dx[i] = from_f32<T>(xh[k][0]);
            }
        }
    }
    // the CTA's partial row
    if constexpr (kRows == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (a.part_w) a.part_w[(int64_t)blockIdx.x * a.d + i * V + j] = dw[k][j];
                    if (kFull && a.part_b) a.part_b[(int64_t)blockIdx.x * a.d + i * V + j] = db[k][j];
                }
            }
        }
    } else {
        // the rows' warps one after the other, through shared memory
        __shared__ float sum[kFull ? 2 : 1][kTpr * kNormElems];
        for (int q = 0; q < kRows; ++q) {
            if ((int)threadIdx.x / kTpr == q) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int i = k * kTpr + t;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        sum[0][i * V + j] = (q ? sum[0][i * V + j] : 0.f) + dw[k][j];
                        if (kFull) sum[kFull ? 1 : 0][i * V + j] = (q ? sum[kFull ? 1 : 0][i * V + j] : 0.f) + db[k][j];
                    }
                }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < (int)a.d; i += kThreads) {
            if (a.part_w) a.part_w[(int64_t)blockIdx.x * a.d + i] = sum[0][i];
            if (kFull && a.part_b) a.part_b[(int64_t)blockIdx.x * a.d + i] = sum[kFull ? 1 : 0][i];
        }
    }
}

// ---------------------------------------------------------------- partial rows

constexpr int kNormFoldCols = 32, kNormFoldRows = 16;

struct NormFoldArgs {
    const float *part_w, *part_b;   // [rows, d] or null
    int rows;
    int64_t d;
    float *dweight, *dbias;
    int accumulate;
};

// out[c] (+)= sum over the partial rows in a fixed order: kNormFoldRows
// threads share a column, each taking every kNormFoldRows-th row.
__global__ void __launch_bounds__(kNormFoldCols * kNormFoldRows)
k_norm_fold(NormFoldArgs a) {
    __shared__ float red[kNormFoldRows][kNormFoldCols + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float* part = blockIdx.y == 0 && a.part_w ? a.part_w : a.part_b;
    float* out = blockIdx.y == 0 && a.part_w ? a.dweight : a.dbias;
    const int tx = threadIdx.x % kNormFoldCols, ty = threadIdx.x / kNormFoldCols;
    const int64_t c = (int64_t)blockIdx.x * kNormFoldCols + tx;
    float s = 0.f;
    if (c < a.d) {
#pragma unroll 4
        for (int r = ty; r < a.rows; r += kNormFoldRows) s += __ldcs(part + (int64_t)r * a.d + c);
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < a.d) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kNormFoldRows; ++k) t += red[k][tx];
        out[c] = a.accumulate ? out[c] + t : t;
    }
}

}  // namespace flp
