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

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

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
    int64_t dp;      // d rounded up to 4: a partial row
    float* part_w;   // [min(n, kNormParts), dp] partial sums of dy xh, or null
    float* part_b;   // [min(n, kNormParts), dp] partial sums of dy, or null
    float *dweight, *dbias;   // what the partial rows are folded into
    int accumulate;
    const void* add;   // rows added to dx (the residual stream's gradient), of x's type; null or kAdd
    int64_t ld_add;
};

// Most rows of partial weight gradients: a constant, so that the order of the sum
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
// tile holds.  Bound by its element-wise reads (4096 x 20480 BF16, RMS norm: forward 157 us,
// 2.1 TB/s; the backward, from 8193 columns on, at 8192 x 12288 425 us, 1.4 TB/s).
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
            const float r0 = a.add ? to_f32(static_cast<const T*>(a.add)[r * a.ld_add + i]) : 0.f;
            dx[i] = from_f32<T>(a.add ? __fmaf_rn(g - c1 - xh * c2, rstd, r0) : (g - c1 - xh * c2) * rstd);
        }
    }
}

// Partial sums over the rows p, p + kNormAnyParts, ... of one column per thread, p < n.
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
    if (a.part_w) a.part_w[(int64_t)p * a.dp + c] = sw;
    if (a.part_b) a.part_b[(int64_t)p * a.dp + c] = sb;
}

// ---------------------------------------------------------------- partial rows

// out[c] (+)= sum over the partial rows in an order fixed by their number, 8
// columns (a sector) a team of warps and turn.  A warp reads 4 rows at a time, 16
// loads in flight a lane, so a team has a warp per 64 rows.  (With the whole CTA on
// each 8 columns, a few rows' sums took 27 us at 7 x 1024 and 17 at 64 x 4096, now
// 4.6 and 6.2; with 32 columns a CTA most CTAs of a narrow norm had none.)
__host__ __device__ __forceinline__ int norm_fold_team(int rows, int warps) {
    int w = 1;
    while (w < warps && 64 * w < rows) w *= 2;
    return w;
}
template <int kWarps>
__device__ __forceinline__ void norm_fold(const NormBwdArgs& a, int rows, float (*red)[8]) {
    const int col = threadIdx.x & 7, sub = (threadIdx.x >> 3) & 3, warp = threadIdx.x >> 5;
    const int w = norm_fold_team(rows, kWarps), teams = kWarps / w, team = warp / w, ty = warp % w;
    const int groups = (int)((a.d + 7) / 8), in_w = a.part_w ? groups : 0, all = in_w + (a.part_b ? groups : 0);
    for (int g0 = blockIdx.x * teams; g0 < all; g0 += gridDim.x * teams) {
        const int g = g0 + team;
        const bool second = g >= in_w;
        const float* part = second ? a.part_b : a.part_w;
        float* out = second ? a.dbias : a.dweight;
        const int64_t c = (int64_t)(second ? g - in_w : g) * 8 + col;
        const bool mine = g < all && c < a.d;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        if (mine) {
            for (int r = ty * 4 + sub; r < rows; r += 64 * w) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int q = r + 4 * k * w;
                    v[k] = q < rows ? __ldcg(part + (int64_t)q * a.dp + c) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) s[k & 3] += v[k];
            }
        }
        float t = (s[0] + s[1]) + (s[2] + s[3]);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        if (w > 1) {   // alike in the whole CTA
            __syncthreads();   // the last turn's readers
            if (sub == 0) red[warp][col] = t;
            __syncthreads();
            t = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) t += k < w ? red[team * w + k][col] : 0.f;
        }
        if (ty == 0 && sub == 0 && mine) out[c] = a.accumulate ? out[c] + t : t;
    }
}

constexpr int kNormFoldThreads = 256;
template <int kThreads>
__global__ void __launch_bounds__(kThreads)
k_norm_fold(NormBwdArgs a, int rows) {
    __shared__ float red[kThreads / 32][8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    norm_fold<kThreads / 32>(a, rows, red);
}

// ---------------------------------------------------------------- rows in registers

// A row is held by kTpr threads, at most kNormElems elements each: part of a warp
// up to 256 columns, a warp up to 512, in the forward two up to 1024 (no block-wide sums,
// several rows a CTA), then one CTA per row.  Persistent CTAs step through the rows and copy the
// next ones into a ring in shared memory with cp.async, so that the loads of several
// rows are in flight while one is reduced and written.
//
// A thread owns vectors of V elements, V being 16 bytes of the wider of x and dy,
// so that the lanes' copies of both are contiguous (with 8 elements a lane the
// FP32 dy was fetched in two halves of every sector: the backward kernel at
// 32768 x 4096 took 217 us, now 150).
// kAligned (16-byte aligned rows of whole vectors): a thread copies only its own
// vectors and reads back only its own; the ring needs no barrier.
// Otherwise (any alignment, stride and width): the row's threads copy the aligned
// 16-byte blocks that hold the row and shift their vectors out of two neighbours;
// results go back through shared memory as aligned blocks, the row's first and last
// element by element.  (Element loads and stores, one value a lane, were bound by
// their instructions: 5003 x 1031 FP16, forward and backward, 44 us, now 36.  Aligned
// rows by blocks: the backward at 16384 x 4096 120 us, 69 by vectors.)
//
// What bounds it: memory (32768 x 4096 BF16: forward 88 us, 6.1 TB/s, backward with FP32
// dy 150 us, 7.1 TB/s; 2 M rows of 64: 5.2 and 5.0 TB/s), but for the instructions of the
// shifted rows and their latencies (130182 x 1031: 2.3 and 2.1 TB/s; 68% of the issue slots
// in the forward, 46% at 24% occupancy in the backward).
constexpr int kNormElems = 16;
template <int kTpr>
constexpr int kNormThreads = kTpr < 128 ? 128 : kTpr;
// CTAs per SM that the registers (forward 64, backward 128 a thread) and the rings allow
template <int kTpr>
constexpr int kNormFwdCtas = 1024 / kNormThreads<kTpr>;
template <int kTpr>
constexpr int kNormBwdCtas = 512 / kNormThreads<kTpr>;
// rows of the ring: 160 .. 192 KB per SM; in the forward one less where an unaligned row's
// staged result would not fit beside it (rows of FP32 by the most threads), so that every
// width is summed in one order, wherever its rows lie
template <class T, int kTpr, bool kAligned>
constexpr int kNormFwdStages = sizeof(T) == 2 ? 5 : kAligned || kTpr < 1024 ? 3 : 2;
template <class T, class G>
constexpr int kNormBwdStages = 24 / (int)(sizeof(T) + sizeof(G));

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of an aligned 16-byte block, zeros after them.
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// V consecutive values as raw words, and their FP32 values.
template <int kBytes>
struct NormWords {
    uint32_t w[kBytes / 4];
};
template <int kBytes>
__device__ __forceinline__ NormWords<kBytes> norm_lds(uint32_t a) {
    NormWords<kBytes> r;
    if constexpr (kBytes == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(a) : "memory");
    else asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(a) : "memory");
    return r;
}
template <int kBytes>
__device__ __forceinline__ NormWords<kBytes> norm_ldg(const void* p) {
    NormWords<kBytes> r;
    if constexpr (kBytes == 16) {
        const uint4 q = __ldg(static_cast<const uint4*>(p));
        r.w[0] = q.x; r.w[1] = q.y; r.w[2] = q.z; r.w[3] = q.w;
    } else {
        const uint2 q = __ldg(static_cast<const uint2*>(p));
        r.w[0] = q.x; r.w[1] = q.y;
    }
    return r;
}
// The same of memory that this kernel may write (dx in place of what is added to it).
template <int kBytes>
__device__ __forceinline__ NormWords<kBytes> norm_ld(const void* p) {
    NormWords<kBytes> r;
    if constexpr (kBytes == 16)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "l"(p) : "memory");
    else asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "l"(p) : "memory");
    return r;
}
template <int kBytes>
__device__ __forceinline__ void norm_stg(void* p, const NormWords<kBytes>& r) {
    if constexpr (kBytes == 16) *static_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else *static_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
}
template <class T, int V>
__device__ __forceinline__ void norm_unpack(const NormWords<V * (int)sizeof(T)>& q, float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = __uint_as_float(q.w[k]);
    } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q.w[k]));
                v[2 * k] = f.x;
                v[2 * k + 1] = f.y;
            } else {
                v[2 * k] = __uint_as_float(q.w[k] << 16);
                v[2 * k + 1] = __uint_as_float(q.w[k] & 0xffff0000u);
            }
        }
    }
}
template <class T, int V>
__device__ __forceinline__ NormWords<V * (int)sizeof(T)> norm_pack(const float (&v)[V]) {
    NormWords<V * (int)sizeof(T)> q;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) q.w[k] = __float_as_uint(v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
                q.w[k] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                q.w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    return q;
}

// Elements [i, i + V) of a vector of type W, in 16-byte loads at most.
template <class W, int V>
__device__ __forceinline__ void norm_vec_load(const W* p, int i, float (&o)[V]) {
    if constexpr (V * sizeof(W) <= 16) {
        norm_unpack<W, V>(norm_ldg<V * (int)sizeof(W)>(p + i), o);
    } else {
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            float q[4];
            norm_unpack<W, 4>(norm_ldg<16>(p + i + 4 * h), q);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[4 * h + j] = q[j];
        }
    }
}

// Barrier of a row's threads.
template <int kTpr>
__device__ __forceinline__ void norm_row_sync() {
    if constexpr (kTpr <= 32) __syncwarp();
    else if constexpr (kTpr == kNormThreads<kTpr>) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / kTpr), "n"(kTpr) : "memory");
}

// Sums of kCount values over the threads of a row, the same in each of them.
// `red` holds two buffers of 32 x kCount floats used in turn (`turn`), so one
// barrier per sum is enough.
template <int kTpr, int kCount>
__device__ __forceinline__ void norm_row_sum(float (&v)[kCount], float* red, int& turn) {
#pragma unroll
    for (int o = (kTpr < 32 ? kTpr : 32) / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int c = 0; c < kCount; ++c) v[c] += __shfl_xor_sync(0xffffffffu, v[c], o);
    if constexpr (kTpr > 32) {
        constexpr int kWarps = kTpr / 32;
        const int warp = threadIdx.x >> 5, first = warp / kWarps * kWarps;   // of the row
        float* buf = red + turn * 64;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int c = 0; c < kCount; ++c) buf[c * 32 + warp] = v[c];
        norm_row_sync<kTpr>();
#pragma unroll
        for (int c = 0; c < kCount; ++c) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += buf[c * 32 + first + k];
            v[c] = s;
        }
    }
}

// Bytes of a ring slot of one unaligned row: its 16-byte blocks, one more than
// aligned ones would take.
template <class T>
__host__ __device__ constexpr uint32_t norm_pitch(int64_t d) {
    return (uint32_t)((d * (int64_t)sizeof(T) + 15) / 16 + 1) * 16;
}
template <class T>
__device__ __forceinline__ uint32_t norm_misaligned(const T* p) {
    return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
}

// Copies row `r` of `base` (rows of d elements, ld apart) into the ring: kAligned:
// this thread's vectors, into its own places from `dst` on; else this thread's
// blocks of the row, whose first byte comes to dst + (address mod 16).
template <class T, int V, int kTpr, bool kAligned>
__device__ __forceinline__ void norm_issue(const T* base, int64_t r, int64_t ld, int d, int t, uint32_t dst) {
    const T* p = base + r * ld;
    if constexpr (kAligned) {
        constexpr int NV = kNormElems / V, kBytes = V * (int)sizeof(T);
        const int nvec = d / V;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int v = k * kTpr + t;
            if (v < nvec) cp_async<kBytes>(dst + k * kNormThreads<kTpr> * kBytes, p + v * V);
        }
    } else {
        const int mis = (int)norm_misaligned(p);
        const int bytes = mis + d * (int)sizeof(T);
        const char* first = reinterpret_cast<const char*>(p) - mis;
        for (int b = t * 16; b < bytes; b += kTpr * 16) {
            const char* src = first + b;
            if (src >= reinterpret_cast<const char*>(base)) {
                cp_async_part(dst + b, src, bytes - b < 16 ? bytes - b : 16);
            } else {   // this block starts before the whole buffer: element by element
                for (int o = mis; o < 16 && o < bytes; o += (int)sizeof(T)) {
                    if constexpr (sizeof(T) == 4)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + o),
                                     "r"(*reinterpret_cast<const unsigned int*>(first + o)) : "memory");
                    else
                        asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + o),
                                     "h"(*reinterpret_cast<const unsigned short*>(first + o)) : "memory");
                }
            }
        }
    }
}
// kBytes (8 or 16) bytes of shared memory from byte `at` on, an element's multiple:
// two aligned pieces, shifted together.
template <int kBytes>
__device__ __forceinline__ NormWords<kBytes> norm_lds_shifted(uint32_t at) {
    constexpr int N = kBytes / 4;
    const uint32_t a = at & ~(uint32_t)(kBytes - 1);
    const NormWords<kBytes> lo = norm_lds<kBytes>(a), hi = norm_lds<kBytes>(a + kBytes);
    uint32_t w[2 * N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        w[k] = lo.w[k];
        w[N + k] = hi.w[k];
    }
    const uint32_t words = (at >> 2) & (N - 1), bits = (at & 3u) * 8;
    // by whole words (the same for the whole row), then by half a word
#pragma unroll
    for (int s = N / 2; s >= 1; s >>= 1) {
        if (words & s) {
#pragma unroll
            for (int k = 0; k + s < 2 * N; ++k) w[k] = w[k + s];
        }
    }
    NormWords<kBytes> r;
#pragma unroll
    for (int k = 0; k < N; ++k) r.w[k] = __funnelshift_r(w[k], w[k + 1], bits);
    return r;
}
// Vector k kTpr + t of the row copied to `src`; !kAligned: `src` is the row's first byte.
template <class T, int V, int kTpr, bool kAligned>
__device__ __forceinline__ void norm_slot(uint32_t src, int k, int t, float (&o)[V]) {
    constexpr int kBytes = V * (int)sizeof(T);
    if constexpr (kAligned) norm_unpack<T, V>(norm_lds<kBytes>(src + k * kNormThreads<kTpr> * kBytes), o);
    else norm_unpack<T, V>(norm_lds_shifted<kBytes>(src + (k * kTpr + t) * kBytes), o);
}
// After the wait for this thread's copies: those of the row's other threads.
template <int kTpr, bool kAligned>
__device__ __forceinline__ void norm_copied() {
    if constexpr (!kAligned) norm_row_sync<kTpr>();
}
// The row of d elements staged at `src` (16-byte aligned) to p, at any alignment.
template <class T, int kTpr>
__device__ __forceinline__ void norm_store_row(T* p, int d, int t, uint32_t src) {
    const int mis = (int)norm_misaligned(p), bytes = mis + d * (int)sizeof(T);
    char* first = reinterpret_cast<char*>(p) - mis;
    for (int b = t * 16; b < bytes; b += kTpr * 16) {
        if (b >= mis && b + 16 <= bytes) {
            norm_stg<16>(first + b, norm_lds_shifted<16>(src + b - mis));
        } else {
            for (int o = b > mis ? b : mis; o < b + 16 && o < bytes; o += (int)sizeof(T)) {
                if constexpr (sizeof(T) == 4) {
                    uint32_t v;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(src + o - mis) : "memory");
                    *reinterpret_cast<uint32_t*>(first + o) = v;
                } else {
                    unsigned short v;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(src + o - mis) : "memory");
                    *reinterpret_cast<unsigned short*>(first + o) = v;
                }
            }
        }
    }
}
template <int kBytes>
__device__ __forceinline__ void norm_sts(uint32_t a, const NormWords<kBytes>& r) {
    if constexpr (kBytes == 16)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                     "r"(r.w[3]) : "memory");
    else asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(r.w[0]), "r"(r.w[1]) : "memory");
}
// Vector i of a weight or bias vector of d elements; a vector that is cut by the end, or
// a whole array that is not aligned for it, element by element (absent ones 0).
template <class W, int V, bool kAligned>
__device__ __forceinline__ void norm_vec_get(const W* p, bool aligned, int i, int d, float (&o)[V]) {
    if (kAligned || (aligned && (i + 1) * V <= d)) {
        norm_vec_load<W, V>(p, i * V, o);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = i * V + j < d ? to_f32(__ldg(p + i * V + j)) : 0.f;
    }
}

template <class T, class W, int kTpr, bool kCenter, bool kAligned>
__global__ void __launch_bounds__(kNormThreads<kTpr>, kNormFwdCtas<kTpr>)
k_norm_fwd(NormFwdArgs a) {
    constexpr int V = 16 / (int)sizeof(T), NV = kNormElems / V;
    constexpr int kThreads = kNormThreads<kTpr>, kRows = kThreads / kTpr, kStages = kNormFwdStages<T, kTpr, kAligned>;
    extern __shared__ __align__(16) unsigned char norm_smem[];
    __shared__ float red[2 * 64];
    int turn = 0;
    const int t = threadIdx.x % kTpr, d = (int)a.d, nvec = (d + V - 1) / V;
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / kTpr;
    // kAligned: the thread's places; else the row's slot, and after the ring its staged result
    const uint32_t pitch = kAligned ? kThreads * kNormElems * (uint32_t)sizeof(T) : norm_pitch<T>(d) * kRows;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(norm_smem) +
                          (kAligned ? threadIdx.x * 16 : threadIdx.x / kTpr * norm_pitch<T>(d));
    const T* x = static_cast<const T*>(a.x);
    const W *w = static_cast<const W*>(a.w.p), *b = static_cast<const W*>(a.b.p);
    const bool w_al = norm_misaligned(w) == 0, b_al = norm_misaligned(b) == 0;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
        if (r + k * step < a.n) norm_issue<T, V, kTpr, kAligned>(x, r + k * step, a.ld_x, d, t, ring + k * pitch);
        cp_async_commit();
    }
    int stage = 0;
    // the rows of a warp take their turns together, the last of them without a row
    const int64_t before = kTpr < 32 ? (threadIdx.x & 31) / kTpr : 0;
    for (; r - before < a.n; r += step) {
        const bool live = kTpr >= 32 || r < a.n;
        float v[NV][V];
        const int64_t ahead = r + (kStages - 1) * step;
        const int into = stage == 0 ? kStages - 1 : stage - 1;
        if (ahead < a.n) norm_issue<T, V, kTpr, kAligned>(x, ahead, a.ld_x, d, t, ring + into * pitch);
        cp_async_commit();
        cp_async_wait<kStages - 1>();
        norm_copied<kTpr, kAligned>();
        const uint32_t src = ring + stage * pitch + (kAligned ? 0 : norm_misaligned(x + r * a.ld_x));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec && live) {
                norm_slot<T, V, kTpr, kAligned>(src, k, t, v[k]);
                if constexpr (!kAligned) {
                    if ((i + 1) * V > d) {
#pragma unroll
                        for (int j = 0; j < V; ++j) v[k][j] = i * V + j < d ? v[k][j] : 0.f;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = 0.f;
            }
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
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
            const int i = k * kTpr + t;
            if (!kCenter || i < nvec) {
                const int have = kAligned || !kCenter ? V : d - i * V;   // what lies past the row is not mu away
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float c = v[k][j] - mu;
                    if (kAligned || !kCenter || j < have) q[0] += c * c;
                }
            }
        }
        norm_row_sum<kTpr, 1>(q, red, turn);
        const float rstd = __frsqrt_rn(q[0] * a.inv_d + a.eps);
        T* y = static_cast<T*>(a.y) + r * a.ld_y;
        const uint32_t out = ring + kStages * pitch;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec && live) {
                float f[V];
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = (v[k][j] - mu) * rstd;
                if (w != nullptr) {
                    norm_vec_get<W, V, kAligned>(w, w_al, i, d, f);
#pragma unroll
                    for (int j = 0; j < V; ++j) v[k][j] *= f[j];
                }
                if (b != nullptr) {
                    norm_vec_get<W, V, kAligned>(b, b_al, i, d, f);
#pragma unroll
                    for (int j = 0; j < V; ++j) v[k][j] += f[j];
                }
                if constexpr (kAligned) norm_stg(y + i * V, norm_pack<T, V>(v[k]));
                else norm_sts(out + i * 16, norm_pack<T, V>(v[k]));
            }
        }
        if constexpr (!kAligned) {
            norm_copied<kTpr, kAligned>();   // the whole row is staged
            if (live) norm_store_row<T, kTpr>(y, d, t, out);
        }
        if (t == 0 && live) {
            if (kCenter && a.mean) a.mean[r] = mu;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

// dx and this CTA's partial row of dw (and db): the first `parts` CTAs step through the
// rows.  The partial rows are folded after a barrier of the grid (a cooperative launch;
// `grid_fold`), saving the launch of k_norm_fold: it costs a caller as much as the kernel
// on small batches.
// kFull: with centring (unless a.mean is null) and db; else RMS norm without db.
// kAdd: a.add is added to dx.  Its row is loaded into registers while the sums are taken, not
// through the ring (a row's turn of 4096 columns is about 2 us, a load 1).
template <class T, class G, int kTpr, bool kFull, bool kAligned, bool kAdd = false>
__global__ void __launch_bounds__(kNormThreads<kTpr>, kNormBwdCtas<kTpr>)
k_norm_bwd(NormBwdArgs a, int parts, int grid_fold) {
    constexpr int V = 16 / (int)sizeof(G), NV = kNormElems / V;
    constexpr int kThreads = kNormThreads<kTpr>, kRows = kThreads / kTpr;
    constexpr int kStages = kNormBwdStages<T, G>;
    extern __shared__ __align__(16) unsigned char norm_smem[];
    __shared__ float red[2 * 64];
    int turn = 0;
    const int t = threadIdx.x % kTpr, d = (int)a.d, nvec = (d + V - 1) / V;
    // the CTAs from `parts` on are here for the fold alone: no row of theirs has a partial row
    const int64_t step = (int64_t)parts * kRows;
    int64_t r = ((int)blockIdx.x < parts ? (int64_t)blockIdx.x * kRows : a.n) + threadIdx.x / kTpr;
    // kAligned: the thread's places; else the rows' slots, and after the ring the staged dx
    const uint32_t xpitch = kAligned ? kThreads * kNormElems * (uint32_t)sizeof(T) : norm_pitch<T>(d) * kRows;
    const uint32_t pitch = xpitch + (kAligned ? kThreads * kNormElems * (uint32_t)sizeof(G) : norm_pitch<G>(d) * kRows);
    const uint32_t smem = (uint32_t)__cvta_generic_to_shared(norm_smem);
    const uint32_t ring_x =
        smem + (kAligned ? threadIdx.x * V * (uint32_t)sizeof(T) : threadIdx.x / kTpr * norm_pitch<T>(d));
    const uint32_t ring_g =
        smem + xpitch + (kAligned ? threadIdx.x * V * (uint32_t)sizeof(G) : threadIdx.x / kTpr * norm_pitch<G>(d));
    const T* x = static_cast<const T*>(a.x);
    const G* dy = static_cast<const G*>(a.dy);
    const bool center = kFull && a.mean != nullptr;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
        if (r + k * step < a.n) {
            norm_issue<T, V, kTpr, kAligned>(x, r + k * step, a.ld_x, d, t, ring_x + k * pitch);
            norm_issue<G, V, kTpr, kAligned>(dy, r + k * step, a.ld_dy, d, t, ring_g + k * pitch);
        }
        cp_async_commit();
    }
    float w[NV][V], dw[NV][V], db[kFull ? NV : 1][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = k * kTpr + t;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[k][j] = i < nvec ? 1.f : 0.f;
            dw[k][j] = 0.f;
            if (kFull) db[k][j] = 0.f;
        }
    }
    if (a.w.p != nullptr) {
        const bool al = norm_misaligned(static_cast<const char*>(a.w.p)) == 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec) {
                if (sizeof(T) == 4 || a.w.dtype == 2)
                    norm_vec_get<float, V, kAligned>(static_cast<const float*>(a.w.p), al, i, d, w[k]);
                else norm_vec_get<T, V, kAligned>(static_cast<const T*>(a.w.p), al, i, d, w[k]);
            }
        }
    }
    float mu_next = 0.f, rstd_next = 0.f;
    if (r < a.n) {
        mu_next = center ? __ldg(a.mean + r) : 0.f;
        rstd_next = __ldg(a.rstd + r);
    }
    int stage = 0;
    const int64_t before = kTpr < 32 ? (threadIdx.x & 31) / kTpr : 0;
    for (; r - before < a.n; r += step) {
        const bool live = kTpr >= 32 || r < a.n;
        const float mu = mu_next, rstd = rstd_next;
        if (r + step < a.n) {
            mu_next = center ? __ldg(a.mean + r + step) : 0.f;
            rstd_next = __ldg(a.rstd + r + step);
        }
        const int64_t ahead = r + (kStages - 1) * step;
        const int into = stage == 0 ? kStages - 1 : stage - 1;
        if (ahead < a.n) {
            norm_issue<T, V, kTpr, kAligned>(x, ahead, a.ld_x, d, t, ring_x + into * pitch);
            norm_issue<G, V, kTpr, kAligned>(dy, ahead, a.ld_dy, d, t, ring_g + into * pitch);
        }
        cp_async_commit();
        cp_async_wait<kStages - 1>();
        norm_copied<kTpr, kAligned>();
        NormWords<V * (int)sizeof(T)> add[kAdd && kAligned ? NV : 1];
        const T* add_row = kAdd ? static_cast<const T*>(a.add) + r * a.ld_add : nullptr;
        if constexpr (kAdd && kAligned) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (k * kTpr + t < nvec && live) add[k] = norm_ld<V * (int)sizeof(T)>(add_row + (k * kTpr + t) * V);
        }
        const uint32_t sx = ring_x + stage * pitch + (kAligned ? 0 : norm_misaligned(x + r * a.ld_x));
        const uint32_t sg = ring_g + stage * pitch + (kAligned ? 0 : norm_misaligned(dy + r * a.ld_dy));
        float xh[NV][V], g[NV][V];   // xh, then dx; dy, then dy w
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec && live) {
                norm_slot<T, V, kTpr, kAligned>(sx, k, t, xh[k]);
                norm_slot<G, V, kTpr, kAligned>(sg, k, t, g[k]);
                if constexpr (!kAligned) {
                    if ((i + 1) * V > d) {   // past the row: nothing
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            xh[k][j] = i * V + j < d ? xh[k][j] : mu;
                            g[k][j] = i * V + j < d ? g[k][j] : 0.f;
                        }
                    }
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
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if constexpr (kFull) {
            norm_row_sum<kTpr, 2>(s, red, turn);
        } else {
            float s0[1] = {s[0]};
            norm_row_sum<kTpr, 1>(s0, red, turn);
            s[0] = s0[0];
        }
        const float c2 = s[0] * a.inv_d, c1 = center ? s[1] * a.inv_d : 0.f;
        T* dx = static_cast<T*>(a.dx) + r * a.ld_dx;
        const uint32_t out = smem + kStages * pitch + threadIdx.x / kTpr * norm_pitch<T>(d);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec && live) {
                if constexpr (kAdd) {
                    float e[V];
                    if constexpr (kAligned) {
                        norm_unpack<T, V>(add[k], e);
                    } else {
#pragma unroll
                        for (int j = 0; j < V; ++j) e[j] = i * V + j < d ? to_f32(add_row[i * V + j]) : 0.f;
                    }
                    // fused in either form: the bits of a row do not depend on where it lies
#pragma unroll
                    for (int j = 0; j < V; ++j) xh[k][j] = __fmaf_rn(g[k][j] - c1 - xh[k][j] * c2, rstd, e[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) xh[k][j] = (g[k][j] - c1 - xh[k][j] * c2) * rstd;
                }
                if constexpr (kAligned) norm_stg(dx + i * V, norm_pack<T, V>(xh[k]));
                else norm_sts(out + i * V * (uint32_t)sizeof(T), norm_pack<T, V>(xh[k]));
            }
        }
        if constexpr (!kAligned) {
            norm_copied<kTpr, kAligned>();   // the whole row is staged
            if (live) norm_store_row<T, kTpr>(dx, d, t, out);
        }
    }
    // the CTA's partial row
    if ((int)blockIdx.x >= parts) {
        // only here to fold
    } else if constexpr (kRows == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = k * kTpr + t;
            if (i < nvec) {
                const int64_t at = (int64_t)blockIdx.x * a.dp + i * V;
#pragma unroll
                for (int h = 0; h < V; h += 4) {   // past the row, but inside its padding: zeros
                    if (!kAligned && i * V + h >= d) break;
                    if (a.part_w)
                        *reinterpret_cast<float4*>(a.part_w + at + h) =
                            make_float4(dw[k][h], dw[k][h + 1], dw[k][h + 2], dw[k][h + 3]);
                    if constexpr (kFull)
                        if (a.part_b)
                            *reinterpret_cast<float4*>(a.part_b + at + h) =
                                make_float4(db[k][h], db[k][h + 1], db[k][h + 2], db[k][h + 3]);
                }
            }
        }
    } else {
        // the rows of a warp by shuffles, then the warps (or pairs of them) one after the
        // other, through shared memory
        __shared__ float sum[kFull ? 2 : 1][kTpr * kNormElems];
        constexpr int kGroup = kTpr < 32 ? 32 : kTpr;
#pragma unroll
        for (int o = kTpr; o < 32; o <<= 1)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    dw[k][j] += __shfl_xor_sync(0xffffffffu, dw[k][j], o);
                    if (kFull) db[k][j] += __shfl_xor_sync(0xffffffffu, db[k][j], o);
                }
        for (int q = 0; q < kThreads / kGroup; ++q) {
            if ((int)threadIdx.x / kGroup == q && (int)threadIdx.x % kGroup < kTpr) {
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
        for (int i = threadIdx.x; i < d; i += kThreads) {
            if (a.part_w) a.part_w[(int64_t)blockIdx.x * a.dp + i] = sum[0][i];
            if (kFull && a.part_b) a.part_b[(int64_t)blockIdx.x * a.dp + i] = sum[kFull ? 1 : 0][i];
        }
    }
    if (grid_fold) {
        __shared__ float fold[kThreads / 32][8];
        cooperative_groups::this_grid().sync();
        norm_fold<kThreads / 32>(a, parts, fold);
    }
}

}  // namespace flp
