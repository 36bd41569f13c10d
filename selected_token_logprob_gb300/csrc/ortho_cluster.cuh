// The Newton-Schulz orthogonalisation of a matrix with a side of at most 128 in
// one launch: a cluster of up to 16 CTAs holds X for all steps, each CTA a slice
// of its columns.
//
// Per step (numerics as in the tiled kernels, but X is carried in FP32):
//   Gram   each CTA multiplies its slice, X_c X_c^T, on the tensor cores; the
//          FP32 partials are added over the cluster in CTA order through
//          distributed shared memory, each CTA adding some of the rows and
//          writing the FP16 A0 and the FP32 diagonal into every CTA;
//   Poly   every CTA forms B0 and e for itself (128 x 128 products);
//   Apply  X, in tensor memory, is scaled by a + e_i row by row and the tensor
//          cores add B0 X_hi onto it; its FP16 rounding becomes the next X_hi.  But for
//          the last steps, whose noise is hardly multiplied any more, they add B0 X_lo,
//          too, X_lo = X - X_hi in FP16, so that no row has to leave it out (f in
//          ortho_kernels.cuh; with f five steps were off by 2e-3 on a 5 x 5 matrix where
//          e had 8e-4.  64 x 1024: 27.4 us without X_lo, now 28.8).
// X_hi lies in shared memory as blocks of 64 columns whose 128-byte rows are
// K-major for Gram (K = columns) and MN-major for Apply (K = rows): one copy
// serves both.  What bounds it is the chain of latencies of a step (two cluster
// barriers, three waits for the tensor cores): about 5 us, against 16 us of the
// three launches of the tiled form.
#pragma once

#include "ortho_kernels.cuh"

namespace flp {

constexpr int kOrthCluThreads = 256;      // warps w and w + 4 share 32 rows, and split the columns
constexpr int kOrthCluMaxBlocks = 6;      // 64-column blocks of X a CTA: 384 columns of tensor memory
constexpr int kOrthCluMaxCtas = 16;
constexpr int kOrthMaxSteps = 64;
constexpr uint32_t kOrthBlockBytes = 128 * 128;   // 128 rows of 64 FP16
constexpr uint32_t kOrthGramCol = 384;            // tensor-memory column of Gram's and Poly's result
constexpr uint32_t kOrthCluX = 0;
constexpr uint32_t kOrthCluA = kOrthCluX + kOrthCluMaxBlocks * kOrthBlockBytes;   // A0, then B0 in its place
constexpr uint32_t kOrthCluP = kOrthCluA + 2 * kOrthBlockBytes;   // FP32 partials, X_lo, or staged columns
constexpr uint32_t kOrthCluD = kOrthCluP + kOrthCluMaxBlocks * kOrthBlockBytes;
constexpr uint32_t kOrthCluE = kOrthCluD + 512;
constexpr uint32_t kOrthCluMisc = kOrthCluE + 512;   // sums of the CTAs, barrier, TMEM address, scale
constexpr size_t kOrthCluSmem = 1024 + kOrthCluMisc + 256;
static_assert(kOrthCluSmem <= 232448, "shared memory per CTA");

struct OrthCluArgs {
    const void* x;
    int64_t ld, stride;
    int64_t m, n;             // of X (m <= 128)
    int mp;                   // 64 or 128
    int blocks;               // 64-column blocks of X
    int transposed, vec;      // X = x^T; x's rows are whole, aligned 16-byte vectors
    int steps;
    float eps, scale;
    void* out;
    int out_dtype, vec_out;
    int64_t ld_out, stride_out;
    float coef[3 * kOrthMaxSteps];
    float stray[kOrthMaxSteps];
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void dsm_st2(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void dsm_st(uint32_t a, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
// MN-major operand whose 64-column blocks lie kOrthBlockBytes apart.
__device__ __forceinline__ uint64_t orth_desc_mn_block(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kOrthBlockBytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__host__ __device__ constexpr uint32_t orth_idesc_n(int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// Address of 16-byte piece j of row r of a 64-column block.
__device__ __forceinline__ uint32_t orth_block_piece(uint32_t block, int r, int j) {
    return block + (uint32_t)r * 128 + (uint32_t)((j ^ (r & 7)) * 16);
}
template <class T>
__global__ void __launch_bounds__(kOrthCluThreads, 1)
k_orth_cluster(const __grid_constant__ OrthCluArgs p) {
    extern __shared__ __align__(1024) unsigned char clu_smem_raw[];
    const uint32_t raw = smem_u32(clu_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in every CTA
    const uint32_t sx = base + kOrthCluX, sa = base + kOrthCluA, sp = base + kOrthCluP, sd = base + kOrthCluD,
                   se = base + kOrthCluE, sums = base + kOrthCluMisc, bar = sums + 64, slot = sums + 80,
                   red = sums + 96, sums_top = sums + 128, sums_again = sums + 192;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane;
    const bool rows_here = quarter * 32 < p.mp;   // uniform over the warp
    uint32_t rank, ctas;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int64_t batch = blockIdx.x / ctas;
    const int blk0 = (int)((int64_t)p.blocks * rank / ctas), blk1 = (int)((int64_t)p.blocks * (rank + 1) / ctas);
    const int nblk = blk1 - blk0, chunks = nblk * 2;   // of 32 columns
    const int64_t col0 = (int64_t)blk0 * 64;

    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    cluster_sync_all();   // every CTA runs before its shared memory is written from outside
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t mma_phase = 0;
    // All threads: the MMAs that thread 0 committed are done.  A wait that runs out
    // sets the error word and goes on (every CTA has to reach the cluster barriers).
    auto mma_wait = [&] {
        if (!mbar_wait(bar, mma_phase, kOrthWaitCycles)) atomicExch(&g_orth_error, 1);
        mma_phase ^= 1u;
        tc_fence_after();
    };

    // ---------------- x into tensor memory as it is, and its sum of squares
    const T* x = static_cast<const T*>(p.x) + batch * p.stride;
    float sq[4] = {0.f, 0.f, 0.f, 0.f};
    const bool direct = p.transposed || p.vec;
    if (direct) {
        for (int c = half; rows_here && c < chunks; c += 2) {
            float v[32];
            const int64_t j0 = col0 + 32 * c;
            if (p.transposed) {   // 32 lanes, 32 neighbours of a row of x
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = row < p.m && j0 + j < p.n ? orth_f32(x[(j0 + j) * p.ld + row]) : 0.f;
            } else {
                constexpr int V = 16 / sizeof(T);
#pragma unroll
                for (int h = 0; h < 32 / V; ++h) {
                    float f[V];
                    const bool in = row < p.m && j0 + V * h < p.n;   // a row holds whole vectors
                    if (in) orth_vec<T>(x + row * p.ld + j0 + V * h, f);
#pragma unroll
                    for (int k = 0; k < V; ++k) v[V * h + k] = in ? f[k] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) sq[j & 3] += v[j] * v[j];
            __syncwarp();
            tmem_st32(lanes + 32 * c, v);
        }
    } else {
        // rows at any alignment: 64 columns at a time through shared memory, so
        // that the lanes read neighbours
        float f[32];
        auto fetch = [&](int b) {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const int i = (k >> 1) * 8 + warp;
                const int64_t j = col0 + 64 * b + (k & 1) * 32 + lane;
                f[k] = i < p.m && j < p.n ? orth_f32(x[i * p.ld + j]) : 0.f;
            }
        };
        fetch(0);
        for (int b = 0; b < nblk; ++b) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 32; ++k)
                sts_f32(sp + (((k >> 1) * 8 + warp) * 65 + (k & 1) * 32 + lane) * 4, f[k]);
            __syncthreads();
            if (b + 1 < nblk) fetch(b + 1);
            if (rows_here) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    v[j] = lds_f32(sp + (row * 65 + 32 * half + j) * 4);
                    sq[j & 3] += v[j] * v[j];
                }
                __syncwarp();
                tmem_st32(lanes + 64 * b + 32 * half, v);
            }
        }
    }
    tmem_st_wait();
    // Sum (or largest) of t over the cluster, the same in every thread; by way of `to`,
    // a float for every CTA that no other call uses.
    auto over_cluster = [&](float t, uint32_t to, auto join) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) t = join(t, __shfl_xor_sync(0xffffffffu, t, o));
        if (lane == 0) sts_f32(red + 4 * warp, t);
        __syncthreads();
        if (threadIdx.x < ctas) {   // this CTA's into every CTA
            t = 0.f;
            for (int w = 0; w < kOrthCluThreads / 32; ++w) t = join(t, lds_f32(red + 4 * w));
            dsm_st(map_to_rank(to + 4 * rank, threadIdx.x), t);
        }
        __syncwarp();
        cluster_sync_all();
        t = 0.f;
        for (uint32_t k = 0; k < ctas; ++k) t = join(t, lds_f32(to + 4 * k));
        return t;
    };
    auto add = [](float a, float b) { return a + b; };
    OrthSum total{over_cluster((sq[0] + sq[1]) + (sq[2] + sq[3]), sums, add), 0};
    if (!orth_sum_plain(total.s)) {   // alike in the whole cluster: as in the partial sums
        auto each = [&](auto take) {
            for (int c = half; rows_here && c < chunks; c += 2) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(lanes + 32 * c, r);
#pragma unroll
                for (int j = 0; j < 32; ++j) take(j, __uint_as_float(r[j]));
            }
        };
        float top = 0.f;
        each([&](int, float v) { top = fmaxf(top, fabsf(v)); });
        top = over_cluster(top, sums_top, [](float a, float b) { return fmaxf(a, b); });
        if (top > 0.f && isfinite(top)) {
            total.e = ilogbf(top);
            const float2 by = orth_scale_of(total.e);
            float again[4] = {0.f, 0.f, 0.f, 0.f};   // in the first sum's order
            each([&](int j, float v) {
                v = v * by.x * by.y;
                again[j & 3] += v * v;
            });
            total.s = over_cluster((again[0] + again[1]) + (again[2] + again[3]), sums_again, add);
        }
    }
    // tensor memory holds kOrthScale^2 X
    float2 mult = orth_inverse(total, p.eps, kOrthScale * kOrthScale);

    constexpr float kInv = 1.f / kOrthScale;
    for (int step = 0;; ++step) {
        // ---------------- X (times mult, the first time) to its FP16 rounding
        if (rows_here) {
            for (int c = half; c < chunks; c += 2) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(lanes + 32 * c, r);
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * mult.x * mult.y;
                if (step == 0) tmem_st32(lanes + 32 * c, v);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sts_v4(orth_block_piece(sx + (c >> 1) * kOrthBlockBytes, row, (c & 1) * 4 + q),
                           orth_pack(v[8 * q] * kInv, v[8 * q + 1] * kInv),
                           orth_pack(v[8 * q + 2] * kInv, v[8 * q + 3] * kInv),
                           orth_pack(v[8 * q + 4] * kInv, v[8 * q + 5] * kInv),
                           orth_pack(v[8 * q + 6] * kInv, v[8 * q + 7] * kInv));
            }
            if (step == 0) tmem_st_wait();
        }
        mult = {1.f, 1.f};
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        // ---------------- Gram
        if (threadIdx.x == 0) {
            const uint32_t idesc = orth_idesc_n(p.mp, false);
            for (int b = 0; b < nblk; ++b) {
                const uint64_t desc = orth_desc_k(sx + b * kOrthBlockBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_bf16(tmem + kOrthGramCol, desc + 2 * k, desc + 2 * k, idesc, (b | k) != 0 ? 1u : 0u);
            }
            umma_commit(bar);
        }
        mma_wait();
        const int width = p.mp / 2, from = half * width;   // this thread's columns of the m x m matrices
        if (ctas == 1) {
            if (rows_here) {
                for (int c = from; c < from + width; c += 32) {
                    uint32_t r[32];
                    __syncwarp();
                    tmem_ld32(lanes + kOrthGramCol + c, r);
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float a = __uint_as_float(r[j]) * kInv;
                        if (c + j == row) {
                            sts_f32(sd + 4 * row, a * kInv);
                            a = 0.f;
                        }
                        r[j] = __float_as_uint(a);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = orth_pack(__uint_as_float(r[8 * q + 2 * k]), __uint_as_float(r[8 * q + 2 * k + 1]));
                        sts_v4(orth_block_piece(sa + (c >> 6) * kOrthBlockBytes, row, ((c >> 3) & 7) + q), w[0], w[1],
                               w[2], w[3]);
                    }
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
        } else {
            if (rows_here) {
                for (int c = from; c < from + width; c += 32) {
                    uint32_t r[32];
                    __syncwarp();
                    tmem_ld32(lanes + kOrthGramCol + c, r);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        sts_v4(orth_part_piece(sp, row, (c >> 2) + q), r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            cluster_sync_all();
            tc_fence_after();
            // rows [rank share, ...) summed over the CTAs, to all of them
            const int share = p.mp / (int)ctas, per_row = p.mp / 4;
            for (int e = threadIdx.x; e < share * per_row; e += kOrthCluThreads) {
                const int i = (int)rank * share + e / per_row, j = e % per_row * 4;
                const uint32_t at = orth_part_piece(sp, i, j >> 2);
                float4 part[kOrthCluMaxCtas];
#pragma unroll
                for (int k = 0; k < kOrthCluMaxCtas; ++k)
                    if (k < (int)ctas) part[k] = dsm_ld(map_to_rank(at, k));
                float4 t = part[0];
#pragma unroll
                for (int k = 1; k < kOrthCluMaxCtas; ++k)
                    if (k < (int)ctas) {
                        t.x += part[k].x;
                        t.y += part[k].y;
                        t.z += part[k].z;
                        t.w += part[k].w;
                    }
                float v[4] = {t.x * kInv, t.y * kInv, t.z * kInv, t.w * kInv};
                float di = 0.f;
                const bool diag = i >= j && i < j + 4;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k == i) {
                        di = v[k] * kInv;
                        v[k] = 0.f;
                    }
                const uint32_t lo = orth_pack(v[0], v[1]), hi = orth_pack(v[2], v[3]);
                const uint32_t to =
                    orth_block_piece(sa + (j >> 6) * kOrthBlockBytes, i, (j >> 3) & 7) + (uint32_t)(j & 4) * 2;
                for (uint32_t k = 0; k < ctas; ++k) {
                    dsm_st2(map_to_rank(to, k), lo, hi);
                    if (diag) dsm_st(map_to_rank(sd + 4 * i, k), di);
                }
            }
            fence_proxy_async_all();
            __syncwarp();
            cluster_sync_all();
            fence_proxy_async_all();
        }
        // ---------------- Poly
        if (threadIdx.x == 0) {
            const uint32_t idesc = orth_idesc_n(p.mp, false);
            for (int k = 0; k < p.mp / 16; ++k) {
                const uint64_t desc = orth_desc_k(sa + (k >> 2) * kOrthBlockBytes) + 2 * (k & 3);
                umma_bf16(tmem + kOrthGramCol, desc, desc, idesc, k != 0 ? 1u : 0u);
            }
            umma_commit(bar);
        }
        mma_wait();
        const float ka = p.coef[3 * step], kb = p.coef[3 * step + 1], kc = p.coef[3 * step + 2];
        if (rows_here) {
            const float di = lds_f32(sd + 4 * row), k0 = kb + kc * di;
            float sq_ii = 0.f;
            for (int c = from; c < from + width; c += 32) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(lanes + kOrthGramCol + c, r);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t at = orth_block_piece(sa + (c >> 6) * kOrthBlockBytes, row, ((c >> 3) & 7) + q);
                    const uint4 a0 = lds_v4(at);
                    const uint32_t ws[4] = {a0.x, a0.y, a0.z, a0.w};
                    uint32_t w[4];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint4 dq = lds_v4(sd + 4 * (c + 8 * q + 4 * g));
                        const uint32_t ds[4] = {dq.x, dq.y, dq.z, dq.w};
                        float v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = 8 * q + 4 * g + k;
                            const uint32_t wk = ws[2 * g + (k >> 1)];
                            const float a = (k & 1) ? h_hi(wk) : h_lo(wk);
                            const float sqr = __uint_as_float(r[j]) * kInv;   // scaled A0^2
                            v[k] = (k0 + kc * __uint_as_float(ds[k])) * a + kc * sqr;
                            if (c + j == row) {
                                sq_ii = sqr * kInv;
                                v[k] = 0.f;
                            }
                        }
                        w[2 * g] = orth_pack(v[0], v[1]);
                        w[2 * g + 1] = orth_pack(v[2], v[3]);
                    }
                    sts_v4(at, w[0], w[1], w[2], w[3]);
                }
            }
            if (row >= from && row < from + width) sts_f32(se + 4 * row, kb * di + kc * (di * di) + kc * sq_ii);
        }
        __syncthreads();   // e
        // ---------------- Apply
        const bool with_lo = p.stray[step] < 1.f;
        if (rows_here) {
            const float ai = ka + lds_f32(se + 4 * row);
            for (int c = half; c < chunks; c += 2) {
                uint32_t r[32];
                float v[32];
                __syncwarp();
                tmem_ld32(lanes + 32 * c, r);
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * ai;
                tmem_st32(lanes + 32 * c, v);
                if (with_lo) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float x0 = __uint_as_float(r[8 * q + 2 * k]) * kInv,
                                        x1 = __uint_as_float(r[8 * q + 2 * k + 1]) * kInv;
                            const uint32_t h = orth_pack(x0, x1);
                            w[k] = orth_pack(x0 - h_lo(h), x1 - h_hi(h));
                        }
                        sts_v4(orth_block_piece(sp + (c >> 1) * kOrthBlockBytes, row, (c & 1) * 4 + q), w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tmem_st_wait();
        }
        fence_proxy_async_smem();   // B0, X_lo
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (threadIdx.x == 0) {
            for (int b = 0; b < nblk; b += 4) {
                const int cols = nblk - b < 4 ? (nblk - b) * 64 : 256;
                const uint32_t idesc = orth_idesc_n(cols, true);
                for (uint32_t x = sx;; x = sp) {   // X_hi, then X_lo
                    for (int k = 0; k < p.mp / 16; ++k)
                        umma_bf16(tmem + b * 64, orth_desc_k(sa + (k >> 2) * kOrthBlockBytes) + 2 * (k & 3),
                                  orth_desc_mn_block(x + b * kOrthBlockBytes) + (2048 >> 4) * k, idesc, 1u);
                    if (!with_lo || x == sp) break;
                }
            }
            umma_commit(bar);
        }
        mma_wait();
        if (step + 1 == p.steps) break;
    }

    // ---------------- the result
    const float fin = p.scale * kInv * kInv;
    const int64_t obase = batch * p.stride_out;
    for (int b = 0; b < nblk; ++b) {
        const int64_t j0 = col0 + 64 * b + 32 * half;
        float v[32];
        if (rows_here) {
            uint32_t r[32];
            __syncwarp();
            tmem_ld32(lanes + 64 * b + 32 * half, r);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * fin;
        }
        if (p.transposed) {
            if (rows_here && row < p.m) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j0 + j < p.n) {
                        const int64_t at = obase + (j0 + j) * p.ld_out + row;
                        if (p.out_dtype == 2) static_cast<float*>(p.out)[at] = v[j];
                        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v[j]);
                    }
            }
        } else if (p.vec_out && p.out_dtype != 2 && col0 + 64 * b + 64 <= p.n) {
            if (rows_here && row < p.m) {
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + obase + row * p.ld_out + j0);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                      pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
            }
        } else {
            __syncthreads();   // the last block's readers
            if (rows_here)
#pragma unroll
                for (int j = 0; j < 32; ++j) sts_f32(sp + (row * 65 + 32 * half + j) * 4, v[j]);
            __syncthreads();
            for (int i = warp; i < p.m; i += kOrthCluThreads / 32) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t j = col0 + 64 * b + 32 * h + lane;
                    if (j < p.n) {
                        const float f = lds_f32(sp + (i * 65 + 32 * h + lane) * 4);
                        if (p.out_dtype == 2) static_cast<float*>(p.out)[obase + i * p.ld_out + j] = f;
                        else static_cast<__nv_bfloat16*>(p.out)[obase + i * p.ld_out + j] = __float2bfloat16_rn(f);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace flp
