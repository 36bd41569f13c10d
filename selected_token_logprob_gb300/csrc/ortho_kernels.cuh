// Newton-Schulz orthogonalisation of a weight's update on the tcgen05 tensor
// cores.  With X the matrix (transposed if it is taller than wide: m <= n) over
// its Frobenius norm, each step is
//   A = X X^T,  B = b A + c A^2,  X <- a X + B X,
// which sends every singular value s to a s + b s^3 + c s^5.
//
// Numerics.  The products run on FP16 operands (scaled by kOrthScale = 2^8, so
// that entries as small as 2^-22 keep all 11 bits) with FP32 accumulators; what
// FP16's rounding would spoil is kept out of it:
//   - X is carried as hi + lo FP16 (22 bits).  The products read hi; the term
//     a X, by which small singular values grow ~485-fold in five steps, is
//     taken from both.
//   - The diagonals of A and B, alike over the rows, would round all the same
//     way.  They are FP32 vectors d and e, and the FP16 matrices A0, B0 hold the
//     rest: with A = D + A0,
//       B_ij = (b + c (d_i + d_j)) A0_ij + c (A0^2)_ij   (i != j)
//       e_i  = b d_i + c d_i^2 + c (A0^2)_ii
//       X'   = (a + e_i) X_i. + B0 X.
// Against 64 bits the result is off by 3e-4 to 1e-3 of its norm (plain FP16: up
// to 5e-2 where the spectrum has a low rank over a floor; BF16: 0.2).
//
// A and B are symmetric: only tiles on and above the diagonal are computed, and
// each is written to both places.
//
// Each product is one launch of persistent CTAs with six warps: one TMA
// producer, one MMA issuer, four epilogue warps (one accumulator row a thread).
// Every wait is bounded: a wait that runs out sets the error word and the CTA's
// abort flag, the copies and MMAs in flight are waited for, TMEM is freed and
// the kernel returns.
#pragma once

#include <cuda_fp16.h>

#include "tc_prims.cuh"

namespace flp {

constexpr float kOrthScale = 256.f;          // of every FP16 operand
constexpr float kOrthLoScale = 2048.f;       // of lo, on top: hi's rounding is below 2^-11
constexpr long long kOrthWaitCycles = 4000000000LL;
constexpr int kOrthThreads = 192;
constexpr int kOrthBM = 128;
constexpr int kOrthBK = 64;
constexpr int kOrthParts = 128;              // partial sums of squares per matrix

static __device__ int g_orth_error;          // 1 = a bounded wait ran out

enum OrthMode { kOrthGram = 0, kOrthPoly = 1, kOrthApply = 2, kOrthFinal = 3 };

struct OrthArgs {
    int64_t batch, m, n;      // m <= n, of X
    int64_t mp, np;           // padded to multiples of 64
    int tiles_m, tiles_n;     // of the output: rows of 128, columns of the kernel's N
    int64_t units;            // output tiles over the batch
    int nkb;                  // K blocks of 64
    float a, b, c;            // this step's coefficients
    __half *mat;              // Gram: A0 out; Poly: A0 in
    __half *mat_out;          // Poly: B0 out
    float *d, *e;             // [batch mp] diagonals
    const __half *x_hi;       // Apply, Final: X
    __half *x_lo;             // Apply: in place; Final: read
    __half *x_out;            // Apply: the next X's hi
    void* out;                // Final
    int out_dtype, transposed, vec_out;
    int64_t ld_out, stride_out;
    float scale;              // Final: of the result
};

__device__ __forceinline__ void orth_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// K-major and MN-major operands with 128-byte swizzle (as the tensor-map boxes
// of 64 elements lay them out); see the descriptors' fields in the PTX ISA.
__device__ __forceinline__ uint64_t orth_desc_k(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t orth_desc_mn(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16 with FP16 operands (type fields 0), FP32 accumulators; bit 16: B MN-major.
template <int kBN, bool kBmn>
__host__ __device__ constexpr uint32_t orth_idesc() {
    return (1u << 4) | ((kBmn ? 1u : 0u) << 16) | ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kOrthBM >> 4) << 24);
}

__device__ __forceinline__ bool orth_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > kOrthWaitCycles) {
                *abort_flag = 1;
                atomicExch(&g_orth_error, 1);
                return false;
            }
        }
    }
}

struct OrthUnit {
    int64_t batch;
    int mb, nb;
};
// Output tile u: row by row; of a symmetric product only tiles with nb >= mb.
template <bool kSym>
__device__ __forceinline__ OrthUnit orth_unit(int64_t u, const OrthArgs& p) {
    OrthUnit w;
    const int64_t per = kSym ? (int64_t)p.tiles_m * (p.tiles_m + 1) / 2 : (int64_t)p.tiles_m * p.tiles_n;
    w.batch = u / per;
    int64_t t = u - w.batch * per;
    if (kSym) {
        int mb = 0;
        while (t >= p.tiles_m - mb) {
            t -= p.tiles_m - mb;
            ++mb;
        }
        w.mb = mb;
        w.nb = mb + (int)t;
    } else {
        w.mb = (int)(t / p.tiles_n);
        w.nb = (int)(t - (int64_t)w.mb * p.tiles_n);
    }
    return w;
}

template <int kBN>
constexpr uint32_t kOrthStageBytes = (kOrthBM + kBN) * kOrthBK * 2;
template <int kBN>
constexpr int kOrthStages = 196608 / (int)kOrthStageBytes<kBN>;
template <int kBN>
constexpr size_t kOrthSmemBytes = 1024 + (size_t)kOrthStages<kBN> * kOrthStageBytes<kBN> + 256;

__device__ __forceinline__ uint32_t orth_pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The 32 accumulators of row i, columns c0 .. c0 + 31 (all inside the padded
// output) of one matrix of the batch.
template <int kMode>
__device__ __forceinline__ void orth_epilogue(const OrthArgs& p, int64_t batch, bool mirror, int64_t i, int64_t c0,
                                              uint32_t (&r)[32]) {
    constexpr float kInv = 1.f / kOrthScale;
    const int64_t row = batch * p.mp + i;
    if constexpr (kMode == kOrthGram || kMode == kOrthPoly) {
        float v[32];
        if constexpr (kMode == kOrthGram) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                v[j] = __uint_as_float(r[j]) * kInv;   // scaled A
                if (c0 + j == i) {
                    p.d[row] = v[j] * kInv;
                    v[j] = 0.f;
                }
            }
        } else {
            const uint4* src = reinterpret_cast<const uint4*>(p.mat + row * p.mp + c0);
            const float di = p.d[row];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 w = src[q];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int j = 8 * q + k;
                    const float a0 = (k & 1) ? h_hi(ws[k >> 1]) : h_lo(ws[k >> 1]);
                    const float dj = p.d[batch * p.mp + c0 + j];
                    const float sq = __uint_as_float(r[j]) * kInv;   // scaled A0^2
                    v[j] = (p.b + p.c * (di + dj)) * a0 + p.c * sq;
                    if (c0 + j == i) {
                        p.e[row] = p.b * di + p.c * (di * di) + p.c * (sq * kInv);
                        v[j] = 0.f;
                    }
                }
            }
        }
        __half* dst = kMode == kOrthGram ? p.mat : p.mat_out;
        uint4* o = reinterpret_cast<uint4*>(dst + row * p.mp + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = make_uint4(orth_pack(v[8 * q], v[8 * q + 1]), orth_pack(v[8 * q + 2], v[8 * q + 3]),
                              orth_pack(v[8 * q + 4], v[8 * q + 5]), orth_pack(v[8 * q + 6], v[8 * q + 7]));
        if (mirror) {
#pragma unroll
            for (int j = 0; j < 32; ++j) dst[(batch * p.mp + c0 + j) * p.mp + i] = __float2half_rn(v[j]);
        }
    } else {
        const float ai = p.a + p.e[row];
        const uint4* hi = reinterpret_cast<const uint4*>(p.x_hi + row * p.np + c0);
        uint4* lo = reinterpret_cast<uint4*>(p.x_lo + row * p.np + c0);
        float v[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 h = hi[q], l = lo[q];
            const uint32_t hs[4] = {h.x, h.y, h.z, h.w}, ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float xh = (k & 1) ? h_hi(hs[k >> 1]) : h_lo(hs[k >> 1]);
                const float xl = (k & 1) ? h_hi(ls[k >> 1]) : h_lo(ls[k >> 1]);
                v[8 * q + k] = ai * (xh + xl * (1.f / kOrthLoScale)) + __uint_as_float(r[8 * q + k]) * kInv;
            }
        }
        if constexpr (kMode == kOrthApply) {
            uint4* o = reinterpret_cast<uint4*>(p.x_out + row * p.np + c0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x0 = v[8 * q + 2 * k], x1 = v[8 * q + 2 * k + 1];
                    hw[k] = orth_pack(x0, x1);
                    lw[k] = orth_pack((x0 - h_lo(hw[k])) * kOrthLoScale, (x1 - h_hi(hw[k])) * kOrthLoScale);
                }
                o[q] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                lo[q] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
            }
        } else {
            if (i >= p.m) return;
            const float s = p.scale * kInv;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= s;
            const int64_t base = batch * p.stride_out;
            if (p.vec_out && !p.transposed && c0 + 32 <= p.n) {
                if (p.out_dtype == 2) {
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + base + i * p.ld_out + c0);
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                } else {
                    uint4* o =
                        reinterpret_cast<uint4*>(static_cast<unsigned short*>(p.out) + base + i * p.ld_out + c0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(v[8 * q + 2 * k], v[8 * q + 2 * k + 1]);
                        o[q] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c0 + j < p.n) {
                        const int64_t at = base + (p.transposed ? (c0 + j) * p.ld_out + i : i * p.ld_out + c0 + j);
                        if (p.out_dtype == 2) static_cast<float*>(p.out)[at] = v[j];
                        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v[j]);
                    }
                }
            }
        }
    }
}

template <int kMode, int kBN>
__global__ void __launch_bounds__(kOrthThreads, 1)
k_orth_product(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, OrthArgs p) {
    constexpr bool kSym = kMode == kOrthGram || kMode == kOrthPoly;
    constexpr int kStages = kOrthStages<kBN>;
    constexpr uint32_t kStageBytes = kOrthStageBytes<kBN>, kABytes = kOrthBM * kOrthBK * 2;
    extern __shared__ __align__(1024) unsigned char orth_smem_raw[];
    const uint32_t raw = smem_u32(orth_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + kStages * kStageBytes;
    const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
    const uint32_t tfull0 = bars + 16 * kStages, tempty0 = tfull0 + 16;
    const uint32_t drain = tempty0 + 16;
    const uint32_t slot = drain + 8;
    unsigned char* slot_gen = orth_smem_raw + (slot - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(slot_gen);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_gen + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, 128);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
    }
    if (warp == 1) {
        tmem_alloc(slot, 2 * kBN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    orth_dep_wait();   // the operands are the previous launch's output

    if (warp == 0) {
        // ---------------- TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                const OrthUnit w = orth_unit<kSym>(u, p);
                const int row0 = (int)(w.batch * p.mp);
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!orth_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + stage * kStageBytes, bar = full0 + 8 * stage;
                    mbar_arrive_expect_tx(bar, kStageBytes);
                    tma_load_2d(dst, &tm_a, kb * kOrthBK, row0 + w.mb * kOrthBM, bar);
                    if constexpr (kSym) {
                        tma_load_2d(dst + kABytes, &tm_b, kb * kOrthBK, row0 + w.nb * kBN, bar);
                    } else {
#pragma unroll
                        for (int j = 0; j < kBN / 64; ++j)
                            tma_load_2d(dst + kABytes + j * 8192, &tm_b, w.nb * kBN + 64 * j, row0 + kb * kOrthBK,
                                        bar);
                    }
                    issued |= 1u << stage;
                    last_par = (last_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                for (int s = 0; s < kStages; ++s)
                    if (issued & (1u << s)) mbar_wait(full0 + 8 * s, (last_par >> s) & 1u, kOrthWaitCycles);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = orth_idesc<kBN, !kSym>();
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; ok && u < p.units; u += gridDim.x) {
                if (!orth_wait(tempty0 + 8 * acc, acc_phase ^ 1u, abort_flag)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem + (uint32_t)(acc * kBN);
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!orth_wait(full0 + 8 * stage, phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t addr = base + stage * kStageBytes;
                    const uint64_t a_desc = orth_desc_k(addr);
                    const uint64_t b_desc = kSym ? orth_desc_k(addr + kABytes) : orth_desc_mn(addr + kABytes);
                    constexpr uint64_t kBStep = kSym ? (32 >> 4) : (2048 >> 4);
#pragma unroll
                    for (int k = 0; k < kOrthBK / 16; ++k)
                        umma_bf16(d_tmem, a_desc + (32 >> 4) * k, b_desc + kBStep * k, idesc,
                                  (kb != 0 || k != 0) ? 1u : 0u);
                    umma_commit(empty0 + 8 * stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit(tfull0 + 8 * acc);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            umma_commit(drain);
            mbar_wait(drain, 0, kOrthWaitCycles);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: one output row per thread
        const int q = warp & 3;
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
        const int64_t cols = kSym ? p.mp : p.np;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
            const OrthUnit w = orth_unit<kSym>(u, p);
            if (!orth_wait(tfull0 + 8 * acc, acc_phase, abort_flag)) break;
            tc_fence_after();
            const int64_t i = (int64_t)w.mb * kOrthBM + q * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < kBN / 32; ++c) {
                const int64_t c0 = (int64_t)w.nb * kBN + c * 32;
                if (c0 >= cols) break;   // uniform over the CTA
                __syncwarp();
                uint32_t r[32];
                tmem_ld32(lane_addr + (uint32_t)(acc * kBN + c * 32), r);
                if (i < p.mp) orth_epilogue<kMode>(p, w.batch, kSym && w.mb != w.nb, i, c0, r);
            }
            tc_fence_before();
            mbar_arrive(tempty0 + 8 * acc);
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kBN);
    }
}

// ---------------------------------------------------------------- the input

struct OrthInput {
    const void* x;            // [rows, ld] of `dtype`, matrices `stride` elements apart
    int64_t rows, cols, ld, stride, batch;
    int transposed;           // X = x^T
    float eps;
    double* parts;            // [batch, kOrthParts]
    __half *hi, *lo;          // [batch mp, np]
    int64_t mp, np;
};

__device__ __forceinline__ float orth_f32(float v) { return v; }
__device__ __forceinline__ float orth_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float orth_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Partial sums of squares: part q of a matrix takes its rows q, q + kOrthParts, ...
template <class T>
__global__ void __launch_bounds__(256)
k_orth_sumsq(OrthInput p) {
    __shared__ double red[8];
    const int64_t b = blockIdx.x / kOrthParts;
    const int q = (int)(blockIdx.x % kOrthParts);
    const T* x = static_cast<const T*>(p.x) + b * p.stride;
    double s = 0.0;
    for (int64_t r = q; r < p.rows; r += kOrthParts) {
        float f = 0.f;
        for (int64_t c = threadIdx.x; c < p.cols; c += 256) {
            const float v = orth_f32(x[r * p.ld + c]);
            f += v * v;
        }
        s += (double)f;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int k = 0; k < 8; ++k) t += red[k];
        p.parts[b * kOrthParts + q] = t;
    }
}

// X (hi, lo) = x / (|x| + eps), zero in the padding; 32 x 32 tiles, turned
// through shared memory when X is x's transpose.
template <class T>
__global__ void __launch_bounds__(256)
k_orth_load(OrthInput p) {
    __shared__ float tile[32][33];
    __shared__ float s_inv;
    const int64_t tn = p.np / 32, tm = p.mp / 32;
    const int64_t b = blockIdx.x / (tn * tm);
    const int64_t t = blockIdx.x - b * tn * tm;
    const int64_t i0 = t / tn * 32, j0 = t % tn * 32;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    if (ty == 0) {
        double s = 0.0;
        for (int k = tx; k < kOrthParts; k += 32) s += p.parts[b * kOrthParts + k];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // an infinite sum of squares (FP32 overflow) makes X NaN, not 0
        if (tx == 0)
            s_inv = isfinite(s) ? (float)((double)kOrthScale / (sqrt(s) + (double)p.eps)) : __int_as_float(0x7fc00000);
    }
    const T* x = static_cast<const T*>(p.x) + b * p.stride;
    // tile[a][c] = x at row (transposed ? j0 : i0) + a, column (transposed ? i0 : j0) + c
    const int64_t r0 = p.transposed ? j0 : i0, c0 = p.transposed ? i0 : j0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = r0 + ty + 8 * k, c = c0 + tx;
        tile[ty + 8 * k][tx] = r < p.rows && c < p.cols ? orth_f32(x[r * p.ld + c]) : 0.f;
    }
    __syncthreads();
    const float inv = s_inv;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int a = ty + 8 * k;
        const float v = (p.transposed ? tile[tx][a] : tile[a][tx]) * inv;
        const __half h = __float2half_rn(v);
        const int64_t at = (b * p.mp + i0 + a) * p.np + j0 + tx;
        p.hi[at] = h;
        p.lo[at] = __float2half_rn((v - __half2float(h)) * kOrthLoScale);
    }
}

}  // namespace flp
