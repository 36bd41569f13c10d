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
//       X'   = (a + e_i) hi_i. + (a + f_i) lo_i. + B0 hi.
//   - f_i is e_i or 0.  With e_i the row of B X takes lo as far as B is diagonal, which
//     is nearly all of it once the singular values are alike.  But B0 lo is missing: in
//     the directions that X does not have it would cancel diag(e) lo, which alone is noise
//     there, and the steps to come multiply it by their a.  Its part outside of the row's
//     own direction is sqrt(1 - rho_i), rho_i = d_i^2 / (A^2)_ii (r / m for a projection
//     of rank r of m, 1 for a row orthogonal to all others), with (A^2)_ii = d_i^2 +
//     (A0^2)_ii.  So f_i = e_i where (1 - rho_i) G <= 35, G the product of a^2 over the
//     steps to come: always in the last two usual steps, at rho >= 0.75 in the third
//     last, 0.98 before that.
// Against 64 bits the result of five usual steps is off by 3e-4 to 2e-3 of its norm on
// spectra from alike to rank 1, with any floor, by 4e-3 at most (few rows, or a row that
// holds most of a low rank; 1e-2 where a side is below 8); f = e throughout: 1e-2 at a rank of m / 2,
// 4e-2 at rank 1; plain FP16: 5e-2 and more; BF16: 0.2.  What is left are the roundings
// of hi, A0 and B0 to 11 bits: a choice of one FP16 product where operands of hi and lo
// would take three.
//
// A and B are symmetric: only tiles on and above the diagonal are computed, and
// each is written to both places.
//
// Each product is one launch: persistent CTAs or CTA pairs (k_orth_product), or,
// where a product has fewer 128 x 128 tiles than the GPU has SMs, a cluster a tile
// (k_orth_split); a matrix with a side of at most 128 takes one launch in all
// (ortho_cluster.cuh).  The persistent form has ten warps: one TMA producer, one MMA
// issuer, eight epilogue warps (one accumulator row a thread, half of a tile's
// columns).  The epilogue of a tile overlaps the next tile's MMAs; what it reads
// beside the accumulators (X's hi and lo, or A0) comes by TMA into boxes of 32 rows
// x 32 columns a warp, which it rewrites in place and stores by TMA (by way of
// registers and plain loads and stores: 78 instead of 65 us for Apply at 8 x 1024 x
// 4096).  Every wait is bounded: a wait that runs out sets the error word and the
// CTA's abort flag, the copies and MMAs in flight are waited for, TMEM is freed and
// the kernel returns.
//
// What bounds it (4096 x 4096, 1.08 ms at 1860 MHz, the power cap's): the tensor cores and
// the copies that feed them, 585 cycles a K block of a 256 x 256 tile (512 being the MMAs'
// own), in 2, 2 and 4 waves a step where 1.8, 1.8 and 3.4 would hold the work: 805 us; the
// input passes 38; start, first copies and last epilogue of 15 launches the rest.  Cutting the K
// blocks of all tiles into equal runs, one a pair, did not pay: the same 1046 us,
// and 644 instead of 617 at 4 x 2048 x 2048.
#pragma once

#include <cuda_fp16.h>
#include <limits.h>

#include "tc_prims.cuh"

namespace flp {

constexpr float kOrthScale = 256.f;          // of every FP16 operand
constexpr float kOrthLoScale = 2048.f;       // of lo, on top: hi's rounding is below 2^-11
constexpr long long kOrthWaitCycles = 4000000000LL;
constexpr int kOrthThreads = 192;
// The persistent kernel's epilogue: two warps per 32 rows, each with half of a tile's
// columns (with one, a chunk of 32 columns took 1350 cycles, the latencies of its own
// instructions, and 8 x 1024 x 4096's products waited for it).
constexpr int kOrthEpiWarps = 8, kOrthProductThreads = 64 + 32 * kOrthEpiWarps;
constexpr int kOrthBK = 64;
constexpr int kOrthParts = 256;              // most partial sums of squares per matrix

static __device__ int g_orth_error;          // 1 = a bounded wait ran out

enum OrthMode { kOrthGram = 0, kOrthPoly = 1, kOrthApply = 2, kOrthFinal = 3 };

struct OrthArgs {
    int64_t m, n;             // m <= n, of X
    int64_t mp, np;           // padded to multiples of 64
    int tiles_m, tiles_n;     // of the output: rows of 128 (a pair: 256), columns of the kernel's N
    int64_t per;              // output tiles of one matrix
    int64_t units;            // over the batch
    int nkb;                  // K blocks of 64
    float a, b, c;            // this step's coefficients
    float stray;              // f_i = e_i where (A0^2)_ii <= stray (A^2)_ii
    __half* mat_out;          // Gram: A0, Poly: B0
    const __half* mat_in;     // A0
    const __half* x_hi;       // X; its next hi, and lo (in place)
    __half *x_out, *x_lo;
    float *d, *e, *f;         // [batch mp]: the diagonals, and of e what lo takes
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
template <int kBM, int kBN, bool kBmn>
__host__ __device__ constexpr uint32_t orth_idesc() {
    return (1u << 4) | ((kBmn ? 1u : 0u) << 16) | ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
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

template <bool kPair>
__device__ __forceinline__ bool orth_wait_acc(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if constexpr (!kPair) return orth_wait(bar, parity, abort_flag);
    if (mbar_try_cluster(bar, parity)) return true;   // the peer's warps arrive on it too
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_cluster(bar, parity)) return true;
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
// Output tile u: row by row; of a symmetric product only tiles that reach the
// diagonal or lie right of it.
template <bool kSym, int kBM, int kBN>
__device__ __forceinline__ OrthUnit orth_unit(int64_t u, const OrthArgs& p) {
    OrthUnit w;
    w.batch = u / p.per;
    int64_t t = u - w.batch * p.per;
    if (kSym) {
        int mb = 0, first = 0;
        while (t >= p.tiles_n - first) {
            t -= p.tiles_n - first;
            ++mb;
            first = mb * kBM / kBN;
        }
        w.mb = mb;
        w.nb = first + (int)t;
    } else {
        w.mb = (int)(t / p.tiles_n);
        w.nb = (int)(t - (int64_t)w.mb * p.tiles_n);
    }
    return w;
}

// Shared memory of a CTA: the stages (128 rows of A and its rows or columns of
// B per K block), a block of barriers, and two boxes of 32 x 32 per epilogue warp and
// matrix.  A TMA copy takes 2000 (idle) to 3100 (loaded) cycles to arrive, so nearly
// all of shared memory goes to the stages (a 256 x 256 pair tile: 6 for Gram and Poly,
// 5 for Apply): with 4 a K block took 776 cycles, 512 being the MMAs' own.
constexpr uint32_t kOrthABytes = 128 * kOrthBK * 2;
template <int kBN, bool kPair>
constexpr uint32_t kOrthBBytes = (kPair ? kBN / 2 : kBN) * kOrthBK * 2;
template <int kBN, bool kPair>
constexpr uint32_t kOrthStageBytes = kOrthABytes + kOrthBBytes<kBN, kPair>;
// 32 rows x 32 columns of one matrix (Gram, Poly), or of hi and of lo
constexpr uint32_t kOrthSquareBytes = 32 * 32 * 2;
template <bool kSym>
constexpr uint32_t kOrthBoxBytes = kSym ? kOrthSquareBytes : 2 * kOrthSquareBytes;
constexpr int kOrthBoxes = 2;              // a warp
template <int kBN, bool kPair, bool kSym>
constexpr int kOrthStages =
    (229376 - kOrthEpiWarps * kOrthBoxes * (int)kOrthBoxBytes<kSym>) / (int)kOrthStageBytes<kBN, kPair>;
template <int kBN, bool kPair, bool kSym>
constexpr size_t kOrthSmemBytes = 1024 + (size_t)kOrthStages<kBN, kPair, kSym> * kOrthStageBytes<kBN, kPair> + 1024 +
                                  kOrthEpiWarps * kOrthBoxes * (size_t)kOrthBoxBytes<kSym>;

__device__ __forceinline__ uint32_t orth_pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 16-byte piece j of row r of a box with 128-byte rows (128-byte swizzle) or
// 64-byte rows (64-byte swizzle), as the tensor maps lay them out.
__device__ __forceinline__ uint32_t orth_piece(uint32_t box, int r, int j) {
    return box + (uint32_t)r * 128 + (uint32_t)((j ^ (r & 7)) * 16);
}
__device__ __forceinline__ uint32_t orth_piece64(uint32_t box, int r, int j) {
    return box + (uint32_t)r * 64 + (uint32_t)((j ^ ((r >> 1) & 3)) * 16);
}

// Whether a row's diagonal of B takes lo: d its diagonal of A, sq of A0^2.  The 35 over
// G in `stray` is a middle: with 20 five steps are off by 1.6e-3 at a rank of m / 2 and
// 1.7e-3 on a square Gaussian matrix, with 35 by 1.9e-3 and 1.4e-3, with 70 by 2.4e-3 and
// 1.3e-3 (the largest over eleven shapes from 4 x 9 to 256 x 1024).
constexpr float kOrthStray = 35.f;
__device__ __forceinline__ bool orth_keeps(float d, float sq, float stray) { return sq <= stray * (d * d + sq); }

// Where a warp's 32 rows of a tile lie.
struct OrthRows {
    int64_t row;      // this thread's row of the batch's padded rows
    int64_t i;        // of its matrix
    int64_t i_warp;   // the warp's first
};

// 32 accumulators of row w.i, columns c0 .. c0 + 31 (c0 a multiple of 32, all
// inside the padded output), with their box; the results go back into it.  `diag`: these columns meet the warp's rows.
template <int kMode>
__device__ __forceinline__ void orth_epilogue(const OrthArgs& p, const OrthRows& w, bool diag, bool mirror,
                                              int64_t batch, int64_t c0, uint32_t box, int lane, uint32_t (&r)[32]) {
    constexpr float kInv = 1.f / kOrthScale;
    float v[32];
    if constexpr (kMode == kOrthGram || kMode == kOrthPoly) {
        if constexpr (kMode == kOrthGram) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * kInv;   // scaled A
            if (diag) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c0 + j == w.i) {
                        p.d[w.row] = v[j] * kInv;
                        v[j] = 0.f;
                    }
            }
        } else {
            const float di = p.d[w.row];
            const float4* dc = reinterpret_cast<const float4*>(p.d + batch * p.mp + c0);
            const float k0 = p.b + p.c * di;
            float sq = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 x = lds_v4(orth_piece64(box, lane, q));
                const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float4 dj = dc[2 * q + g];
                    const float ds[4] = {dj.x, dj.y, dj.z, dj.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = 8 * q + 4 * g + k;
                        const float a0 = (k & 1) ? h_hi(ws[2 * g + (k >> 1)]) : h_lo(ws[2 * g + (k >> 1)]);
                        const float s = __uint_as_float(r[j]) * kInv;   // scaled A0^2
                        if (diag && c0 + j == w.i) sq = s;
                        v[j] = (k0 + p.c * ds[k]) * a0 + p.c * s;
                    }
                }
            }
            if (diag && w.i >= c0 && w.i < c0 + 32) {
                const float ei = p.b * di + p.c * (di * di) + p.c * (sq * kInv);
                p.e[w.row] = ei;
                p.f[w.row] = orth_keeps(di, sq * kInv, p.stray) ? ei : 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c0 + j == w.i) v[j] = 0.f;
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            sts_v4(orth_piece64(box, lane, q), orth_pack(v[8 * q], v[8 * q + 1]),
                   orth_pack(v[8 * q + 2], v[8 * q + 3]), orth_pack(v[8 * q + 4], v[8 * q + 5]),
                   orth_pack(v[8 * q + 6], v[8 * q + 7]));
        if (mirror) {
            __half* o = p.mat_out + (batch * p.mp + c0) * p.mp + w.i;
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j * p.mp] = __float2half_rn(v[j]);
        }
    } else {
        const float ah = p.a + p.e[w.row], al = (p.a + p.f[w.row]) * (1.f / kOrthLoScale);
        const uint32_t lo_box = box + kOrthSquareBytes;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 h = lds_v4(orth_piece64(box, lane, q)), l = lds_v4(orth_piece64(lo_box, lane, q));
            const uint32_t hs[4] = {h.x, h.y, h.z, h.w}, ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float xh = (k & 1) ? h_hi(hs[k >> 1]) : h_lo(hs[k >> 1]);
                const float xl = (k & 1) ? h_hi(ls[k >> 1]) : h_lo(ls[k >> 1]);
                v[8 * q + k] = ah * xh + (al * xl + __uint_as_float(r[8 * q + k]) * kInv);
            }
        }
        if constexpr (kMode == kOrthApply) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x0 = v[8 * q + 2 * k], x1 = v[8 * q + 2 * k + 1];
                    hw[k] = orth_pack(x0, x1);
                    lw[k] = orth_pack((x0 - h_lo(hw[k])) * kOrthLoScale, (x1 - h_hi(hw[k])) * kOrthLoScale);
                }
                sts_v4(orth_piece64(box, lane, q), hw[0], hw[1], hw[2], hw[3]);
                sts_v4(orth_piece64(lo_box, lane, q), lw[0], lw[1], lw[2], lw[3]);
            }
        } else {
            const float s = p.scale * kInv;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= s;
            if (p.transposed) {   // 32 lanes, 32 neighbours of each output row
                if (w.i < p.m) {
                    const int64_t base = batch * p.stride_out;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (c0 + j < p.n) {
                            const int64_t at = base + (c0 + j) * p.ld_out + w.i;
                            if (p.out_dtype == 2) static_cast<float*>(p.out)[at] = v[j];
                            else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v[j]);
                        }
                    }
                }
            } else if (p.out_dtype == 2) {   // both boxes as 32 rows of 128 bytes
                __syncwarp();                // every lane has read its hi and lo
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    sts_v4(orth_piece(box, lane, q), __float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                           __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    sts_v4(orth_piece64(box, lane, q), pack_bf16x2(v[8 * q], v[8 * q + 1]),
                           pack_bf16x2(v[8 * q + 2], v[8 * q + 3]), pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                           pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
            }
        }
    }
}

// Final: a box of 32 rows and columns to the output, a row's 16-byte pieces by
// neighbouring lanes.
template <class T>
__device__ __forceinline__ void orth_write_out(const OrthArgs& p, const OrthRows& w, int64_t batch, int64_t c0,
                                               uint32_t box, int lane) {
    constexpr int kPiece = 16 / (int)sizeof(T), kPieces = 32 / kPiece;   // values a piece, pieces a row
    T* out = static_cast<T*>(p.out) + batch * p.stride_out;
    auto piece = [&](int r, int j) { return sizeof(T) == 4 ? orth_piece(box, r, j) : orth_piece64(box, r, j); };
    if (p.vec_out && c0 + 32 <= p.n) {
#pragma unroll
        for (int g = 0; g < kPieces; ++g) {
            const int r = g * (32 / kPieces) + lane / kPieces, j = lane % kPieces;
            if (w.i_warp + r < p.m)
                *reinterpret_cast<uint4*>(out + (w.i_warp + r) * p.ld_out + c0 + j * kPiece) = lds_v4(piece(r, j));
        }
    } else if (c0 + lane < p.n) {
        for (int r = 0; r < 32 && w.i_warp + r < p.m; ++r) {
            const uint32_t at = piece(r, lane / kPiece) + (lane % kPiece) * (uint32_t)sizeof(T);
            T x;
            if constexpr (sizeof(T) == 4) {
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
            } else {
                unsigned short h;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(at) : "memory");
                x = *reinterpret_cast<const T*>(&h);
            }
            out[(w.i_warp + r) * p.ld_out + c0 + lane] = x;
        }
    }
}

// D tiles = A B^T (Gram, Poly; both operands K-major rows) or A B (Apply, Final;
// B read MN-major).  tm_a, tm_b: operands, boxes of 64 columns x the CTA's rows of
// a K block (MN-major: x 64 rows).  For
// the epilogue boxes of 32 rows x 32 columns: tm_in, tm_lo what it reads (Poly: A0; Apply, Final: hi and lo), tm_out
// what it writes beside lo.
template <int kMode, int kBN, bool kPair>
__global__ void __launch_bounds__(kOrthProductThreads, 1)
k_orth_product(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
               const __grid_constant__ CUtensorMap tm_in, const __grid_constant__ CUtensorMap tm_lo,
               const __grid_constant__ CUtensorMap tm_out, OrthArgs p) {
    constexpr bool kSym = kMode == kOrthGram || kMode == kOrthPoly;
    constexpr int kBM = kPair ? 256 : 128, kStages = kOrthStages<kBN, kPair, kSym>, kBoxes = kOrthBoxes;
    constexpr uint32_t kBoxBytes = kOrthBoxBytes<kSym>;
    constexpr uint32_t kStageBytes = kOrthStageBytes<kBN, kPair>;
    extern __shared__ __align__(1024) unsigned char orth_smem_raw[];
    const uint32_t raw = smem_u32(orth_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in both CTAs of a pair
    const uint32_t bars = base + kStages * kStageBytes;
    const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
    const uint32_t tfull0 = bars + 16 * kStages, tempty0 = tfull0 + 16;
    const uint32_t drain = tempty0 + 16;
    const uint32_t in0 = drain + 8;   // the epilogue warps' boxes
    const uint32_t slot = in0 + 8 * kOrthEpiWarps * kBoxes;
    unsigned char* slot_gen = orth_smem_raw + (slot - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(slot_gen);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_gen + 4);
    const uint32_t boxes = bars + 1024;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair ? cluster_rank() : 0;
    const bool leader = rank == 0;
    const int64_t first = kPair ? cluster_id_x() : blockIdx.x, step = kPair ? cluster_count_x() : gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, (kPair ? 2 : 1) * kOrthEpiWarps);   // one arrival per epilogue warp
        }
        mbar_init(drain, 1);
        for (int k = 0; k < kOrthEpiWarps * kBoxes; ++k) mbar_init(in0 + 8 * k, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
        if (kMode != kOrthGram) prefetch_tmap(&tm_in);
        if (!kSym) prefetch_tmap(&tm_lo);
        if (kMode != kOrthFinal) prefetch_tmap(&tm_out);
    }
    if (warp == 1) {
        if constexpr (kPair) {
            tmem_alloc_pair(slot, 2 * kBN);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(slot, 2 * kBN);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if constexpr (kPair) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    orth_dep_wait();   // the operands are the previous launch's output

    if (warp == 0) {
        // ---------------- TMA producer: this CTA's rows of A and its part of B; in
        // a pair every copy completes on the even CTA's stage barrier
        if (lane == 0) {
            const uint32_t full = kPair ? map_to_rank(full0, 0) : full0;
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            auto load = [&](uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
                if constexpr (kPair) tma_load_2d_pair(dst, map, x, y, bar);
                else tma_load_2d(dst, map, x, y, bar);
            };
            for (int64_t u = first; ok && u < p.units; u += step) {
                const OrthUnit w = orth_unit<kSym, kBM, kBN>(u, p);
                const int row0 = (int)(w.batch * p.mp);
                const int m0 = row0 + w.mb * kBM + (int)rank * 128;
                const int n0 = w.nb * kBN + (kPair ? (int)rank * (kBN / 2) : 0);
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!orth_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + stage * kStageBytes, bar = full + 8 * stage;
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, (kPair ? 2 : 1) * kStageBytes);
                    load(dst, &tm_a, kb * kOrthBK, m0, bar);
                    if constexpr (kSym) {
                        load(dst + kOrthABytes, &tm_b, kb * kOrthBK, row0 + n0, bar);
                    } else {
#pragma unroll
                        for (int j = 0; j < (int)(kOrthBBytes<kBN, kPair> / 8192); ++j)
                            load(dst + kOrthABytes + j * 8192, &tm_b, n0 + 64 * j, row0 + kb * kOrthBK, bar);
                    }
                    issued |= 1u << stage;
                    last_par = (last_par & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok && leader) {
                for (int s = 0; s < kStages; ++s)
                    if (issued & (1u << s)) mbar_wait(full0 + 8 * s, (last_par >> s) & 1u, kOrthWaitCycles);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (of a pair: the even CTA's, for both)
        if (leader && lane == 0) {
            constexpr uint32_t idesc = orth_idesc<kBM, kBN, !kSym>();
            const uint32_t empty_peer = kPair ? map_to_rank(empty0, 1) : 0, tfull_peer = kPair ? map_to_rank(tfull0, 1) : 0;
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            auto commit = [&](uint32_t bar, uint32_t peer) {
                if constexpr (kPair) {
                    umma_commit_pair(bar);
                    umma_commit_pair(peer);
                } else {
                    umma_commit(bar);
                }
            };
            for (int64_t u = first; ok && u < p.units; u += step) {
                if (!orth_wait_acc<kPair>(tempty0 + 8 * acc, acc_phase ^ 1u, abort_flag)) break;
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
                    const uint64_t b_desc = kSym ? orth_desc_k(addr + kOrthABytes) : orth_desc_mn(addr + kOrthABytes);
                    constexpr uint64_t kBStep = kSym ? (32 >> 4) : (2048 >> 4);
#pragma unroll
                    for (int k = 0; k < kOrthBK / 16; ++k) {
                        const uint32_t more = (kb != 0 || k != 0) ? 1u : 0u;
                        if constexpr (kPair) umma_bf16_pair(d_tmem, a_desc + (32 >> 4) * k, b_desc + kBStep * k, idesc, more);
                        else umma_bf16(d_tmem, a_desc + (32 >> 4) * k, b_desc + kBStep * k, idesc, more);
                    }
                    commit(empty0 + 8 * stage, empty_peer + 8 * stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                commit(tfull0 + 8 * acc, tfull_peer + 8 * acc);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            if constexpr (kPair) umma_commit_pair(drain);
            else umma_commit(drain);
            mbar_wait(drain, 0, kOrthWaitCycles);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: 32 rows and half of the columns a warp
        const int q = warp & 3, e = warp - 2;   // tensor memory's lanes go by warp mod 4
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t tempty = kPair ? map_to_rank(tempty0, 0) : tempty0;
        const int64_t cols = kSym ? p.mp : p.np;
        const uint32_t my_boxes = boxes + (uint32_t)e * kBoxes * kBoxBytes, my_in = in0 + (uint32_t)e * 8 * kBoxes;
        constexpr bool kReads = kMode != kOrthGram;
        constexpr int kWide = 32;   // columns of a chunk
        int acc = 0, buf = 0;
        uint32_t acc_phase = 0, in_phase = 0, pending = 0;   // bit per box
        bool ok = true;
        for (int64_t u = first; ok && u < p.units; u += step) {
            const OrthUnit w = orth_unit<kSym, kBM, kBN>(u, p);
            OrthRows o;
            o.i_warp = (int64_t)w.mb * kBM + (int64_t)rank * 128 + q * 32;
            o.i = o.i_warp + lane;
            o.row = w.batch * p.mp + o.i;
            const int64_t n0 = (int64_t)w.nb * kBN;
            const int y = (int)(w.batch * p.mp + o.i_warp);
            const bool mirror = kSym && n0 >= (int64_t)(w.mb + 1) * kBM;
            int chunks = o.i_warp < p.mp ? (int)((cols - n0) / kWide) : 0;   // cols and n0 are multiples of 64
            if (chunks > kBN / kWide) chunks = kBN / kWide;
            const int part = (chunks + 1) / 2, c_from = e < 4 ? 0 : part, c_to = e < 4 ? part : chunks;
            auto fetch = [&](int c, int b) {   // lane 0: what chunk c reads
                const uint32_t box = my_boxes + (uint32_t)b * kBoxBytes, bar = my_in + 8 * b;
                mbar_arrive_expect_tx(bar, kBoxBytes);
                tma_load_2d(box, &tm_in, (int)n0 + kWide * c, y, bar);
                if constexpr (!kSym) tma_load_2d(box + kOrthSquareBytes, &tm_lo, (int)n0 + kWide * c, y, bar);
            };
            if (kReads) {
                if (c_from < c_to) {
                    if (lane == 0) {
                        bulk_wait_read<0>();   // the stores out of the boxes have read them
                        fetch(c_from, buf);
                    }
                    pending |= 1u << buf;
                }
            }
            ok = __all_sync(0xffffffffu, orth_wait(tfull0 + 8 * acc, acc_phase, abort_flag));
            if (!ok) break;
            tc_fence_after();
            for (int c = c_from; c < c_to; ++c) {
                const uint32_t box = my_boxes + (uint32_t)buf * kBoxBytes;
                if (kReads) {
                    if (c + 1 < c_to) {
                        const int b = (buf + 1) % kBoxes;
                        if (lane == 0) {
                            bulk_wait_read<0>();   // the store that last used this box
                            fetch(c + 1, b);
                        }
                        pending |= 1u << b;
                    }
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, orth_wait(my_in + 8 * buf, (in_phase >> buf) & 1u, abort_flag));
                    if (!ok) break;
                    in_phase ^= 1u << buf;
                    pending &= ~(1u << buf);
                } else if (lane == 0) {
                    bulk_wait_read<kBoxes - 1>();   // the store that last used this box
                }
                __syncwarp();
                const int64_t c0 = n0 + kWide * c;
                const bool diag = kSym && c0 < o.i_warp + 32 && o.i_warp < c0 + kWide;
                uint32_t r[32];
                tmem_ld32(lane_addr + (uint32_t)(acc * kBN + kWide * c), r);
                orth_epilogue<kMode>(p, o, diag, mirror, w.batch, c0, box, lane, r);
                if constexpr (kMode == kOrthFinal) {
                    if (!p.transposed) {
                        __syncwarp();
                        if (p.out_dtype == 2) orth_write_out<float>(p, o, w.batch, c0, box, lane);
                        else orth_write_out<__nv_bfloat16>(p, o, w.batch, c0, box, lane);
                    }
                    fence_proxy_async_smem();   // before the next copy into this box
                    __syncwarp();
                } else {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tm_out, (int)c0, y, box);
                        if constexpr (!kSym) tma_store_2d(&tm_lo, (int)c0, y, box + kOrthSquareBytes);
                        bulk_commit_group();
                    }
                }
                buf = (buf + 1) % kBoxes;
            }
            if (!ok) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair) mbar_arrive_cluster(tempty + 8 * acc);
                else mbar_arrive(tempty + 8 * acc);
            }
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (!ok && lane == 0) {   // the boxes' copies in flight
            for (int b = 0; b < kBoxes; ++b)
                if (pending & (1u << b)) mbar_wait(my_in + 8 * b, (in_phase >> b) & 1u, kOrthWaitCycles);
        }
        if (lane == 0) bulk_wait_read<0>();   // shared memory is read before the CTA exits
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync_all();   // no copy, arrival or MMA of the pair still targets either CTA
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kPair) tmem_dealloc_pair(tmem, 2 * kBN);
        else tmem_dealloc(tmem, 2 * kBN);
    }
}

// ---------------------------------------------------------------- few tiles

// A product with fewer tiles than SMs is bound by the latencies of one tile: the
// copy engine's rate (a 128 x 128 tile's K block of 32 KB takes about 500 cycles),
// the first copy's 2000 and the epilogue.  Here a cluster of 1, 2 or 4 CTAs shares
// a 128 x 128 tile, each taking a part of K.  A CTA puts its FP32 partial into
// shared memory by column shares and pushes the others' into their CTAs with bulk
// copies (reading them from there took 4000 cycles); each adds its share in CTA
// order and finishes those columns straight from and to global memory, with what it
// reads there loaded before the K loop.
constexpr int kOrthSplitStages = 4;
constexpr uint32_t kOrthSplitRecv = kOrthSplitStages * 32768;   // 64 KB of partials from the others
constexpr size_t kOrthSplitSmem = 1024 + kOrthSplitRecv + 65536 + 256;
static_assert(kOrthSplitSmem <= 232448, "shared memory per CTA");

// Of 16-byte piece j (4 floats) of row r of 128 x 128 FP32 partials.
__device__ __forceinline__ uint32_t orth_part_piece(uint32_t p, int r, int j) {
    return p + (uint32_t)r * 512 + (uint32_t)((j ^ (r & 7)) * 16);
}
__device__ __forceinline__ float4 dsm_ld(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
// Shared memory of this CTA to another's, completing on a barrier there.
__device__ __forceinline__ void dsm_push(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// What the columns c0 .. c0 + 31 of a row need beside the accumulators.
struct OrthInputs {
    uint4 a[4], b[4];   // Poly: A0 and d (two halves); Apply, Final: hi, lo
    uint4 d[4];
};
template <int kMode>
__device__ __forceinline__ void orth_inputs(const OrthArgs& p, int64_t batch, int64_t row, int64_t c0, OrthInputs& in) {
    if constexpr (kMode == kOrthPoly) {
        const uint4* a = reinterpret_cast<const uint4*>(p.mat_in + row * p.mp + c0);
        const uint4* d = reinterpret_cast<const uint4*>(p.d + batch * p.mp + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            in.a[q] = a[q];
            in.b[q] = d[q];
            in.d[q] = d[4 + q];
        }
    } else if constexpr (kMode != kOrthGram) {
        const uint4* h = reinterpret_cast<const uint4*>(p.x_hi + row * p.np + c0);
        const uint4* l = reinterpret_cast<const uint4*>(p.x_lo + row * p.np + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            in.a[q] = h[q];
            in.b[q] = l[q];
        }
    }
}
__device__ __forceinline__ float orth_word_f(const uint4& v, int k) {
    return __uint_as_float(k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w);
}
__device__ __forceinline__ float orth_half_f(const uint4& v, int k) {
    const uint32_t w = (k >> 1) == 0 ? v.x : (k >> 1) == 1 ? v.y : (k >> 1) == 2 ? v.z : v.w;
    return (k & 1) ? h_hi(w) : h_lo(w);
}

// Columns c0 .. c0 + 31 of row `row` (i of its matrix): the accumulators v to the result.
template <int kMode>
__device__ __forceinline__ void orth_finish(const OrthArgs& p, int64_t batch, int64_t row, int64_t i, int64_t c0,
                                            bool mirror, float2 side, const OrthInputs& in, float (&v)[32]) {
    constexpr float kInv = 1.f / kOrthScale;
    if constexpr (kMode == kOrthGram || kMode == kOrthPoly) {
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float s = v[j] * kInv;
            if constexpr (kMode == kOrthGram) {
                v[j] = s;
                if (c0 + j == i) {
                    p.d[row] = s * kInv;
                    v[j] = 0.f;
                }
            } else {   // side.x = d_i
                const float dj = orth_word_f(j < 16 ? in.b[j >> 2] : in.d[(j >> 2) - 4], j & 3);
                v[j] = (p.b + p.c * (side.x + dj)) * orth_half_f(in.a[j >> 3], j & 7) + p.c * s;
                if (c0 + j == i) {
                    sq = s * kInv;
                    v[j] = 0.f;
                }
            }
        }
        if (kMode == kOrthPoly && i >= c0 && i < c0 + 32) {
            const float ei = p.b * side.x + p.c * (side.x * side.x) + p.c * sq;
            p.e[row] = ei;
            p.f[row] = orth_keeps(side.x, sq, p.stray) ? ei : 0.f;
        }
        uint4* o = reinterpret_cast<uint4*>(p.mat_out + row * p.mp + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = make_uint4(orth_pack(v[8 * q], v[8 * q + 1]), orth_pack(v[8 * q + 2], v[8 * q + 3]),
                              orth_pack(v[8 * q + 4], v[8 * q + 5]), orth_pack(v[8 * q + 6], v[8 * q + 7]));
        if (mirror) {
            __half* t = p.mat_out + (batch * p.mp + c0) * p.mp + i;
#pragma unroll
            for (int j = 0; j < 32; ++j) t[j * p.mp] = __float2half_rn(v[j]);
        }
    } else {   // side = a + e_i, and a + f_i over lo's scale
#pragma unroll
        for (int j = 0; j < 32; ++j)
            v[j] = side.x * orth_half_f(in.a[j >> 3], j & 7) + (side.y * orth_half_f(in.b[j >> 3], j & 7) + v[j] * kInv);
        if constexpr (kMode == kOrthApply) {
            uint4* oh = reinterpret_cast<uint4*>(p.x_out + row * p.np + c0);
            uint4* ol = reinterpret_cast<uint4*>(p.x_lo + row * p.np + c0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x0 = v[8 * q + 2 * k], x1 = v[8 * q + 2 * k + 1];
                    hw[k] = orth_pack(x0, x1);
                    lw[k] = orth_pack((x0 - h_lo(hw[k])) * kOrthLoScale, (x1 - h_hi(hw[k])) * kOrthLoScale);
                }
                oh[q] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                ol[q] = make_uint4(lw[0], lw[1], lw[2], lw[3]);
            }
        } else if (i < p.m) {
            const float s = p.scale * kInv;
            const int64_t base = batch * p.stride_out;
            if (p.vec_out && !p.transposed && c0 + 32 <= p.n) {
                if (p.out_dtype == 2) {
                    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + base + i * p.ld_out + c0);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        o[q] = make_float4(s * v[4 * q], s * v[4 * q + 1], s * v[4 * q + 2], s * v[4 * q + 3]);
                } else {
                    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + base + i * p.ld_out + c0);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        o[q] = make_uint4(pack_bf16x2(s * v[8 * q], s * v[8 * q + 1]),
                                          pack_bf16x2(s * v[8 * q + 2], s * v[8 * q + 3]),
                                          pack_bf16x2(s * v[8 * q + 4], s * v[8 * q + 5]),
                                          pack_bf16x2(s * v[8 * q + 6], s * v[8 * q + 7]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (c0 + j < p.n) {
                        const int64_t at = base + (p.transposed ? (c0 + j) * p.ld_out + i : i * p.ld_out + c0 + j);
                        if (p.out_dtype == 2) static_cast<float*>(p.out)[at] = s * v[j];
                        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(s * v[j]);
                    }
                }
            }
        }
    }
}

template <int kMode>
__global__ void __launch_bounds__(kOrthThreads, 1)
k_orth_split(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, OrthArgs p) {
    constexpr bool kSym = kMode == kOrthGram || kMode == kOrthPoly;
    constexpr int kStages = kOrthSplitStages;
    constexpr uint32_t kStageBytes = 32768;
    extern __shared__ __align__(1024) unsigned char orth_smem_raw[];
    const uint32_t raw = smem_u32(orth_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in every CTA of the cluster
    const uint32_t recv = base + kOrthSplitRecv, bars = recv + 65536;
    const uint32_t full0 = bars, empty0 = bars + 8 * kStages, tfull = bars + 16 * kStages, got = tfull + 8, slot = got + 8;
    unsigned char* slot_gen = orth_smem_raw + (slot - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(slot_gen);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_gen + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const uint32_t rank = cluster_rank();
    const OrthUnit w = orth_unit<kSym, 128, 128>(blockIdx.x / split, p);
    const int kb0 = (int)(p.nkb * rank / split), kb1 = (int)(p.nkb * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(tfull, 1);
        mbar_init(got, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (split > 1) mbar_arrive_expect_tx(got, (split - 1) * (65536 / split));
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
    }
    if (warp == 1) {
        tmem_alloc(slot, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (split > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // ready to receive
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    orth_dep_wait();

    // the epilogue's share: 32 rows a warp, 128 / split columns of the tile
    const int q = warp & 3, r = q * 32 + lane;
    const bool epilogue = warp >= 2;
    const int64_t cols = kSym ? p.mp : p.np;
    const int64_t i_warp = (int64_t)w.mb * 128 + q * 32, i = i_warp + lane, row = w.batch * p.mp + i;
    const int lw = split == 1 ? 7 : split == 2 ? 6 : 5;   // log2 of the columns
    const int width = 1 << lw, from = (int)rank * width;   // of the tile's columns
    const int64_t n0 = (int64_t)w.nb * 128;
    int chunks = epilogue && i_warp < p.mp ? width / 32 : 0;
    while (chunks > 0 && n0 + from + 32 * (chunks - 1) >= cols) --chunks;
    OrthInputs in;
    float2 side = {0.f, 0.f};
    if (warp == 0) {
        if (lane == 0) {
            const int row0 = (int)(w.batch * p.mp), m0 = row0 + w.mb * 128;
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!orth_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = base + stage * kStageBytes, bar = full0 + 8 * stage;
                mbar_arrive_expect_tx(bar, kStageBytes);
                tma_load_2d(dst, &tm_a, kb * kOrthBK, m0, bar);
                if constexpr (kSym) {
                    tma_load_2d(dst + kOrthABytes, &tm_b, kb * kOrthBK, row0 + (int)n0, bar);
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        tma_load_2d(dst + kOrthABytes + j * 8192, &tm_b, (int)n0 + 64 * j, row0 + kb * kOrthBK, bar);
                }
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) {
                for (int s = 0; s < kStages; ++s)
                    if (issued & (1u << s)) mbar_wait(full0 + 8 * s, (last_par >> s) & 1u, kOrthWaitCycles);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = orth_idesc<128, 128, !kSym>();
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!orth_wait(full0 + 8 * stage, phase, abort_flag)) break;
                tc_fence_after();
                const uint32_t addr = base + stage * kStageBytes;
                const uint64_t a_desc = orth_desc_k(addr);
                const uint64_t b_desc = kSym ? orth_desc_k(addr + kOrthABytes) : orth_desc_mn(addr + kOrthABytes);
                constexpr uint64_t kBStep = kSym ? (32 >> 4) : (2048 >> 4);
#pragma unroll
                for (int k = 0; k < kOrthBK / 16; ++k)
                    umma_bf16(tmem, a_desc + (32 >> 4) * k, b_desc + kBStep * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
                umma_commit(empty0 + 8 * stage);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            umma_commit(tfull);   // also after a wait that ran out: what was issued drains
        }
    } else if (chunks > 0) {
        if constexpr (kMode == kOrthPoly) side.x = p.d[row];
        else if constexpr (!kSym) side = make_float2(p.a + p.e[row], (p.a + p.f[row]) * (1.f / kOrthLoScale));
        orth_inputs<kMode>(p, w.batch, row, n0 + from, in);
    }
    __syncwarp();
    // Everyone waits for the MMAs: shared memory is free after them, and no CTA leaves
    // before its own are done.
    const bool ok = orth_wait(tfull, 0, abort_flag);
    tc_fence_after();
    const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
    __syncthreads();
    const uint32_t share = (uint32_t)width * 512;              // bytes of a share of the partial tile
    const uint32_t pitch = (uint32_t)width * 4;
    auto piece = [&](uint32_t buf, int j) { return buf + (uint32_t)r * pitch + (uint32_t)((j ^ (r & 7)) * 16); };
    if (split > 1) {
        if (epilogue && i_warp < p.mp) {   // over the stages
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t t[32];
                __syncwarp();
                tmem_ld32(lane_addr + 32 * c, t);
                const uint32_t buf = base + ((uint32_t)(32 * c) >> lw) * share;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sts_v4(piece(buf, ((32 * c) & (width - 1)) / 4 + k), t[4 * k], t[4 * k + 1], t[4 * k + 2], t[4 * k + 3]);
            }
            fence_proxy_async_smem();
        }
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // the others can receive
        __syncthreads();
        if (threadIdx.x == 0)
            for (uint32_t k = 0; k < split; ++k)
                if (k != rank) dsm_push(map_to_rank(recv + rank * share, k), base + k * share, share, map_to_rank(got, k));
        orth_wait(got, 0, abort_flag);
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // has the others' partials
    }
    const bool mirror = kSym && w.nb > w.mb;
    for (int c = 0; c < chunks; ++c) {
        float v[32];
        OrthInputs ahead;
        if (c + 1 < chunks) orth_inputs<kMode>(p, w.batch, row, n0 + from + 32 * (c + 1), ahead);
        if (split > 1) {
#pragma unroll
            for (uint32_t s = 0; s < 4; ++s) {
                if (s < split) {
                    const uint32_t buf = s == rank ? base + rank * share : recv + s * share;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 t = lds_v4(piece(buf, 8 * c + k));
                        const float f[4] = {__uint_as_float(t.x), __uint_as_float(t.y), __uint_as_float(t.z),
                                            __uint_as_float(t.w)};
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[4 * k + j] = s == 0 ? f[j] : v[4 * k + j] + f[j];
                    }
                }
            }
        } else {
            uint32_t t[32];
            __syncwarp();
            tmem_ld32(lane_addr + 32 * c, t);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(t[j]);
        }
        orth_finish<kMode>(p, w.batch, row, i, n0 + from + 32 * c, mirror, side, in, v);
        in = ahead;
    }
    tc_fence_before();
    __syncwarp();
    // the others have this CTA's partials
    if (split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
    (void)ok;
}

// ---------------------------------------------------------------- the input

// A sum of squares, s 4^e.  e is 0 unless the FP32 sum of the squares themselves
// would overflow or lose what underflows.
struct OrthSum {
    float s;
    int e;
};
constexpr float kOrthSumLow = 0x1p-60f, kOrthSumHigh = 0x1p100f;   // between them it is taken as it is
// 2^-e as two factors (2^-e itself may be out of range): values below 2^(e + 1) take the
// first, then the second, without overflow.
__device__ __forceinline__ float2 orth_scale_of(int e) {
    const int h = e / 2;
    return make_float2(__int_as_float((127 - h) << 23), __int_as_float((127 - (e - h)) << 23));
}
__device__ __forceinline__ bool orth_sum_plain(float s) { return s >= kOrthSumLow && s <= kOrthSumHigh; }

struct OrthInput {
    const void* x;            // [rows, ld] of T, matrices `stride` elements apart
    int64_t rows, cols, ld, stride;
    int64_t tiles_m, tiles;   // of X: 64 x 64 tiles down, and of one matrix
    int64_t all_tiles;        // of the batch
    int transposed;           // X = x^T
    int vec;                  // rows of x are whole, aligned 16-byte vectors
    int parts;                // partial sums of a matrix, at most 256
    float eps;
    OrthSum* sums;            // [batch, parts]
    __half *hi, *lo;          // [batch mp, np]
    int64_t mp, np;
};

__device__ __forceinline__ float orth_f32(float v) { return v; }
__device__ __forceinline__ float orth_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float orth_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
// The 16 / sizeof(T) values of a vector.
template <class T>
__device__ __forceinline__ void orth_vec(const T* p, float (&v)[16 / sizeof(T)]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int k = 0; k < 16 / (int)sizeof(T); ++k) v[k] = orth_f32(e[k]);
}

// Partial sums of squares: part q of a matrix takes its rows q, q + parts, ..., a warp
// a run of a row at a time (whole rows left most warps without one where a part
// has few: a call on 8 x 1024 x 4096 took 679 us, now 672).
constexpr int kOrthSumThreads = 512;
// A thread's share of it (kOrthSquares), of the scaled values' (kOrthScaled), or its largest |x|.
enum OrthSumKind { kOrthSquares = 0, kOrthScaled = 1, kOrthLargest = 2 };
template <class T, int kKind>
__device__ __forceinline__ float orth_part(const OrthInput& p, const T* x, int q, float2 by = {1.f, 1.f}) {
    constexpr int V = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int64_t rows = (p.rows - q + p.parts - 1) / p.parts;
    float s[4] = {0.f, 0.f, 0.f, 0.f};   // four chains: the adds of one would wait on each other
    auto take = [&](float& t, float v) {
        if (kKind == kOrthLargest) {
            t = fmaxf(t, fabsf(v));
        } else {
            if (kKind == kOrthScaled) v = v * by.x * by.y;
            t += v * v;
        }
    };
    // a run: four vectors a lane, or 16 values of unaligned rows
    const int64_t have = p.vec ? p.cols / V : p.cols, runs = (have + (p.vec ? 127 : 511)) / (p.vec ? 128 : 512);
    for (int64_t u = threadIdx.x >> 5; u < rows * runs; u += kOrthSumThreads / 32) {
        const int64_t r = u / runs;
        const T* row = x + (q + r * p.parts) * p.ld;
        if (p.vec) {
            const int64_t c = (u - r * runs) * 128 + lane;
            float v[4][V];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + 32 * k < have) orth_vec<T>(row + (c + 32 * k) * V, v[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + 32 * k < have)
#pragma unroll
                    for (int j = 0; j < V; ++j) take(s[k], v[k][j]);
        } else {
            const int64_t c = (u - r * runs) * 512 + lane;
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = c + 32 * k < have ? orth_f32(row[c + 32 * k]) : 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) take(s[k & 3], v[k]);
        }
    }
    if (kKind == kOrthLargest) return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    return (s[0] + s[1]) + (s[2] + s[3]);
}
// Its sum (or largest) over the CTA, the same in every thread.
template <bool kLargest>
__device__ __forceinline__ float orth_cta(float t, float* red) {
    auto join = [](float a, float b) { return kLargest ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t = join(t, __shfl_xor_sync(0xffffffffu, t, o));
    __syncthreads();   // the last one's readers
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
    __syncthreads();
    t = (threadIdx.x & 31) < kOrthSumThreads / 32 ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) t = join(t, __shfl_xor_sync(0xffffffffu, t, o));
    return t;
}
template <class T>
__global__ void __launch_bounds__(kOrthSumThreads, 2)
k_orth_sumsq(OrthInput p) {
    __shared__ float red[kOrthSumThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t b = blockIdx.x / p.parts;
    const int q = (int)(blockIdx.x - b * p.parts);
    const T* x = static_cast<const T*>(p.x) + b * p.stride;
    OrthSum t{orth_cta<false>(orth_part<T, kOrthSquares>(p, x, q), red), 0};
    if (!orth_sum_plain(t.s)) {   // again, with the largest scaled to between 1 and 2
        const float top = orth_cta<true>(orth_part<T, kOrthLargest>(p, x, q), red);
        if (top > 0.f && isfinite(top)) {   // else zeros, or nothing that a scale would mend
            t.e = ilogbf(top);
            t.s = orth_cta<false>(orth_part<T, kOrthScaled>(p, x, q, orth_scale_of(t.e)), red);
        }
    }
    if (threadIdx.x == 0) p.sums[blockIdx.x] = t;
}

// `by` / (|x| + eps) as two factors, for a matrix of the sum of squares t: 0 for a matrix of
// zeros, NaN where the sum is not finite.
__device__ __forceinline__ float2 orth_inverse(OrthSum t, float eps, float by) {
    if (!isfinite(t.s)) return make_float2(1.f, __int_as_float(0x7fc00000));
    const float2 f = orth_scale_of(t.e);
    return make_float2(f.x, t.s > 0.f ? by / (__fsqrt_rn(t.s) + eps * f.x * f.y) * f.y : 0.f);
}

// X (hi, lo) = x / (|x| + eps), zero in the padding: a 64 x 64 tile of X a turn,
// through shared memory (turned there when X is x's transpose) unless x's rows
// are aligned vectors already in X's order.
constexpr int kOrthLoadThreads = 256;
template <class T>
__global__ void __launch_bounds__(kOrthLoadThreads, 5)
k_orth_load(OrthInput p) {
    constexpr int V = 16 / sizeof(T);
    __shared__ float tile[64][65];
    __shared__ float2 s_inv;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    orth_dep_wait();   // the partial sums
    int64_t have = -1;
    float2 inv = {0.f, 0.f};
    for (int64_t u = blockIdx.x; u < p.all_tiles; u += gridDim.x) {
        const int64_t b = u / p.tiles, t = u - b * p.tiles;
        const int64_t j0 = t / p.tiles_m * 64, i0 = t % p.tiles_m * 64;
        if (b != have) {   // the matrix's scale
            __syncthreads();
            if (threadIdx.x < 32) {
                const int2* sums = reinterpret_cast<const int2*>(p.sums + b * p.parts);
                OrthSum w{0.f, INT_MIN};   // the largest exponent of a part that is not 0
                for (int k = threadIdx.x; k < p.parts; k += 32) {
                    const int2 q = __ldcg(sums + k);
                    if (__int_as_float(q.x) != 0.f) w.e = max(w.e, q.y);
                }
                w.e = __reduce_max_sync(0xffffffffu, w.e);
                if (w.e == INT_MIN) w.e = 0;
                for (int k = threadIdx.x; k < p.parts; k += 32) {
                    const int2 q = __ldcg(sums + k);
                    w.s += q.y == w.e ? __int_as_float(q.x) : ldexpf(__int_as_float(q.x), 2 * (q.y - w.e));
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) w.s += __shfl_xor_sync(0xffffffffu, w.s, o);
                if (threadIdx.x == 0) s_inv = orth_inverse(w, p.eps, kOrthScale);
            }
            __syncthreads();
            inv = s_inv;
            have = b;
        }
        const T* x = static_cast<const T*>(p.x) + b * p.stride;
        const bool direct = p.vec && !p.transposed;
        if (!direct) {
            __syncthreads();   // the last tile's readers
            // tile[a][c] = x at row r0 + a, column c0 + c
            const int64_t r0 = p.transposed ? j0 : i0, c0 = p.transposed ? i0 : j0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int e = k * kOrthLoadThreads + threadIdx.x, a = e >> 6, c = e & 63;
                tile[a][c] = r0 + a < p.rows && c0 + c < p.cols ? orth_f32(x[(r0 + a) * p.ld + c0 + c]) : 0.f;
            }
            __syncthreads();
        }
        // 8 neighbouring values of X a thread and turn
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = k * kOrthLoadThreads + threadIdx.x, i = e >> 3, j = (e & 7) * 8;
            float v[8];
            if (direct) {
                const bool in = i0 + i < p.rows;
                const T* src = x + (i0 + i) * p.ld + j0 + j;
#pragma unroll
                for (int h = 0; h < 8 / V; ++h) {
                    float f[V];
                    if (in && j0 + j + V * h < p.cols) orth_vec<T>(src + V * h, f);   // whole vectors in a row
                    else
#pragma unroll
                        for (int q = 0; q < V; ++q) f[q] = 0.f;
#pragma unroll
                    for (int q = 0; q < V; ++q) v[V * h + q] = f[q];
                }
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = p.transposed ? tile[j + q][i] : tile[i][j + q];
            }
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float x0 = v[2 * q] * inv.x * inv.y, x1 = v[2 * q + 1] * inv.x * inv.y;
                hw[q] = orth_pack(x0, x1);
                lw[q] = orth_pack((x0 - h_lo(hw[q])) * kOrthLoScale, (x1 - h_hi(hw[q])) * kOrthLoScale);
            }
            const int64_t at = (b * p.mp + i0 + i) * p.np + j0 + j;
            *reinterpret_cast<uint4*>(p.hi + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(p.lo + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
    }
}

}  // namespace flp
