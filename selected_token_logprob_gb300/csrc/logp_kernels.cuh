// Device code of the selected-token log-probability path for sm_103a.
//
// Forward (RL-Kernel issue #241 "TP-aware deterministic logprob", Background
// and PR 3 bullets): LSE_t = log sum_v exp(s x[t, v]) with FP32 accumulation,
// logp_t = s x[t, y_t] - LSE_t, where s = 1/T is the inverse temperature
// (s = 1 unless rollout logprobs at a temperature are asked for, PR #495
// provider experiment).  Every row is cut into 16 fixed vocabulary tiles of
// width W = 8 * ceil(V / 128); one warp reduces one tile: each lane keeps an
// online (max, sumexp) pair over its fixed share of the tile, the warp merges
// the 32 pairs with a fixed xor butterfly, and a half warp merges the 16 tile
// partials with a fixed pairwise tree in tile-index order (RL-Kernel PR #314,
// Tensor Parallel section: fixed tiles, one fixed merge order).  Nothing in
// this order depends on N, on the row's position or on the grid, so every
// row's bits are batch-invariant, and a vocab shard that reduces its own tiles
// with the same functions reproduces the same partials bit for bit.
//
// Backward (RL-Kernel PR #495 "zero-workspace fused backward", Summary item
// 2): dlogits = s g (onehot - exp(s x - LSE)) from the saved LSE, one read
// and one write per logit, elementwise, written in the logits' dtype.
//
// Logits may be BF16, FP16 or FP32 (PR #495 Tests: FP32/BF16/FP16).  A
// "unit" is 8 consecutive elements of a row (16 bytes for 16-bit types, 32 for
// FP32); lane j of a warp owns units j, j + 32, ... of its tile.  Rows may be
// excluded by an explicit active mask (PR #314, MaskMode).  All index
// arithmetic is 64-bit except tile-local indices of the bulk forward.  The
// only waits are bounded waits of a warp on its own bulk copies.
#pragma once

#include "logp_units.cuh"

namespace flp {

// Sticky device error word: 1 = a bounded wait ran out.  Read and cleared by
// flp_device_error().
__device__ int g_device_error;

// ---------------------------------------------------------------- forward kernels

// Forward with plain loads (any alignment): one CTA of 16 warps per row, warp
// k reduces tile k.
template <Dt D, bool kScaled>
__global__ void __launch_bounds__(kFwdThreads)
k_logp_fwd(const void* __restrict__ x, int64_t n, int64_t v, int64_t ld, int64_t W,
           const int64_t* __restrict__ y, int64_t ignore_index, const uint8_t* __restrict__ mask,
           Scale sc, float* __restrict__ logp, float* __restrict__ lse, float* __restrict__ lse_lo) {
    __shared__ float sh_m[kTiles], sh_s[kTiles];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int EB = Unit<D>::kElemBytes;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        const char* xr = reinterpret_cast<const char*>(x) + t * ld * EB;
        bool act = false;
        float x_y = 0.f;
        if (threadIdx.x == 0) {
            const int64_t yt = __ldg(y + t);
            act = row_active(mask, t, yt, v, ignore_index);
            if (act) x_y = elem_value<D>(xr, yt);
        }
        const int64_t c0 = (int64_t)warp * W;
        const int64_t width = c0 >= v ? 0 : (v - c0 < W ? v - c0 : W);
        const MS p = tile_partial<kScaled>(tile_scan<D, false, kScaled>(xr + c0 * EB, width, lane, sc), sc);
        if (lane == 0) {
            sh_m[warp] = p.m;
            sh_s[warp] = p.s;
        }
        __syncthreads();
        if (warp == 0) {
            const int k = lane & 15;
            const MS f = tile_fold16(MS{sh_m[k], sh_s[k]}, sc.s);
            if (lane == 0)
                finalize_row(f, act, x_y, sc.s, logp + t, lse + t, lse_lo ? lse_lo + t : nullptr);
        }
        __syncthreads();
    }
}

// Forward with bulk copies (16-byte aligned rows whose byte stride is a
// multiple of 16, V < 2^31).  Persistent CTAs of 16 warps; CTA b takes rows
// b, b + grid, b + 2 grid, ...  Each warp streams its tile of successive rows
// through a private ring of kStages shared-memory stages (one group of 128
// units each): lane 0 issues cp.async.bulk for group i + kStages as soon as the
// warp has read group i, so copies of the next row are already in flight while
// a row is finished.  The lanes read the same words, in the same order, as
// tile_scan would load them (a ragged last unit is read from global memory),
// so results are bitwise those of k_logp_fwd.  Tile partials go to a
// double-buffered shared array; after one barrier per row, warp (row mod 16)
// merges them and writes the row.  A wait that runs out sets g_device_error;
// the warp then stops issuing copies and skips waits, and drains its copies in
// flight before exiting.
template <Dt D, bool kScaled>
__global__ void __launch_bounds__(kFwdThreads, kFwdMinBlocks<D>)
k_logp_fwd_bulk(const void* __restrict__ x, int64_t n, int64_t v, int64_t ld, int64_t W,
                const int64_t* __restrict__ y, int64_t ignore_index, const uint8_t* __restrict__ mask,
                Scale sc, float* __restrict__ logp, float* __restrict__ lse,
                float* __restrict__ lse_lo) {
    constexpr int EB = Unit<D>::kElemBytes;
    constexpr int UB = Unit<D>::kBytes;
    constexpr int SB = kStageBytes<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float sh_m[2][kTiles], sh_s[2][kTiles];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t stage0 = smem_u32(smem + warp * kStages * SB);
    const uint32_t bar0 = smem_u32(smem + kTiles * kStages * SB) + warp * kStages * 8;
    if (threadIdx.x < kTiles * kStages) mbar_init(smem_u32(smem + kTiles * kStages * SB) + threadIdx.x * 8, 1);
    fence_mbar_init();
    __syncthreads();

    // tile-local extents fit in 32 bits (the host routes V >= 2^31 elsewhere)
    const int64_t c0 = (int64_t)warp * W;
    const int width = (int)(c0 >= v ? 0 : (v - c0 < W ? v - c0 : W));
    const int nfull = width >> 3, nunit = (width + 7) >> 3;
    const int G = (nunit + kGroupUnits - 1) / kGroupUnits;       // groups per row
    const int Gfull = nfull / kGroupUnits;                       // groups of 128 full units
    const int64_t rows = (n > (int64_t)blockIdx.x) ? (n - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    const int64_t jobs = rows * G;
    const int64_t row_step = (int64_t)gridDim.x * ld * EB;      // bytes

    // Issuer: group iss_g of the row at iss_row (its first byte of this tile),
    // stage iss_st.  Every lane tracks it; lane 0 issues.
    const char* iss_row = reinterpret_cast<const char*>(x) + ((int64_t)blockIdx.x * ld + c0) * EB;
    int iss_g = 0, iss_st = 0;
    int64_t issued = 0;
    auto issue_next = [&]() {
        if (lane == 0) {
            const int nv = nfull - iss_g * kGroupUnits;
            const uint32_t bytes = nv <= 0 ? 0u : (uint32_t)((nv < kGroupUnits ? nv : kGroupUnits) * UB);
            const uint32_t bar = bar0 + iss_st * 8;
            mbar_arrive_expect_tx(bar, bytes);
            if (bytes) bulk_g2s(stage0 + iss_st * SB, iss_row + (int64_t)iss_g * SB, bytes, bar);
        }
        if (++iss_g == G) {
            iss_g = 0;
            iss_row += row_step;
        }
        if (++iss_st == kStages) iss_st = 0;
        ++issued;
    };

    bool ok = true;
    int64_t fail_at = -1;
    while (issued < kStages && issued < jobs) issue_next();

    int st = 0;          // stage of the next group to consume
    uint32_t phase = 0;  // its mbarrier parity
    for (int64_t j = 0; j < rows; ++j) {
        const int64_t t = (int64_t)blockIdx.x + j * gridDim.x;
        const int folder = (int)(j % kTiles);
        const char* xr = reinterpret_cast<const char*>(x) + t * ld * EB;
        bool act = false;
        float x_y = 0.f;
        if (warp == folder && lane == 0) {
            const int64_t yt = __ldg(y + t);
            act = row_active(mask, t, yt, v, ignore_index);
            if (act) x_y = elem_value<D>(xr, yt);
        }
        const char* tile = xr + c0 * EB;
        float m = -INFINITY, s = 0.f;
        for (int g = 0; g < G; ++g) {
            if (ok) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar0 + st * 8, phase, kWaitLimitCycles));
                if (!ok) fail_at = j * G + g;
            }
            const uint32_t sbase = stage0 + st * SB + lane * UB;
            Unit<D> q[kGroup];
            if (g < Gfull) {
#pragma unroll
                for (int u = 0; u < kGroup; ++u) unit_load_shared<D>(sbase + u * (kWarp * UB), q[u]);
                __syncwarp();
                if (ok && issued < jobs) {
                    if (lane == 0) fence_proxy_async_smem();
                    issue_next();
                }
                group_update<D, true, kScaled>(q, kGroup, m, s, sc);
            } else {
                const int v0 = g * kGroupUnits;
                int nvalid = 0;
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    const int jv = v0 + kWarp * u + lane;
                    if (jv < nfull) {
                        unit_load_shared<D>(sbase + u * (kWarp * UB), q[u]);
                        nvalid = u + 1;
                    } else if (jv < nunit) {
                        unit_load<D, false>(tile, (int64_t)jv * 8, width, q[u]);
                        nvalid = u + 1;
                    } else {
                        unit_fill_neg_inf<D>(q[u]);
                    }
                }
                __syncwarp();
                if (ok && issued < jobs) {
                    if (lane == 0) fence_proxy_async_smem();
                    issue_next();
                }
                if (nvalid == kGroup) group_update<D, true, kScaled>(q, nvalid, m, s, sc);
                else group_update<D, false, kScaled>(q, nvalid, m, s, sc);
            }
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }
        const MS p = tile_partial<kScaled>(MS{m, s}, sc);
        if (lane == 0) {
            sh_m[j & 1][warp] = p.m;
            sh_s[j & 1][warp] = p.s;
        }
        __syncthreads();
        if (warp == folder) {
            const int k = lane & 15;
            const MS f = tile_fold16(MS{sh_m[j & 1][k], sh_s[j & 1][k]}, sc.s);
            if (lane == 0)
                finalize_row(f, act, x_y, sc.s, logp + t, lse + t, lse_lo ? lse_lo + t : nullptr);
        }
    }
    if (!ok) {
        if (lane == 0) atomicExch(&g_device_error, 1);
        // drain the copies issued but never waited for (at most kStages)
        for (int64_t k = fail_at; k < issued; ++k)
            (void)mbar_wait(bar0 + (int)(k % kStages) * 8, (uint32_t)((k / kStages) & 1), kWaitLimitCycles);
    }
}

// Shard partials: one CTA per row, warp w reduces the shard's local tile w
// (global tile tile0 + w) with the same tile_scan/warp_merge as the forward.
template <Dt D, bool kVec, bool kScaled>
__global__ void __launch_bounds__(kFwdThreads)
k_logp_partials(const void* __restrict__ xs, int64_t n, int64_t ld, int64_t real_width, int64_t W,
                int tile0, int64_t vocab_start, const int64_t* __restrict__ y, Scale sc,
                float* __restrict__ pm, float* __restrict__ ps, float* __restrict__ sel) {
    constexpr int EB = Unit<D>::kElemBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t t = blockIdx.x; t < n; t += gridDim.x) {
        const char* xr = reinterpret_cast<const char*>(xs) + t * ld * EB;
        if (threadIdx.x == 0) {
            const int64_t yt = __ldg(y + t);
            if (yt >= vocab_start && yt < vocab_start + real_width)
                sel[t] = elem_value<D>(xr, yt - vocab_start);
        }
        const int64_t c0 = (int64_t)warp * W;
        const int64_t width = real_width - c0 < W ? real_width - c0 : W;
        const MS p = tile_partial<kScaled>(tile_scan<D, kVec, kScaled>(xr + c0 * EB, width, lane, sc), sc);
        if (lane == 0) {
            pm[t * kTiles + tile0 + warp] = p.m;
            ps[t * kTiles + tile0 + warp] = p.s;
        }
    }
}

// Merge of tile partials: one half warp per row, the same tile_fold16 and
// finalize_row as the forward.  The partials may come from several ranks of
// a vocabulary-parallel group, gathered side by side: rank r's [n, 16] maxima,
// [n, 16] sums and [n] selected logits start rank_stride floats after rank
// r - 1's, and tile k is read from rank (tile_rank >> 4k) & 15, the rank that
// reduced it; the selected logit of row t from the rank owning the tile of
// its target, y_t / W.  On one GPU (all shards writing one buffer) the stride
// and the table are 0.  Only transport differs, so the bits are the same.
__global__ void __launch_bounds__(256)
k_logp_merge(const float* __restrict__ pm, const float* __restrict__ ps,
             const float* __restrict__ sel, const int64_t* __restrict__ y, int64_t ignore_index,
             const uint8_t* __restrict__ mask, int64_t n, int64_t v, int n_tiles, float s,
             float* __restrict__ logp, float* __restrict__ lse, float* __restrict__ lse_lo,
             int64_t rank_stride, uint64_t tile_rank, int64_t W) {
    const int lane = threadIdx.x & 31, k = lane & 15;
    const int64_t warp_g = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t n_warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t my_off = (int64_t)((tile_rank >> (4 * k)) & 15u) * rank_stride;
    for (int64_t pair = warp_g; 2 * pair < n; pair += n_warps) {
        const int64_t t = 2 * pair + (lane >> 4);
        const bool valid = t < n;
        MS p{-INFINITY, 0.f};
        if (valid && k < n_tiles) {
            p.m = __ldg(pm + my_off + t * kTiles + k);
            p.s = __ldg(ps + my_off + t * kTiles + k);
        }
        const MS f = tile_fold16(p, s);
        if (valid && k == 0) {
            const int64_t yt = __ldg(y + t);
            const bool act = row_active(mask, t, yt, v, ignore_index);
            const int64_t owner = act ? (int64_t)((tile_rank >> (4 * (int)(yt / W))) & 15u) : 0;
            const float x_y = act ? __ldg(sel + owner * rank_stride + t) : 0.f;
            finalize_row(f, act, x_y, s, logp + t, lse + t, lse_lo ? lse_lo + t : nullptr);
        }
    }
}

// ---------------------------------------------------------------- backward

// Backward: one CTA per (segment of kBwdSegCols columns, row), elementwise.
// Per active row: LSE = lse (+ lse_lo) is split as lse_r + delta with lse_r
// on a 2^-16 grid, so that t = s x - lse_r is exact for the bulk of BF16
// logits at s = 1 (one rounding otherwise); exp(t) = 2^a (1 + c) with
// a = t log2 e rounded and c = t - a ln 2 recovered by two fused multiply-adds
// against a two-float ln 2 (the rounding error of a, carried to first order);
// coef = -s g exp(-delta) folds s, g and delta in once per
// row, with the exp2 bias correction.  Logits below about (LSE - 200) / s are raised to that bound first (their
// exp is below e^-199, zero in binary32), which also keeps a -inf logit from
// producing inf - inf.  Rows of |LSE| from kBwdFarLse on, where the bound comes near LSE itself, are
// computed without it (bwd_unit_far).  The target column is s g (1 - p) = -s g expm1(s x - LSE),
// without cancellation.  Values below 2^-126 flush to zero.  Each thread loads
// its eight units before computing any, so eight (FP32: sixteen) 16-byte loads
// are in flight per thread.
//
// Vocabulary shards: the buffer holds global columns [y_off, y_off + v) of a
// v_total-column vocabulary (unsharded: y_off = 0, v_total = v).  A row is
// active by its global target (in [0, v_total)); the one-hot term lands on
// local column y_t - y_off only when that lies in [0, v).  Every element is
// computed from the same per-row constants as in the unsharded call, so the
// shards' outputs side by side are the unsharded gradient bit for bit.
struct LogpBwdArgs {
    const void* x;
    int64_t n, v, ld;
    const int64_t* y;
    int64_t ignore_index;
    const uint8_t* mask;
    float s, inv_s;
    const float *lse, *lse_lo, *g;
    void* dx;
    int64_t ld_out, y_off, v_total;
};

// This CTA's segment of a row of a large |LSE| l.
template <Dt D, bool kVecIn, bool kVecOut, bool kInPlace>
__device__ __forceinline__ void logp_bwd_far_row(const LogpBwdArgs& a, int64_t t, int64_t yt, float l) {
    constexpr int EB = Unit<D>::kElemBytes;
    const float lo = __fadd_rn(__fsub_rn(l, l), a.lse_lo ? __ldg(a.lse_lo + t) : 0.f), gs = __fmul_rn(a.s, __ldg(a.g + t));
    const char* xr = static_cast<const char*>(a.x) + t * a.ld * EB;
    char* dr = static_cast<char*>(a.dx) + t * a.ld_out * EB;
    const int64_t col0 = (int64_t)blockIdx.x * kBwdSegCols + (int64_t)threadIdx.x * 8;
#pragma unroll 1
    for (int u = 0; u < kBwdUnitsPerThread; ++u) {
        const int64_t c = col0 + (int64_t)u * kBwdThreads * 8;
        if (c >= a.v) break;
        Unit<D> w;
        uint32_t o[Unit<D>::kWords];
        bwd_load<D, kVecIn, kInPlace>(xr, c, a.v, w);
        bwd_unit_far<D>(w, a.s, gs, l, lo, yt - a.y_off - c, o);
        bwd_store<D, kVecOut>(dr, c, a.v, o);
    }
}
// Of all its rows, those of a large |LSE|.
template <Dt D, bool kVecIn, bool kVecOut, bool kInPlace>
__device__ __noinline__ void logp_bwd_far_rows(const LogpBwdArgs& a) {
#pragma unroll 1
    for (int64_t t = blockIdx.y; t < a.n; t += gridDim.y) {
        const int64_t yt = __ldg(a.y + t);
        const float l = __ldg(a.lse + t);
        if (row_active(a.mask, t, yt, a.v_total, a.ignore_index) && bwd_far(l))
            logp_bwd_far_row<D, kVecIn, kVecOut, kInPlace>(a, t, yt, l);
    }
}

template <Dt D, bool kVecIn, bool kVecOut, bool kInPlace>
__global__ void __launch_bounds__(kBwdThreads, kBwdMinBlocks<D>)
k_logp_bwd(const __grid_constant__ LogpBwdArgs a) {
    constexpr int EB = Unit<D>::kElemBytes;
    constexpr int NW = Unit<D>::kWords;
    const int64_t v = a.v;
    // grid: x = segment of the row, y = row (strided when n > gridDim.y)
    const int64_t col0 = (int64_t)blockIdx.x * kBwdSegCols + (int64_t)threadIdx.x * 8;
    // Rows of a large |LSE|: where rows are vectors their code in the loop costs nothing, element by element
    // it does (2048 x 32003 FP16 in place 172 us, 166 by a call behind the loop; the call costs vectors 1%).
    constexpr bool kFarInLoop = kVecIn && kVecOut;
    bool far = false;
#pragma unroll 1
    for (int64_t t = blockIdx.y; t < a.n; t += gridDim.y) {
        const char* xr = static_cast<const char*>(a.x) + t * a.ld * EB;
        char* dr = static_cast<char*>(a.dx) + t * a.ld_out * EB;
        const int64_t yt = __ldg(a.y + t);
        const float l = __ldg(a.lse + t);
        const int64_t cs = (int64_t)kBwdThreads * 8;
        if (!row_active(a.mask, t, yt, a.v_total, a.ignore_index)) {
            uint32_t z[NW];
#pragma unroll
            for (int k = 0; k < NW; ++k) z[k] = 0u;
#pragma unroll
            for (int u = 0; u < kBwdUnitsPerThread; ++u)
                if (col0 + u * cs < v) bwd_store<D, kVecOut>(dr, col0 + u * cs, v, z);
            continue;
        }
        auto leave = [&] {   // a row of a large |LSE|
            if constexpr (kFarInLoop) logp_bwd_far_row<D, kVecIn, kVecOut, kInPlace>(a, t, yt, l);
            else far = true;
        };
        // asked behind the loads, which then do not wait for l (8192 x 151936 BF16 735 us, 738 before them); in
        // place that costs registers (720, 711 before them)
        if (kInPlace && bwd_far(l)) {
            leave();
            continue;
        }
        BwdRow r;
        const float l_lo = a.lse_lo ? __ldg(a.lse_lo + t) : 0.f;
        r.s = a.s;
        r.gs = __fmul_rn(a.s, __ldg(a.g + t));
        r.lr = __fmul_rn(rintf(__fmul_rn(l, 65536.f)), 1.f / 65536.f);
        r.delta = __fadd_rn(__fsub_rn(l, r.lr), l_lo);           // l - lr is exact
        // -s g e^-delta, times (1 + b) for the mean bias b of ex2.approx
        const float coef = __fmaf_rn(r.gs, __fsub_rn(bwd_rest(r.delta), kEx2BiasComp), -r.gs);
        const float fl = __fmul_rn(__fsub_rn(l, 200.f), a.inv_s);   // ~ (LSE - 200) / s
        r.floor_f = fl;
        r.floor_w = 0xff80ff80u;
        if constexpr (D == Dt::BF16) {
            const uint32_t b = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(fl));
            r.floor_w = b | (b << 16);
        }
        r.neg_lr = f2(-r.lr, -r.lr);
        r.s2 = f2(a.s, a.s);
        r.coef2 = f2(coef, coef);

        Unit<D> w[kBwdUnitsPerThread];
#pragma unroll
        for (int u = 0; u < kBwdUnitsPerThread; ++u)
            if (col0 + u * cs < v) bwd_load<D, kVecIn, kInPlace>(xr, col0 + u * cs, v, w[u]);
        if (!kInPlace && bwd_far(l)) {
            leave();
            continue;
        }
#pragma unroll
        for (int u = 0; u < kBwdUnitsPerThread; ++u) {
            if (col0 + u * cs < v) {
                uint32_t o[NW];
                bwd_unit<D>(w[u], r, yt - a.y_off - (col0 + u * cs), o);
                bwd_store<D, kVecOut>(dr, col0 + u * cs, v, o);
            }
        }
    }
    if constexpr (!kFarInLoop) {
        if (far) logp_bwd_far_rows<D, kVecIn, kVecOut, kInPlace>(a);
    }
}

// Mean relative error of ex2.approx.ftz.f32 against the double exp2 over a
// fixed grid of 2^20 arguments in [-24, 0) (one CTA; fixed reduction order).
__device__ double g_ex2_bias;
__global__ void __launch_bounds__(1024) k_ex2_bias_selftest() {
    __shared__ double sh[32];
    double acc = 0.0;
    for (int i = threadIdx.x; i < (1 << 20); i += 1024) {
        const float a = -24.0f * (float)i / (float)(1 << 20) - 1.0e-6f * (float)(i & 1023);
        const double ref = exp2((double)a);
        acc += ((double)ex2_ftz(a) - ref) / ref;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < 32; ++w) t += sh[w];
        g_ex2_bias = t / (double)(1 << 20);
    }
}

// Result word of the bounded-wait self-test.
__device__ int g_selftest_result;

// Self-test of the bounded wait: one thread waits on an mbarrier that nothing
// arrives on, with a short cycle limit, and records whether the wait gave up.
__global__ void k_wait_timeout_selftest(long long limit) {
    __shared__ __align__(8) uint64_t bar;
    const uint32_t b = smem_u32(&bar);
    mbar_init(b, 1);
    fence_mbar_init();
    const bool done = mbar_wait(b, 0, limit);
    g_selftest_result = done ? 0 : 1;
    if (!done) atomicExch(&g_device_error, 1);
}

}  // namespace flp
