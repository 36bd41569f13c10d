// Units of a row by dtype, the online (max, sumexp) of a lane over a vocabulary
// tile, its fixed merges, the end of a row, and a unit's gradient: what the
// log-probability kernels share.  The method and the order of its sums are described in logp_kernels.cuh.
#pragma once

#include "logp_prims.cuh"

namespace flp {

enum class Dt : int { BF16 = 0, F16 = 1, F32 = 2 };

constexpr int kTiles = 16;                   // vocabulary tiles per row (K)
constexpr int kWarp = 32;
constexpr int kFwdThreads = kTiles * kWarp;  // one warp per tile
constexpr int kGroup = 4;                    // units per lane per online step
constexpr int kGroupUnits = kWarp * kGroup;  // units of a tile per group (128)
constexpr int kStages = 3;                   // bulk-copy ring depth per warp
constexpr int kBwdThreads = 128;
constexpr int kBwdUnitsPerThread = 8;
constexpr int64_t kBwdSegCols = (int64_t)kBwdThreads * kBwdUnitsPerThread * 8;
// Bounded waits give up after this many SM cycles (about 2 s at 2 GHz).
constexpr long long kWaitLimitCycles = 4000000000LL;

// Mathematical constants: ln 2 to double precision, its binary32 head and
// tail (head + tail = ln 2 to about 2^-48 relative), and log2(e) rounded to
// binary32.
constexpr double kLn2 = 0.6931471805599453094172321214581766;
constexpr float kLn2Hi = (float)kLn2;
constexpr float kLn2Lo = (float)(kLn2 - (double)kLn2Hi);
constexpr float kLog2e = (float)(1.0 / kLn2);

// Mean relative error of ex2.approx.ftz.f32 on this GPU family: -4.95e-8
// (measured over 4M arguments in [-24, 0]; flat in the argument; re-measured
// by flp_selftest_ex2_bias).  Every tile sum is built from such terms, so it
// is scaled by (1 + kEx2BiasComp) once, in tile_partial.
constexpr float kEx2BiasComp = 4.95e-8f;

struct MS {
    float m;  // running maximum of the raw logits (an input element, or -inf)
    float s;  // sum of exp(s (x - m)) over the elements seen
};

// Inverse temperature s and s log2(e) as a two-float (hi + lo).
struct Scale {
    float s, hi, lo;
};

// ---------------------------------------------------------------- units by dtype

template <Dt D>
struct Unit {
    static constexpr int kWords = (D == Dt::F32) ? 8 : 4;
    static constexpr int kBytes = kWords * 4;
    static constexpr int kElemBytes = (D == Dt::F32) ? 4 : 2;
    static constexpr uint32_t kNegInfBits = (D == Dt::BF16) ? 0xff80u : (D == Dt::F16) ? 0xfc00u : 0xff800000u;
    uint32_t w[kWords];
};

template <Dt D>
constexpr int kStageBytes = kGroupUnits * Unit<D>::kBytes;
template <Dt D>
constexpr int kFwdSmemBytes = kTiles * kStages * kStageBytes<D> + kTiles * kStages * 8;
template <Dt D>
constexpr int kFwdMinBlocks = (D == Dt::F32) ? 1 : 2;
// backward CTAs of 128 threads per SM: register caps 64 (16-bit) and 96 (FP32)
template <Dt D>
constexpr int kBwdMinBlocks = (D == Dt::F32) ? 5 : 8;

template <Dt D>
__device__ __forceinline__ uint32_t elem_bits(const void* base, int64_t i) {
    if constexpr (D == Dt::F32) return __ldg(reinterpret_cast<const unsigned int*>(base) + i);
    else return (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(base) + i);
}
template <Dt D>
__device__ __forceinline__ uint32_t elem_bits_plain(const void* base, int64_t i) {
    if constexpr (D == Dt::F32) return reinterpret_cast<const unsigned int*>(base)[i];
    else return (uint32_t)reinterpret_cast<const unsigned short*>(base)[i];
}
template <Dt D>
__device__ __forceinline__ float bits_value(uint32_t b) {
    if constexpr (D == Dt::BF16) return __uint_as_float(b << 16);
    else if constexpr (D == Dt::F16) return __half2float(__ushort_as_half((unsigned short)b));
    else return __uint_as_float(b);
}
template <Dt D>
__device__ __forceinline__ float elem_value(const void* base, int64_t i) {
    return bits_value<D>(elem_bits<D>(base, i));
}

template <Dt D>
__device__ __forceinline__ void unit_fill_neg_inf(Unit<D>& u) {
    constexpr uint32_t w = (D == Dt::F32) ? Unit<D>::kNegInfBits : (Unit<D>::kNegInfBits * 0x10001u);
#pragma unroll
    for (int k = 0; k < Unit<D>::kWords; ++k) u.w[k] = w;
}

// The unit of the 8 columns [col, col + 8) of a tile; columns >= width read
// as -inf (padded columns are masked, PR #314 ReductionSpec).  The vector path
// needs a 16-byte aligned tile; both paths give the same words.
template <Dt D, bool kVec>
__device__ __forceinline__ void unit_load(const void* __restrict__ tile, int64_t col, int64_t width,
                                          Unit<D>& u) {
    constexpr uint32_t NI = Unit<D>::kNegInfBits;
    if (kVec && col + 8 <= width) {
        const char* p = reinterpret_cast<const char*>(tile) + col * Unit<D>::kElemBytes;
        const uint4 a = ld_nc_v4(p);
        u.w[0] = a.x; u.w[1] = a.y; u.w[2] = a.z; u.w[3] = a.w;
        if constexpr (D == Dt::F32) {
            const uint4 b = ld_nc_v4(p + 16);
            u.w[4] = b.x; u.w[5] = b.y; u.w[6] = b.z; u.w[7] = b.w;
        }
    } else if constexpr (D == Dt::F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u.w[j] = (col + j < width) ? elem_bits<D>(tile, col + j) : NI;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = (col + 2 * k < width) ? elem_bits<D>(tile, col + 2 * k) : NI;
            const uint32_t hi = (col + 2 * k + 1 < width) ? elem_bits<D>(tile, col + 2 * k + 1) : NI;
            u.w[k] = lo | (hi << 16);
        }
    }
}

template <Dt D>
__device__ __forceinline__ void unit_load_shared(uint32_t addr, Unit<D>& u) {
    const uint4 a = lds_v4(addr);
    u.w[0] = a.x; u.w[1] = a.y; u.w[2] = a.z; u.w[3] = a.w;
    if constexpr (D == Dt::F32) {
        const uint4 b = lds_v4(addr + 16);
        u.w[4] = b.x; u.w[5] = b.y; u.w[6] = b.z; u.w[7] = b.w;
    }
}

// max(m, all elements of the group's units), by packed 16-bit maxima.
template <Dt D>
__device__ __forceinline__ float group_max(const Unit<D> (&q)[kGroup], float m) {
    if constexpr (D == Dt::F32) {
        float r = m;
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) r = fmaxf(r, __uint_as_float(q[u].w[j]));
        return r;
    } else {
        auto mx = [](uint32_t a, uint32_t b) { return D == Dt::BF16 ? bf2_max(a, b) : h2_max(a, b); };
        uint32_t w = mx(mx(q[0].w[0], q[0].w[1]), mx(q[0].w[2], q[0].w[3]));
#pragma unroll
        for (int u = 1; u < kGroup; ++u) w = mx(w, mx(mx(q[u].w[0], q[u].w[1]), mx(q[u].w[2], q[u].w[3])));
        const float lo = (D == Dt::BF16) ? bf_lo(w) : h_lo(w);
        const float hi = (D == Dt::BF16) ? bf_hi(w) : h_hi(w);
        return fmaxf(m, fmaxf(lo, hi));
    }
}

// (x_{2k} - b, x_{2k+1} - b) of a unit, each rounded once.
template <Dt D>
__device__ __forceinline__ u64 pair_sub(const Unit<D>& u, int k, float b) {
    if constexpr (D == Dt::BF16) return bf2_sub(u.w[k], b);
    else if constexpr (D == Dt::F16) return h2_sub(u.w[k], b);
    else return f2_add(f2(__uint_as_float(u.w[2 * k]), __uint_as_float(u.w[2 * k + 1])), f2(-b, -b));
}

// t log2(e) s: one product when s = 1, else against the two-float s log2(e).
template <bool kScaled>
__device__ __forceinline__ u64 to_log2(u64 t, const Scale& sc) {
    if constexpr (kScaled) return f2_fma(t, f2(sc.hi, sc.hi), f2_mul(t, f2(sc.lo, sc.lo)));
    else return f2_mul(t, f2(kLog2e, kLog2e));
}
template <bool kScaled>
__device__ __forceinline__ float to_log2_1(float t, const Scale& sc) {
    if constexpr (kScaled) return __fmaf_rn(t, sc.hi, __fmul_rn(t, sc.lo));
    else return __fmul_rn(t, kLog2e);
}

// ---------------------------------------------------------------- forward reduction

// One online step of a lane over kGroup units (with kFull all hold data,
// otherwise units [0, nvalid) do and the others are -inf).  Maxima are kept in
// units of the raw logits x; the scale enters only the exponent:
// gm = max(m, elements); each element's term 2^((x - gm) s log2 e) on the
// special-function unit (x - gm is exact for 16-bit inputs); the terms summed
// by a fixed pairwise tree (element pairs ((p0 + p1) + (p2 + p3)) lane-wise,
// units ((u0 + u1) + (u2 + u3)), then the even and odd lanes);
// s_acc = s_acc * exp(s (m - gm)) + group sum.
template <Dt D, bool kFull, bool kScaled>
__device__ __forceinline__ void group_update(const Unit<D> (&q)[kGroup], int nvalid, float& m,
                                             float& s, const Scale& sc) {
    const float gm = group_max<D>(q, m);
    if (gm == -INFINITY) return;  // nothing finite seen yet: (m, s) stays (-inf, 0)
    u64 vsum[kGroup];
#pragma unroll
    for (int u = 0; u < kGroup; ++u) {
        if (kFull || u < nvalid) {
            u64 p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float a0, a1;
                f2_split(to_log2<kScaled>(pair_sub<D>(q[u], k, gm), sc), a0, a1);
                p[k] = f2(ex2_ftz(a0), ex2_ftz(a1));
            }
            vsum[u] = f2_add(f2_add(p[0], p[1]), f2_add(p[2], p[3]));
        } else {
            vsum[u] = 0ull;
        }
    }
    static_assert(kGroup == 4, "the group tree is written for four units");
    float e, o;
    f2_split(f2_add(f2_add(vsum[0], vsum[1]), f2_add(vsum[2], vsum[3])), e, o);
    const float gs = __fadd_rn(e, o);
    const float r = (m == gm) ? 1.f : ex2_ftz(to_log2_1<kScaled>(__fsub_rn(m, gm), sc));
    s = __fmaf_rn(s, r, gs);
    m = gm;
}

// Online (max, sumexp) of one lane over a tile of `width` columns with plain
// loads: unit j of the tile belongs to lane j mod 32, visited in increasing j,
// kGroup at a time (units v0 + 32u + lane of group v0 / 128).  The bulk-copy
// forward feeds group_update with the same words in the same order.
template <Dt D, bool kVec, bool kScaled>
__device__ __forceinline__ MS tile_scan(const void* __restrict__ tile, int64_t width, int lane,
                                        const Scale& sc) {
    const int64_t nunit = (width + 7) >> 3;
    float m = -INFINITY, s = 0.f;
    for (int64_t v0 = 0; v0 < nunit; v0 += kGroupUnits) {
        Unit<D> q[kGroup];
        int nvalid = 0;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            const int64_t j = v0 + (int64_t)kWarp * u + lane;
            if (j < nunit) {
                unit_load<D, kVec>(tile, j * 8, width, q[u]);
                nvalid = u + 1;
            } else {
                unit_fill_neg_inf<D>(q[u]);
            }
        }
        if (nvalid == kGroup) group_update<D, true, kScaled>(q, nvalid, m, s, sc);
        else group_update<D, false, kScaled>(q, nvalid, m, s, sc);
    }
    return MS{m, s};
}

// Merge of two (max, sumexp) pairs: the pair holding the larger max keeps its
// sum, the other is scaled by exp(s (m_small - M)).  Symmetric in its
// arguments (IEEE addition commutes), so both lanes of a butterfly get the
// same bits.
template <bool kScaled>
__device__ __forceinline__ MS ms_merge(MS a, MS b, const Scale& sc) {
    const bool a_big = a.m >= b.m;
    const float M = a_big ? a.m : b.m;
    const float m_small = a_big ? b.m : a.m;
    const float s_big = a_big ? a.s : b.s;
    const float s_small = a_big ? b.s : a.s;
    float r;
    if (m_small == -INFINITY) r = 0.f;
    else if (m_small == M) r = 1.f;
    else r = ex2_ftz(to_log2_1<kScaled>(__fsub_rn(m_small, M), sc));
    return MS{M, __fmaf_rn(s_small, r, s_big)};
}

// Fixed xor butterfly over the 32 lanes of a warp (offsets 16, 8, 4, 2, 1);
// every lane ends with the same pair.
template <bool kScaled>
__device__ __forceinline__ MS warp_merge(MS p, const Scale& sc) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        MS o;
        o.m = __shfl_xor_sync(0xffffffffu, p.m, off);
        o.s = __shfl_xor_sync(0xffffffffu, p.s, off);
        p = ms_merge<kScaled>(p, o, sc);
    }
    return p;
}

// The partial of a whole tile: the warp butterfly of the lane pairs, with the
// sum corrected for the mean bias of the special-function unit's exp2 (one
// fused multiply-add).  Every path (forward, plain forward, shard partials)
// forms tile partials here, so they stay bitwise equal.
template <bool kScaled>
__device__ __forceinline__ MS tile_partial(MS lane_pair, const Scale& sc) {
    MS p = warp_merge<kScaled>(lane_pair, sc);
    p.s = __fmaf_rn(p.s, kEx2BiasComp, p.s);
    return p;
}

// Merge of the 16 tile partials of one row held by a 16-lane half warp
// (lane k of the half holds tile k; tiles beyond the vocabulary hold the
// identity (-inf, 0)).  M = max m_k; S = sum_k s_k exp(s (m_k - M)) summed as
// a fixed pairwise tree in tile-index order (issue #241 PR 3 merge formula).
// m_k - M is exact for 16-bit inputs; exp is the accurate library expf.  All
// 32 lanes call this together; every lane gets (M, S) of its half.
__device__ __forceinline__ MS tile_fold16(MS p, float s) {
    float M = p.m;
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off, 16));
    float term = (p.m == -INFINITY) ? 0.f : __fmul_rn(p.s, expf(__fmul_rn(s, __fsub_rn(p.m, M))));
#pragma unroll
    for (int off = 1; off <= 8; off <<= 1)
        term = __fadd_rn(term, __shfl_xor_sync(0xffffffffu, term, off, 16));
    return MS{M, term};
}

// LSE = s M + log S and logp = s x_y - LSE, carried in double (s M and s x_y
// are exact there) and each output rounded once to binary32 (the "downcast at
// final write" of issue #241 Goal).  lse_lo, when given, receives the binary32
// rounding residual of the LSE (LSE - lse), so that lse + lse_lo carries the
// LSE to about 2^-48 relative for the backward.  From kLseFar on double has few
// digits left for log S in s M + log S: there it is added last.
constexpr float kLseFar = 134217728.f;   // 2^27
__device__ __forceinline__ void finalize_row(MS f, bool active, float x_y, float s, float* logp_out,
                                             float* lse_out, float* lse_lo_out) {
    const double log_s = log((double)f.s);
    const double l = (f.m == -INFINITY) ? -(double)INFINITY : (double)s * (double)f.m + log_s;
    const float lf = __double2float_rn(l);
    *lse_out = lf;
    if (fabsf(__fmul_rn(s, f.m)) >= kLseFar && isfinite(f.m)) {   // known before the FP64 above
        const double top = (double)s * (double)f.m;
        if (lse_lo_out) *lse_lo_out = isfinite(lf) ? __double2float_rn((top - (double)lf) + log_s) : 0.f;
        *logp_out = active ? __double2float_rn(((double)s * (double)x_y - top) - log_s) : 0.f;
        return;
    }
    if (lse_lo_out) *lse_lo_out = isfinite(lf) ? __double2float_rn(l - (double)lf) : 0.f;
    *logp_out = active ? __double2float_rn((double)s * (double)x_y - l) : 0.f;
}

__device__ __forceinline__ bool row_active(const uint8_t* mask, int64_t t, int64_t y, int64_t v,
                                           int64_t ignore_index) {
    return (mask == nullptr || __ldg(mask + t) != 0) && y >= 0 && y < v && y != ignore_index;
}

// ---------------------------------------------------------------- backward

// Per-row constants of the backward (see k_logp_bwd).
struct BwdRow {
    u64 neg_lr;        // (-lse_r, -lse_r)
    u64 s2;            // (s, s)
    u64 coef2;         // (coef, coef), coef = -s g (1 - delta)
    uint32_t floor_w;  // BF16: packed floor for the raw logits
    float floor_f;     // FP16/FP32: floor for the raw logits
    float lr, delta, gs, s;
};

// 1 - e^-delta for what the rounded LSE leaves (LSE = lr + delta): delta itself, of which the square is
// below a rounding, up to 2^-11.  From |LSE| = 2^13 on it may be more, 2^-6 at 2^18: three terms of the
// series (the next is below 2^-28).
__device__ __forceinline__ float bwd_rest(float delta) {
    const float more = __fmul_rn(delta, __fmaf_rn(delta, __fmaf_rn(delta, 1.f / 6.f, -0.5f), 1.f));
    return fabsf(delta) < 0x1p-11f ? delta : more;
}

// The pair (x_{2k}, x_{2k+1}) of a unit widened to binary32 and raised to the
// row's floor.
template <Dt D>
__device__ __forceinline__ u64 bwd_pair(const Unit<D>& u, int k, const BwdRow& r) {
    if constexpr (D == Dt::BF16) {
        const uint32_t w = bf2_max(u.w[k], r.floor_w);
        return f2(bf_lo(w), bf_hi(w));
    } else if constexpr (D == Dt::F16) {
        return f2(fmaxf(h_lo(u.w[k]), r.floor_f), fmaxf(h_hi(u.w[k]), r.floor_f));
    } else {
        return f2(fmaxf(__uint_as_float(u.w[2 * k]), r.floor_f),
                  fmaxf(__uint_as_float(u.w[2 * k + 1]), r.floor_f));
    }
}

// Output word(s) of a gradient pair in dtype D (for FP32 two words).
template <Dt D>
__device__ __forceinline__ void put_pair(uint32_t (&o)[Unit<D>::kWords], int k, float d0, float d1) {
    if constexpr (D == Dt::BF16) o[k] = pack_bf16x2(d0, d1);
    else if constexpr (D == Dt::F16) o[k] = pack_f16x2(d0, d1);
    else {
        o[2 * k] = __float_as_uint(d0);
        o[2 * k + 1] = __float_as_uint(d1);
    }
}

// Gradient of one unit (8 columns) into output words o, target column jt (or
// outside [0, 8)).
template <Dt D>
__device__ __forceinline__ void bwd_unit(const Unit<D>& u, const BwdRow& r, int64_t jt,
                                         uint32_t (&o)[Unit<D>::kWords]) {
    const u64 l2e = f2(kLog2e, kLog2e);
    const u64 nln2hi = f2(-kLn2Hi, -kLn2Hi), nln2lo = f2(-kLn2Lo, -kLn2Lo);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const u64 tt = f2_fma(bwd_pair<D>(u, k, r), r.s2, r.neg_lr);
        const u64 a = f2_mul(tt, l2e);
        const u64 c = f2_fma(a, nln2lo, f2_fma(a, nln2hi, tt));
        float a0, a1;
        f2_split(a, a0, a1);
        const u64 q = f2_mul(f2(ex2_ftz(a0), ex2_ftz(a1)), r.coef2);
        float d0, d1;
        f2_split(f2_fma(q, c, q), d0, d1);
        put_pair<D>(o, k, d0, d1);
    }
    if (jt >= 0 && jt < 8) {
        // target column: s g (1 - p) without cancellation, patched into its word
        // (the element is picked by unrolled selects: no run-time index)
        const int kt = (int)(jt >> 1);
        float xt = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            f2_split(bwd_pair<D>(u, k, r), lo, hi);
            if (k == kt) xt = (jt & 1) ? hi : lo;
        }
        const float dt = __fmul_rn(-r.gs, expm1f(__fsub_rn(__fmaf_rn(r.s, xt, -r.lr), r.delta)));
        if constexpr (D == Dt::F32) {
            // blend by masks (a predicated store per word would be folded into
            // one store at a run-time index, which needs local memory)
            const uint32_t bits = __float_as_uint(dt);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t msk = 0u - (uint32_t)(j == (int)jt);
                o[j] = (o[j] & ~msk) | (bits & msk);
            }
        } else {
            const uint32_t bt = ((D == Dt::BF16) ? pack_bf16x2(dt, dt) : pack_f16x2(dt, dt)) & 0xffffu;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k == kt) o[k] = (jt & 1) ? ((o[k] & 0xffffu) | (bt << 16)) : ((o[k] & 0xffff0000u) | bt);
        }
    }
}

// A row of a large |LSE|, beside which a floor may be LSE itself (or of one that is not finite).
constexpr float kBwdFarLse = 262144.f;
__device__ __forceinline__ bool bwd_far(float l) { return !(fabsf(l) < kBwdFarLse); }
// Gradient of a unit in such a row: the logits as they are, p = e^lp with lp = (s x - l) - lo, not below
// -200, where p is 0.  lo: the rounding residual of l = LSE, NaN where that is not finite.
template <Dt D>
__device__ __forceinline__ void bwd_unit_far(const Unit<D>& u, float s, float gs, float l, float lo, int64_t jt,
                                             uint32_t (&o)[Unit<D>::kWords]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x[2], d[2];
        if constexpr (D == Dt::F32) {
            x[0] = __uint_as_float(u.w[2 * k]);
            x[1] = __uint_as_float(u.w[2 * k + 1]);
        } else {
            x[0] = D == Dt::BF16 ? bf_lo(u.w[k]) : h_lo(u.w[k]);
            x[1] = D == Dt::BF16 ? bf_hi(u.w[k]) : h_hi(u.w[k]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float lp = __fsub_rn(__fmaf_rn(s, x[e], -l), lo);
            lp = lp < -200.f ? -200.f : lp;   // a NaN stays
            d[e] = __fmul_rn(-gs, 2 * k + e == jt ? expm1f(lp) : expf(lp));
        }
        put_pair<D>(o, k, d[0], d[1]);
    }
}

template <Dt D, bool kVecIn, bool kInPlace>
__device__ __forceinline__ void bwd_load(const char* xr, int64_t col, int64_t v, Unit<D>& u) {
    constexpr int EB = Unit<D>::kElemBytes;
    if (kVecIn && col + 8 <= v) {
        const char* p = xr + col * EB;
        const uint4 a = kInPlace ? ld_v4(p) : ld_nc_v4(p);
        u.w[0] = a.x; u.w[1] = a.y; u.w[2] = a.z; u.w[3] = a.w;
        if constexpr (D == Dt::F32) {
            const uint4 b = kInPlace ? ld_v4(p + 16) : ld_nc_v4(p + 16);
            u.w[4] = b.x; u.w[5] = b.y; u.w[6] = b.z; u.w[7] = b.w;
        }
    } else if constexpr (D == Dt::F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            u.w[j] = (col + j < v) ? (kInPlace ? elem_bits_plain<D>(xr, col + j) : elem_bits<D>(xr, col + j)) : 0u;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t lo = 0, hi = 0;
            if (col + 2 * k < v)
                lo = kInPlace ? elem_bits_plain<D>(xr, col + 2 * k) : elem_bits<D>(xr, col + 2 * k);
            if (col + 2 * k + 1 < v)
                hi = kInPlace ? elem_bits_plain<D>(xr, col + 2 * k + 1) : elem_bits<D>(xr, col + 2 * k + 1);
            u.w[k] = lo | (hi << 16);
        }
    }
}

template <Dt D, bool kVecOut>
__device__ __forceinline__ void bwd_store(char* dr, int64_t col, int64_t v,
                                          const uint32_t (&o)[Unit<D>::kWords]) {
    constexpr int EB = Unit<D>::kElemBytes;
    if (kVecOut && col + 8 <= v) {
        st_cs_v4(dr + col * EB, make_uint4(o[0], o[1], o[2], o[3]));
        if constexpr (D == Dt::F32) st_cs_v4(dr + col * EB + 16, make_uint4(o[4], o[5], o[6], o[7]));
    } else if constexpr (D == Dt::F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < v) reinterpret_cast<uint32_t*>(dr)[col + j] = o[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < v)
                reinterpret_cast<uint16_t*>(dr)[col + j] =
                    (uint16_t)((j & 1) ? (o[j >> 1] >> 16) : (o[j >> 1] & 0xffffu));
    }
}

}  // namespace flp
