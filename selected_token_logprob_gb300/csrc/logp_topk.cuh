// Selected-token log-probability with entropy and the k best alternatives, and the
// gradient of all three, for sm_103a.
//
// Per row, with z = s x (s the inverse temperature), M = max z:
//   S = sum e^(z - M), T = sum e^(z - M) (z - M),
//   LSE = M + log S, logp = z_y - LSE, H = log S - T / S
// (both terms of the entropy H are >= 0: nothing cancels), and the k largest logits,
// of equal ones the lowest column first.  The tiles, the online sums and their merges are
// those of the plain forward (logp_kernels.cuh), of 1 to 16 tiles a row, but a term's exponent is one fused
// multiply-add, x c - m c with c = s log2 e: what rounding m c loses is the same for a lane's
// group and is given back to the group's sums.  (With the plain forward's difference and
// two-float product a logit took 12.3 instructions, and the issue slots, not memory, were
// the bound: 2048 x 151936 136 us, 107 so, of which 93 is memory.)  T is a second sum beside S, in units of
// log 2, and moved along when the running maximum grows:
//   T <- 2^d (T + d S) for a shift of the maximum by d (log2 units).
//
// The forward is two kernels.  k_logp_topk_scan reads the logits once: per warp one
// vocabulary tile of a row, giving the tile's (M, S, T) and, per lane and run of
// `per` groups, the largest logit (a "slot" of 32 per elements; the group's maximum is
// taken for the online sum anyway).  k_logp_topk_finish, a warp per row, merges the
// tiles and finds the top k: an element of the top k lies in a slot whose maximum is one
// of the k largest, so that about k slots (a few KB, still in L2) are read again and
// the rest of the row is not.
//
// Backward, elementwise as the plain one: with p = e^logp, G = g + sum of the
// alternatives' upstream gradients,
//   dx = s (g 1_y + sum_j gt_j 1_idj - p (G + gh (logp + H))).
//
// What bounds them: memory.
#pragma once

#include "logp_units.cuh"

namespace flp {

// Sticky error word of the waits on bulk copies here (1 = one ran out).
static __device__ int g_topk_error;

// Units of a lane in one online step, 64 values of 16 bits or 32 of FP32 (4 KB a warp), and of the
// warp.  With half of that what a step costs beside its terms (the wait, the next copy, the
// maximum, the floor, the rescaling) was more than a third of all instructions.
template <Dt D>
constexpr int kTopkGroup = D == Dt::F32 ? 4 : 8;
template <Dt D>
constexpr int kTopkGroupUnits = kWarp * kTopkGroup<D>;
template <Dt D>
constexpr int kTopkStage = kTopkGroupUnits<D> * Unit<D>::kBytes;
constexpr int kTopkMax = 64;          // alternatives
constexpr int kTopkSlotRuns = 6;      // slots per lane and tile at most (u16 numbers, 24 KB of FP32 a row)
constexpr int kTopkFinishWarps = 8;
constexpr int kTopkList = 256;        // slots read again without the slow path
constexpr int kTopkCands = 512;       // elements compared with one another

struct TopkArgs {
    const void* x;
    int64_t n, v, ld, W;     // W: width of a tile, a multiple of 8
    int tiles;               // of a row: 1, 2, 4, 8 or 16
    const int64_t* y;        // null: no targets
    int64_t ignore_index;
    const uint8_t* mask;
    Scale sc;
    float far;               // 200 / s: a logit that far below the maximum adds nothing
    float4* parts;           // [n, tiles] (M, S, T, 0) of a tile
    void* slots;             // [n, runs, tiles, 32] largest logits, or null
    int per, runs;           // groups per slot, slots per lane and tile
};

struct TopkOut {
    float *logp, *lse, *lse_lo, *entropy;   // [n]; logp null without targets, lse_lo nullable
    int64_t* ids;                           // [n, k]
    float* top;                             // [n, k]
    int k;
    bool vec;                               // rows are 16-byte aligned
};

struct MST {
    float m, s, t;   // maximum of the raw logits, sum e^(s (x - m)), sum of the same times s (x - m) log2 e
};

__device__ __forceinline__ bool topk_active(const TopkArgs& a, int64_t t) {
    if (a.mask != nullptr && __ldg(a.mask + t) == 0) return false;
    if (a.y == nullptr) return true;
    const int64_t y = __ldg(a.y + t);
    return y >= 0 && y < a.v && y != a.ignore_index;
}

// Maxima that keep a NaN.
__device__ __forceinline__ uint32_t bf2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float f_max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
template <Dt D>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
    if constexpr (D == Dt::BF16) return bf2_max_nan(a, b);
    else if constexpr (D == Dt::F16) return h2_max_nan(a, b);
    else return __float_as_uint(f_max_nan(__uint_as_float(a), __uint_as_float(b)));
}
// The largest of a word's elements (16-bit: two).
template <Dt D>
__device__ __forceinline__ float word_value(uint32_t w) {
    if constexpr (D == Dt::BF16) return f_max_nan(bf_lo(w), bf_hi(w));
    else if constexpr (D == Dt::F16) return f_max_nan(h_lo(w), h_hi(w));
    else return __uint_as_float(w);
}
template <Dt D>
constexpr uint32_t kWordNegInf = (D == Dt::F32) ? Unit<D>::kNegInfBits : Unit<D>::kNegInfBits * 0x10001u;

// Whole numbers in the order of the values: -0 as +0, every NaN above +inf.
__device__ __forceinline__ uint32_t topk_key(float f) {
    const uint32_t b = __float_as_uint(__fadd_rn(f, 0.f));
    if (f != f) return 0xffffffffu;
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float topk_value(uint32_t key) {
    if (key == 0xffffffffu) return __uint_as_float(0x7fffffffu);
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;

// The unit's words raised to a floor (a packed word, or FP32) that lies at the type's lowest number or
// above it: -inf becomes a number, so that 0 times it is 0; terms that far below the maximum are 0
// either way.
template <Dt D>
constexpr float kTopkLowest = D == Dt::F16 ? -65504.f : D == Dt::BF16 ? -0x1.fep127f : -0x1.fffffep127f;
template <Dt D>
__device__ __forceinline__ uint32_t topk_floor(float fl) {
    if constexpr (D == Dt::F32) {
        return __float_as_uint(fl);
    } else {
        const uint32_t b = D == Dt::BF16 ? (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(fl))
                                         : (uint32_t)__half_as_ushort(__float2half_rd(fl));
        return b | (b << 16);
    }
}
template <Dt D>
__device__ __forceinline__ void topk_raise(Unit<D>& u, uint32_t fl) {
#pragma unroll
    for (int k = 0; k < Unit<D>::kWords; ++k) {
        if constexpr (D == Dt::BF16) u.w[k] = bf2_max_nan(u.w[k], fl);
        else if constexpr (D == Dt::F16) u.w[k] = h2_max_nan(u.w[k], fl);
        else u.w[k] = __float_as_uint(f_max_nan(__uint_as_float(u.w[k]), __uint_as_float(fl)));
    }
}

// The values 2 k and 2 k + 1 of a unit.
template <Dt D>
__device__ __forceinline__ u64 topk_pair(const Unit<D>& u, int k) {
    if constexpr (D == Dt::F32) return f2(__uint_as_float(u.w[2 * k]), __uint_as_float(u.w[2 * k + 1]));
    else if constexpr (D == Dt::BF16) return f2(bf_lo(u.w[k]), bf_hi(u.w[k]));
    else return f2(h_lo(u.w[k]), h_hi(u.w[k]));
}

// Sums of a group's terms 2^e and of 2^e e.  e = x c + g, of values raised to the floor; kDiff: (x - gm) c of
// the values themselves, then not below kTopkLeast, where a term is 0 (-inf must not meet it).
constexpr float kTopkLeast = -300.f;
template <Dt D, bool kFull, bool kDiff>
__device__ __forceinline__ void topk_sums(const Unit<D> (&q)[kTopkGroup<D>], int nvalid, float gm, float g, const Scale& sc,
                                          float& gs, float& gt) {
    constexpr int kN = kTopkGroup<D>;
    const u64 c2 = f2(sc.hi, sc.hi), g2 = f2(g, g);
    u64 vsum[kN], tsum[kN];
#pragma unroll
    for (int u = 0; u < kN; ++u) {
        if (kFull || u < nvalid) {
            u64 p[4], tt = 0ull;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                u64 e = kDiff ? to_log2<true>(pair_sub<D>(q[u], k, gm), sc) : f2_fma(topk_pair<D>(q[u], k), c2, g2);
                float a0, a1;
                f2_split(e, a0, a1);
                if constexpr (kDiff) {
                    a0 = f_max_nan(a0, kTopkLeast);
                    a1 = f_max_nan(a1, kTopkLeast);
                    e = f2(a0, a1);
                }
                p[k] = f2(ex2_ftz(a0), ex2_ftz(a1));
                tt = k == 0 ? f2_mul(p[k], e) : f2_fma(p[k], e, tt);
            }
            vsum[u] = f2_add(f2_add(p[0], p[1]), f2_add(p[2], p[3]));
            tsum[u] = tt;
        } else {
            vsum[u] = tsum[u] = 0ull;
        }
    }
#pragma unroll
    for (int d = kN / 2; d >= 1; d /= 2)
#pragma unroll
        for (int u = 0; u < d; ++u) {
            vsum[u] = f2_add(vsum[u], vsum[u + d]);
            tsum[u] = f2_add(tsum[u], tsum[u + d]);
        }
    float e, o;
    f2_split(vsum[0], e, o);
    gs = __fadd_rn(e, o);
    f2_split(tsum[0], e, o);
    gt = __fadd_rn(e, o);
}

// One online step of a lane over a group of kTopkGroup units (those from nvalid on are
// -inf unless kFull).  Returns the maximum of the group's elements, packed as they are.
//
// Terms are 2^(x c + g) with g = -(gm c) rounded; r, what the rounding lost, is the same for all of
// them: the group's sum is 2^r = 1 + r ln 2 of that (|r| <= 2^-12: the next term is below 2^-25), its
// T is moved by r.  Where |gm c| is larger, or the floor below the type's lowest number, the difference is
// taken first: next to a large maximum a floor would be the maximum itself, at the lowest number -inf
// would count as it does.
template <Dt D, bool kFull>
__device__ __forceinline__ uint32_t topk_update(Unit<D> (&q)[kTopkGroup<D>], int nvalid, MST& a, const Scale& sc, float far) {
    uint32_t w = q[0].w[0];
#pragma unroll
    for (int u = 0; u < kTopkGroup<D>; ++u)
#pragma unroll
        for (int k = 0; k < Unit<D>::kWords; ++k)
            if (u + k > 0) w = word_max<D>(w, q[u].w[k]);
    const float gm = f_max_nan(a.m, word_value<D>(w));
    if (gm == -INFINITY) return w;   // nothing finite seen yet: (m, s, t) stays (-inf, 0, 0)
    const float g = __fmul_rn(-gm, sc.hi), fl = __fsub_rn(gm, far);
    float gs, gt;
    if (fabsf(g) < 4096.f && fl >= kTopkLowest<D>) {
        const uint32_t raise = topk_floor<D>(fl);
#pragma unroll
        for (int u = 0; u < kTopkGroup<D>; ++u)
            if (kFull || u < nvalid) topk_raise<D>(q[u], raise);
        topk_sums<D, kFull, false>(q, nvalid, gm, g, sc, gs, gt);
        const float r = __fmaf_rn(-gm, sc.hi, -g), more = __fmul_rn(r, (float)kLn2);
        gt = __fmaf_rn(r, gs, gt);
        gt = __fmaf_rn(gt, more, gt);
        gs = __fmaf_rn(gs, more, gs);
    } else {
        topk_sums<D, kFull, true>(q, nvalid, gm, g, sc, gs, gt);
    }
    if (a.m == gm) {
        a.s = __fadd_rn(a.s, gs);
        a.t = __fadd_rn(a.t, gt);
    } else {
        const float d = to_log2_1<true>(__fsub_rn(a.m, gm), sc), f = ex2_ftz(d);
        a.t = __fmaf_rn(f, __fmaf_rn(a.s, fmaxf(d, -1e30f), a.t), gt);
        a.s = __fmaf_rn(a.s, f, gs);
    }
    a.m = gm;
    return w;
}

// As ms_merge, with T; a NaN is the larger one, whatever it meets.
__device__ __forceinline__ MST mst_merge(MST a, MST b, const Scale& sc) {
    const bool a_big = a.m >= b.m || a.m != a.m;
    const MST big = a_big ? a : b, small = a_big ? b : a;
    float r, d = 0.f;
    if (small.m == -INFINITY) r = 0.f;
    else if (small.m == big.m) r = 1.f;
    else {
        d = to_log2_1<true>(__fsub_rn(small.m, big.m), sc);
        r = ex2_ftz(d);
        d = fmaxf(d, -1e30f);
    }
    return MST{big.m, __fmaf_rn(small.s, r, big.s), __fmaf_rn(r, __fmaf_rn(small.s, d, small.t), big.t)};
}
// The partial of a tile out of its lanes', with the bias of ex2 taken off S and T.
__device__ __forceinline__ MST topk_tile_partial(MST p, const Scale& sc) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        MST o;
        o.m = __shfl_xor_sync(0xffffffffu, p.m, off);
        o.s = __shfl_xor_sync(0xffffffffu, p.s, off);
        o.t = __shfl_xor_sync(0xffffffffu, p.t, off);
        p = mst_merge(p, o, sc);
    }
    p.s = __fmaf_rn(p.s, kEx2BiasComp, p.s);
    p.t = __fmaf_rn(p.t, kEx2BiasComp, p.t);
    return p;
}

// ---------------------------------------------------------------- scan

// What a tile's warp writes: slots as its runs of groups end, at the end the partial.
template <Dt D>
struct TopkTile {
    char* slot;       // this lane's next slot
    uint32_t w;       // maximum of the run so far
    int in_run, run, step;
    __device__ __forceinline__ void begin(const TopkArgs& a, int64_t t, int tile, int lane) {
        constexpr int SB = Unit<D>::kElemBytes;
        slot = static_cast<char*>(a.slots) + ((t * a.runs * a.tiles + tile) * (int64_t)kWarp + lane) * SB;
        step = a.tiles * kWarp * SB;
        w = kWordNegInf<D>;
        in_run = run = 0;
    }
    __device__ __forceinline__ void put() {
        const float f = word_value<D>(w);
        if constexpr (D == Dt::F32) *reinterpret_cast<float*>(slot) = f;
        else if constexpr (D == Dt::BF16)   // exact: f is one of the elements
            *reinterpret_cast<uint16_t*>(slot) = (uint16_t)(pack_bf16x2(f, f) & 0xffffu);
        else *reinterpret_cast<uint16_t*>(slot) = (uint16_t)(pack_f16x2(f, f) & 0xffffu);
        slot += step;
        w = kWordNegInf<D>;
        in_run = 0;
        ++run;
    }
    __device__ __forceinline__ void group(const TopkArgs& a, uint32_t gw) {
        if (a.slots == nullptr) return;
        w = word_max<D>(w, gw);
        if (++in_run == a.per) put();
    }
    __device__ __forceinline__ void end(const TopkArgs& a, int64_t t, int tile, int lane, MST lane_sum) {
        if (a.slots != nullptr) {
            if (in_run > 0) put();
            while (run < a.runs) put();   // runs that this tile does not reach
        }
        const MST p = topk_tile_partial(lane_sum, a.sc);
        if (lane == 0) a.parts[t * a.tiles + tile] = make_float4(p.m, p.s, p.t, 0.f);
    }
};

// The active ones of the rows first, first + step, ...: 32 rows are looked at together.
struct TopkRows {
    int64_t first, step, rows, at;   // row number `at` and on are not looked at yet
    uint32_t bits;
    __device__ __forceinline__ int64_t next(const TopkArgs& a, int lane) {
        while (bits == 0) {
            if (at >= rows) return -1;
            const int64_t j = at + lane;
            bits = __ballot_sync(0xffffffffu, j < rows && topk_active(a, first + j * step));
            at += kWarp;
        }
        const int b = __ffs(bits) - 1;
        bits &= bits - 1;
        return first + (at - kWarp + b) * step;
    }
};

// The unit of 16 (FP32: 32) bytes at byte `at` of shared memory, any multiple of the element: the
// aligned pieces that hold it, shifted together (by words, alike for a row, then by half a word).
template <Dt D>
__device__ __forceinline__ void topk_lds_shifted(uint32_t at, Unit<D>& u) {
    constexpr int N = Unit<D>::kWords;
    uint32_t w[N + 4];
#pragma unroll
    for (int k = 0; k < N / 4 + 1; ++k) {
        const uint4 q = lds_v4((at & ~15u) + 16 * k);
        w[4 * k] = q.x; w[4 * k + 1] = q.y; w[4 * k + 2] = q.z; w[4 * k + 3] = q.w;
    }
#pragma unroll
    for (int s = 2; s >= 1; s >>= 1) {
        if ((at >> 2) & s) {
#pragma unroll
            for (int k = 0; k + s < N + 4; ++k) w[k] = w[k + s];
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (D == Dt::F32) u.w[k] = w[k];
        else u.w[k] = __funnelshift_r(w[k], w[k + 1], (at & 2u) * 8);
    }
}

// Persistent CTAs of kWarps warps, a warp per tile of a row and the same tile of every row it
// comes to, fed by a ring of kStages groups of its own with bulk copies; the warps wait for
// nothing but their own copies.  Many rows: 16 warps and 3 stages (192 KB on their way a
// SM).  Few: 4 warps and 6 stages, so that a wide row spreads over four SMs and a whole tile of a
// vocabulary up to 196608 is on its way at once.
//
// kShift: rows of any alignment: the 16-byte blocks that hold a group are copied (the first and the
// last may reach up to 15 bytes beyond the row, inside the block of one of its values) and
// the units shifted out of two neighbours.  (By element loads 2048 x 151936 BF16 took 364 us, 156
// so.)
template <Dt D>
constexpr int kTopkStagePad = 16;
template <Dt D, int kWarps, int kRing>
constexpr int kTopkRingBytes = kWarps * kRing * (kTopkStage<D> + kTopkStagePad<D> + 8);
template <Dt D, int kWarps, int kRing, bool kShift>
__global__ void __launch_bounds__(kWarps * kWarp, 1)
k_logp_topk_scan(TopkArgs a) {
    constexpr int EB = Unit<D>::kElemBytes, UB = Unit<D>::kBytes, SB = kTopkStage<D>, PB = SB + kTopkStagePad<D>,
                  kStages = kRing, kN = kTopkGroup<D>, kGU = kTopkGroupUnits<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t who = (int64_t)blockIdx.x * kWarps + warp, all = (int64_t)gridDim.x * kWarps;   // multiples of tiles
    const int my_tile = (int)(who % a.tiles);
    const uint32_t stage0 = smem_u32(smem + warp * kStages * PB);
    const uint32_t bar0 = smem_u32(smem + kWarps * kStages * PB) + warp * kStages * 8;
    if (lane < kStages) mbar_init(bar0 + lane * 8, 1);
    fence_mbar_init();
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // tile-local extents fit in 32 bits (v < 2^31)
    const int64_t c0 = (int64_t)my_tile * a.W;
    const int width = (int)(c0 >= a.v ? 0 : (a.v - c0 < a.W ? a.v - c0 : a.W));
    const int nfull = width >> 3, nunit = (width + 7) >> 3;
    const int G = (nunit + kGU - 1) / kGU, Gfull = nfull / kGU;
    const int64_t first = who / a.tiles, step = all / a.tiles;
    const int64_t rows = a.n > first ? (a.n - 1 - first) / step + 1 : 0;
    const char* tile0 = static_cast<const char*>(a.x) + c0 * EB;

    TopkRows ahead{first, step, rows, 0, 0u}, mine = ahead;
    int64_t iss_t = G > 0 ? ahead.next(a, lane) : -1;
    const char* iss_at = tile0 + iss_t * a.ld * EB;   // of group iss_g
    int iss_g = 0, iss_st = 0, in_flight = 0;
    auto issue_next = [&]() {   // the next group of copies, if there is one
        if (iss_t < 0) return;
        if (lane == 0) {
            const int nv = nfull - iss_g * kGU;
            uint32_t bytes = nv <= 0 ? 0u : (uint32_t)((nv < kGU ? nv : kGU) * UB);
            const uint32_t bar = bar0 + iss_st * 8;
            const char* src = iss_at;
            if constexpr (kShift) {
                const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(src) & 15u);
                src -= mis;
                if (bytes != 0 && mis != 0) bytes += 16;
            }
            mbar_arrive_expect_tx(bar, bytes);
            if (bytes) bulk_g2s(stage0 + iss_st * PB, src, bytes, bar);
        }
        ++in_flight;
        iss_at += SB;
        if (++iss_st == kStages) iss_st = 0;
        if (++iss_g == G) {
            iss_g = 0;
            iss_t = ahead.next(a, lane);
            iss_at = tile0 + iss_t * a.ld * EB;
        }
    };
    for (int k = 0; k < kStages; ++k) issue_next();

    bool ok = true;
    int st = 0;
    uint32_t phase = 0;
    for (int64_t t = mine.next(a, lane); t >= 0; t = mine.next(a, lane)) {
        const char* tile = tile0 + t * a.ld * EB;
        TopkTile<D> out;
        out.begin(a, t, my_tile, lane);
        MST sum{-INFINITY, 0.f, 0.f};
        for (int g = 0; g < G && ok; ++g) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar0 + st * 8, phase, kWaitLimitCycles));
            if (!ok) break;
            --in_flight;
            const uint32_t mis = kShift ? (uint32_t)(reinterpret_cast<uintptr_t>(tile) & 15u) : 0u;
            const uint32_t sbase = stage0 + st * PB + lane * UB + mis;
            auto unit_at = [&](int u, Unit<D>& q) {
                if constexpr (kShift) topk_lds_shifted<D>(sbase + u * (kWarp * UB), q);
                else unit_load_shared<D>(sbase + u * (kWarp * UB), q);
            };
            Unit<D> q[kN];
            int nvalid = kN;
            if (g < Gfull) {
#pragma unroll
                for (int u = 0; u < kTopkGroup<D>; ++u) unit_at(u, q[u]);
            } else {
                nvalid = 0;
#pragma unroll
                for (int u = 0; u < kTopkGroup<D>; ++u) {
                    const int j = g * kGU + kWarp * u + lane;
                    if (j < nfull) {
                        unit_at(u, q[u]);
                        nvalid = u + 1;
                    } else if (j < nunit) {   // the ragged last unit
                        unit_load<D, false>(tile, (int64_t)j * 8, width, q[u]);
                        nvalid = u + 1;
                    } else {
                        unit_fill_neg_inf<D>(q[u]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) fence_proxy_async_smem();
            issue_next();
            out.group(a, nvalid == kN ? topk_update<D, true>(q, nvalid, sum, a.sc, a.far)
                                          : topk_update<D, false>(q, nvalid, sum, a.sc, a.far));
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }
        if (!ok) break;
        out.end(a, t, my_tile, lane, sum);
    }
    if (!ok) {   // wait (bounded) for the copies still in flight
        if (lane == 0) atomicExch(&g_topk_error, 1);
        for (int k = 0; k < in_flight; ++k) {
            (void)mbar_wait(bar0 + st * 8, phase, kWaitLimitCycles);
            if (++st == kStages) {
                st = 0;
                phase ^= 1u;
            }
        }
    }
}

// ---------------------------------------------------------------- finish

// The 8 columns [8 j, 8 j + 8) of a row of v, padded with -inf.
template <Dt D>
__device__ __forceinline__ void topk_unit(const char* row, int64_t col, int64_t end, bool vec, Unit<D>& u) {
    if (vec) unit_load<D, true>(row, col, end, u);
    else unit_load<D, false>(row, col, end, u);
}
// Element e of consecutive words.
template <Dt D>
__device__ __forceinline__ float topk_element(const uint32_t* w, int e) {
    if constexpr (D == Dt::F32) return __uint_as_float(w[e]);
    else if constexpr (D == Dt::BF16) return e & 1 ? bf_hi(w[e >> 1]) : bf_lo(w[e >> 1]);
    else return e & 1 ? h_hi(w[e >> 1]) : h_lo(w[e >> 1]);
}
// The first of a lane's cnt places behind `all` of them, which are then so many more.
__device__ __forceinline__ int topk_places(int cnt, int lane, int& all) {
    int upto = cnt;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
    }
    const int at = all + upto - cnt;
    all += __shfl_sync(0xffffffffu, upto, 31);
    return at;
}

// A warp's place in shared memory.
struct TopkScratch {
    u64 cand[kTopkCands];        // key of the value above, ~column below; in the slow path counts
    uint16_t list[kTopkList];
};
static_assert(kTopkCands * 8 >= 256 * 4, "the counts of a digit fit");
static_assert(kTopkSlotRuns * kTiles <= 96, "a lane has a bit for each of its slots");

struct TopkRow {
    const char* x;
    int64_t v;
    bool vec;
    int64_t* ids;
    float* top;
    double s, m;           // scale, largest logit
    const double* log_s;   // log S
    int k;
    __device__ __forceinline__ void put(int rank, uint32_t key, uint32_t col) const {
        ids[rank] = (int64_t)col;
        top[rank] = __double2float_rn(s * ((double)topk_value(key) - m) - *log_s);
    }
};

// The first `need` columns whose value has key `key`, as ranks `rank` and on.
template <Dt D>
__device__ void topk_take_equal(const TopkRow& r, uint32_t key, int rank, int need, int lane) {
    for (int64_t c = 0; c < r.v && need > 0; c += 8 * kWarp) {
        const int64_t col = c + 8 * lane;
        Unit<D> u;
        unit_fill_neg_inf<D>(u);
        if (col < r.v) topk_unit<D>(r.x, col, r.v, r.vec, u);
        uint32_t hit = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < r.v && topk_key(topk_element<D>(u.w, e)) == key) hit |= 1u << e;
        const int cnt = __popc(hit);
        int before = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += o;
        }
        const int all = __shfl_sync(0xffffffffu, before, 31);
        before -= cnt;
        for (int e = 0; e < 8; ++e)
            if (hit >> e & 1u) {
                if (before < need) r.put(rank + before, key, (uint32_t)(col + e));
                ++before;
            }
        rank += all;
        need -= all;
    }
}

// The candidates in their order.
__device__ __forceinline__ void topk_rank(const TopkRow& r, const u64* cand, int nc, int lane) {
    for (int i = lane; i < nc; i += kWarp) {
        const u64 c = cand[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < nc; ++j) rank += cand[j] > c;
        if (rank < r.k) r.put(rank, (uint32_t)(c >> 32), ~(uint32_t)c);
    }
}

// Any row, by the digits of the k-th largest key (five passes over it): where so many
// values are alike that the candidates have no room.
template <Dt D>
__device__ void topk_slow(const TopkRow& r, TopkScratch& sh, int lane) {
    uint32_t* count = reinterpret_cast<uint32_t*>(sh.cand);
    uint32_t key = 0, known = 0;
    int need = r.k;   // of those that begin with `key`
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = lane; i < 256; i += kWarp) count[i] = 0;
        __syncwarp();
        for (int64_t c = 8 * lane; c < r.v; c += 8 * kWarp) {
            Unit<D> u;
            topk_unit<D>(r.x, c, r.v, r.vec, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t q = topk_key(topk_element<D>(u.w, e));
                if (c + e < r.v && (q & known) == key) atomicAdd(count + (q >> shift & 255u), 1u);
            }
        }
        __syncwarp();
        // lane l has the digits 255 - 8 l and the seven below: counted from the top
        uint32_t mine = 0;
        for (int i = 0; i < 8; ++i) mine += count[255 - 8 * lane - i];
        uint32_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += o;
        }
        const uint32_t before = upto - mine;
        const bool here = before < (uint32_t)need && (uint32_t)need <= upto;
        int digit = 0, left = need - (int)before;
        if (here) {
            digit = 255 - 8 * lane;
            while (left > (int)count[digit]) left -= (int)count[digit--];
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;   // the digits hold v >= k values
        digit = __shfl_sync(0xffffffffu, digit, src);
        need = __shfl_sync(0xffffffffu, left, src);
        key |= (uint32_t)digit << shift;
        known |= 255u << shift;
        __syncwarp();
    }
    int nc = 0;
    for (int64_t c0 = 0; c0 < r.v && nc < r.k - need; c0 += 8 * kWarp) {
        const int64_t c = c0 + 8 * lane;
        Unit<D> u;
        unit_fill_neg_inf<D>(u);
        if (c < r.v) topk_unit<D>(r.x, c, r.v, r.vec, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t q = topk_key(topk_element<D>(u.w, e));
            const bool hit = c + e < r.v && q > key;
            const uint32_t bal = __ballot_sync(0xffffffffu, hit);
            if (hit) sh.cand[nc + __popc(bal & ((1u << lane) - 1u))] = (u64)q << 32 | (uint32_t)~(uint32_t)(c + e);
            nc += __popc(bal);   // r.k - need of them in all: below kTopkMax
        }
    }
    __syncwarp();
    topk_rank(r, sh.cand, nc, lane);
    topk_take_equal<D>(r, key, r.k - need, need, lane);
}

// A warp per row: the row's sums out of its tiles' and its k best columns out of the slots.
//
// The k-th largest of 128 maxima (four a lane, each over its share of the slots) bounds the
// k-th largest slot from below; the slots from that bound on (k and a few more) are listed and
// read again, their elements from the bound on compared with one another.  A -inf bound
// (fewer finite values than k) takes the finite ones alone, then -inf columns in order.
template <Dt D>
__global__ void __launch_bounds__(kTopkFinishWarps * kWarp)
k_logp_topk_finish(TopkArgs a, TopkOut o) {
    constexpr int EB = Unit<D>::kElemBytes;
    constexpr int kPerChunk = 16 / EB;   // slots of a lane's 16 bytes
    constexpr int kBatch = 6, kUnits = D == Dt::F32 ? 2 : 4;   // loads of a lane that wait together
    __shared__ TopkScratch scratch[kTopkFinishWarps];
    __shared__ float row_m[kTopkFinishWarps], row_s[kTopkFinishWarps], row_t[kTopkFinishWarps], row_x[kTopkFinishWarps];
    __shared__ double row_log[kTopkFinishWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = o.k;
    TopkScratch& sh = scratch[warp];
    for (int64_t t0 = (int64_t)blockIdx.x * kTopkFinishWarps; t0 < a.n; t0 += (int64_t)gridDim.x * kTopkFinishWarps) {
        const int64_t t = t0 + warp;
        const bool live = t < a.n, act = live && topk_active(a, t);
        const char* xr = static_cast<const char*>(a.x) + (live ? t : 0) * a.ld * EB;
        float row_max = 0.f;
        if (act) {
            float x_y = 0.f;
            if (a.y != nullptr) x_y = elem_value<D>(xr, __ldg(a.y + t));
            MST p{-INFINITY, 0.f, 0.f};
            if ((lane & 15) < a.tiles) {
                const float4 q = a.parts[t * a.tiles + (lane & 15)];
                p = MST{q.x, q.y, q.z};
            }
            const MS f = tile_fold16(MS{p.m, p.s}, a.sc.s);
            float term = 0.f;
            if (p.m != -INFINITY) {
                const float d = __fmul_rn(a.sc.s, __fsub_rn(p.m, f.m));
                term = __fmul_rn(expf(d), __fmaf_rn(p.s, fmaxf(__fmul_rn(d, kLog2e), -1e30f), p.t));
            }
#pragma unroll
            for (int off = 1; off <= 8; off <<= 1) term = __fadd_rn(term, __shfl_xor_sync(0xffffffffu, term, off, 16));
            row_max = f.m;
            if (lane == 0) {
                row_m[warp] = f.m;
                row_s[warp] = f.s;
                row_t[warp] = term;
                row_x[warp] = x_y;
            }
        } else if (live) {
            for (int j = lane; j < k; j += kWarp) {
                o.ids[t * k + j] = -1;
                o.top[t * k + j] = 0.f;
            }
            if (lane == 0) row_s[warp] = -1.f;   // not active
        }
        __syncthreads();
        // one warp for all rows' ends: an instruction of FP64 takes as long for one lane as for 32
        if (warp == kTopkFinishWarps - 1 && lane < kTopkFinishWarps && t0 + lane < a.n) {
            const int64_t r = t0 + lane;
            const bool on = !(row_s[lane] == -1.f);
            const float m = row_m[lane], sum = row_s[lane];
            float l = 0.f, lo = 0.f, lp = 0.f, h = 0.f;
            if (on) {
                const double log_s = log((double)sum);
                // -inf for a row of -inf alone; beside a NaN m is -inf too, but the sum is NaN
                const double lse = m == -INFINITY && sum == 0.f ? -(double)INFINITY : (double)a.sc.s * (double)m + log_s;
                row_log[lane] = log_s;
                l = __double2float_rn(lse);
                lo = isfinite(l) ? __double2float_rn(lse - (double)l) : 0.f;
                if (fabsf(__fmul_rn(a.sc.s, m)) >= kLseFar && isfinite(l))   // as finalize_row
                    lo = __double2float_rn(((double)a.sc.s * (double)m - (double)l) + log_s);
                // around the maximum, as the alternatives: next to a large one LSE has no digits left for log S
                lp = __double2float_rn((double)a.sc.s * ((double)row_x[lane] - (double)m) - log_s);
                h = __fmaf_rn(-(float)kLn2, __fdiv_rn(row_t[lane], sum), logf(sum));
                h = h < 0.f ? 0.f : h;   // of one value: log S is the rounding of S alone
            }
            if (o.logp) o.logp[r] = lp;
            o.lse[r] = l;
            if (o.lse_lo) o.lse_lo[r] = lo;
            o.entropy[r] = h;
        }
        if (k == 0) {
            __syncthreads();
            continue;
        }
        int nl = 0, nc = 0;
        const TopkRow r{xr, a.v, o.vec, o.ids + t * k, o.top + t * k, (double)a.sc.s, (double)row_max, row_log + warp, k};
        if (act) {
        const int nslot = a.tiles * a.runs * kWarp;
        const uint4* slots = reinterpret_cast<const uint4*>(static_cast<const char*>(a.slots) + t * nslot * EB);
        const int chunks = (nslot + kPerChunk * kWarp - 1) / (kPerChunk * kWarp), lanes = nslot / kPerChunk;   // of 16 bytes
        uint32_t best[4] = {kWordNegInf<D>, kWordNegInf<D>, kWordNegInf<D>, kWordNegInf<D>};
        if (nslot <= 4 * kWarp) {   // each on its own
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = j * kWarp + lane;
                best[j] = 0;
                if (i < nslot) best[j] = topk_key(topk_element<D>(reinterpret_cast<const uint32_t*>(slots) + i / (4 / EB), i % (4 / EB)));
            }
        } else {
            for (int c0 = 0; c0 < chunks; c0 += kBatch) {   // the loads of a batch together
                uint4 q[kBatch];
#pragma unroll
                for (int c = 0; c < kBatch; ++c) {
                    const int i = (c0 + c) * kWarp + lane;
                    q[c] = i < lanes ? slots[i]
                                     : make_uint4(kWordNegInf<D>, kWordNegInf<D>, kWordNegInf<D>, kWordNegInf<D>);
                }
#pragma unroll
                for (int c = 0; c < kBatch; ++c) {
                    best[0] = word_max<D>(best[0], q[c].x);
                    best[1] = word_max<D>(best[1], q[c].y);
                    best[2] = word_max<D>(best[2], q[c].z);
                    best[3] = word_max<D>(best[3], q[c].w);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) best[j] = topk_key(word_value<D>(best[j]));
        }
        auto order = [&](int i0, int i1) {
            const uint32_t hi = max(best[i0], best[i1]), lo = min(best[i0], best[i1]);
            best[i0] = hi;
            best[i1] = lo;
        };
        order(0, 1); order(2, 3); order(0, 2); order(1, 3); order(1, 2);
        uint32_t bound = 0;
        for (int j = 0; j < k; ++j) {
            bound = __reduce_max_sync(0xffffffffu, best[0]);
            const uint32_t who = __ballot_sync(0xffffffffu, best[0] == bound);
            if (lane == __ffs(who) - 1) {
                best[0] = best[1];
                best[1] = best[2];
                best[2] = best[3];
                best[3] = 0;
            }
        }
        if (bound <= kKeyNegInf) bound = kKeyNegInf + 1;   // finite values only
        const float least = topk_value(bound);             // (a NaN: everything, and so the slow path)
        auto enough = [&](float f) { return !(f < least); };
        // the slots from the bound on: a bit each, then places in order of the lanes
        uint32_t hit[3] = {0u, 0u, 0u};
        int cnt = 0;
#pragma unroll
        for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int cc = 0; cc < 32 / kPerChunk; ++cc) {
                const int c = h * (32 / kPerChunk) + cc;
                if (c * kWarp + lane < lanes) {
                    const uint4 q = slots[c * kWarp + lane];
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < kPerChunk; ++e)
                        hit[h] |= (uint32_t)enough(topk_element<D>(w, e)) << (cc * kPerChunk + e);
                }
            }
#pragma unroll
        for (int h = 0; h < 3; ++h) cnt += __popc(hit[h]);
        int at = topk_places(cnt, lane, nl);
#pragma unroll
        for (int h = 0; h < 3; ++h)
            for (uint32_t b = hit[h]; b != 0; b &= b - 1) {
                const int i = h * 32 + __ffs(b) - 1;
                if (at < kTopkList)
                    sh.list[at] = (uint16_t)((i / kPerChunk * kWarp + lane) * kPerChunk + i % kPerChunk);
                ++at;
            }
        __syncwarp();
        if (nl <= kTopkList) {
            // kN lanes a slot, its units of a group each
            constexpr int kN = kTopkGroup<D>, kSlots = kWarp / kN;
            const int64_t nunit_row = a.W >> 3;
            const int tile_bits = __ffs(a.tiles) - 1;   // a power of two
            for (int gq = 0; gq < a.per; ++gq)
                for (int i0 = 0; i0 < nl && nc <= kTopkCands; i0 += kUnits * kSlots) {
                    Unit<D> u[kUnits];   // loaded together
                    uint32_t col[kUnits];
#pragma unroll
                    for (int b = 0; b < kUnits; ++b) {
                        const int i = i0 + b * kSlots + lane / kN;
                        unit_fill_neg_inf<D>(u[b]);
                        col[b] = 0;
                        if (i < nl) {
                            const int s = sh.list[i], tr = s / kWarp, tile = tr & (a.tiles - 1), run = tr >> tile_bits;
                            const int64_t j = ((int64_t)run * a.per + gq) * kTopkGroupUnits<D> + kWarp * (lane % kN) + (s & 31);
                            const int64_t c = (int64_t)tile * a.W + j * 8;
                            const int64_t end = min(a.v, (int64_t)(tile + 1) * a.W);
                            col[b] = (uint32_t)c;
                            if (j < nunit_row && c < end) topk_unit<D>(xr, c, end, o.vec, u[b]);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < kUnits; ++b) {
                        uint32_t hits = 0;   // columns outside are -inf: below the bound
#pragma unroll
                        for (int e = 0; e < 8; ++e) hits |= (uint32_t)enough(topk_element<D>(u[b].w, e)) << e;
                        if (!__any_sync(0xffffffffu, hits)) continue;
                        int to = topk_places(__popc(hits), lane, nc);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (hits >> e & 1u) {
                                if (to < kTopkCands)
                                    sh.cand[to] = (u64)topk_key(topk_element<D>(u[b].w, e)) << 32 |
                                                  (uint32_t)~(col[b] + (uint32_t)e);
                                ++to;
                            }
                    }
                }
        }
        }
        __syncthreads();   // the candidates of the warp, and the logarithms
        if (act) {
            if (nl > kTopkList || nc > kTopkCands) {
                topk_slow<D>(r, sh, lane);
            } else {
                topk_rank(r, sh.cand, nc, lane);
                if (nc < k) topk_take_equal<D>(r, kKeyNegInf, nc, k - nc, lane);
            }
        }
        __syncthreads();   // the next rows use the same places
    }
}

// ---------------------------------------------------------------- backward

struct TopkBwdArgs {
    const void* x;
    int64_t n, v, ld;
    const int64_t* y;      // nullable
    int64_t ignore_index;
    const uint8_t* mask;
    float s, inv_s;
    const float *lse, *lse_lo, *entropy;
    const int64_t* ids;    // [n, k]
    int k;
    const float *g, *gh, *gt;   // [n], [n], [n, k]; each nullable
    void* dx;
    int64_t ld_out;
};

// The 8 values from p on, at any address: the aligned 16-byte pieces that hold them (up to 15 bytes
// beyond, inside the piece of one of them), shifted together.  The shift is the same for a row.
// kPlain: of memory that this kernel writes; kWhole: the values are whole pieces.
template <Dt D, bool kPlain, bool kWhole>
__device__ __forceinline__ void topk_load_any(const char* p, Unit<D>& u) {
    constexpr int N = Unit<D>::kWords;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const char* base = p - off;
    uint32_t w[N + 4];
#pragma unroll
    for (int k = 0; k < N / 4 + 1; ++k) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (k < N / 4 || (!kWhole && off != 0))
            q = kPlain ? ld_v4(base + 16 * k) : __ldg(reinterpret_cast<const uint4*>(base) + k);
        w[4 * k] = q.x; w[4 * k + 1] = q.y; w[4 * k + 2] = q.z; w[4 * k + 3] = q.w;
    }
    if constexpr (!kWhole) {
#pragma unroll
        for (int s = 2; s >= 1; s >>= 1) {
            if ((off >> 2) & s) {
#pragma unroll
                for (int k = 0; k + s < N + 4; ++k) w[k] = w[k + s];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (D == Dt::F32 || kWhole) u.w[k] = w[k];
        else u.w[k] = __funnelshift_r(w[k], w[k + 1], (off & 2u) * 8);
    }
}

// The columns with a one-hot term, number 0 the target, then the alternatives: this thread's (-1:
// none), and all in shared memory, which a barrier of the CTA makes readable.
__device__ __forceinline__ int64_t topk_bwd_columns(const TopkBwdArgs& a, int64_t t, int64_t yt, int64_t* sh_col,
                                                    float* sh_w) {
    const int tid = threadIdx.x;
    int64_t col = -1;
    float wt = 0.f;
    if (tid == 0) {
        col = a.g ? yt : -1;
        wt = col >= 0 ? __ldg(a.g + t) : 0.f;
    } else if (a.gt != nullptr && tid <= a.k) {
        col = __ldg(a.ids + t * a.k + tid - 1);
        if (col < 0 || col >= a.v) col = -1;
        wt = col >= 0 ? __ldg(a.gt + t * a.k + tid - 1) : 0.f;
    }
    if (tid <= kTopkMax) {
        sh_col[tid] = col;
        sh_w[tid] = wt;
    }
    return col;
}
// G: three of the places a lane, then the butterfly.
__device__ __forceinline__ float topk_bwd_total(const float* sh_w, int lane) {
    float G = __fadd_rn(sh_w[lane], sh_w[lane + 32]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) G = __fadd_rn(G, __shfl_xor_sync(0xffffffffu, G, off));
    return __fadd_rn(G, sh_w[kTopkMax]);
}
// s ((w - G) - G expm1(lp) - gh p (lp + H)), w the sum of the gradients of that column.
template <bool kEntropy>
__device__ __forceinline__ float topk_bwd_special(const TopkBwdArgs& a, int64_t col, const int64_t* sh_col,
                                                  const float* sh_w, float lp, float G, float gh, float H) {
    float sum = 0.f;
    for (int j = 0; j <= a.k; ++j) sum += sh_col[j] == col ? sh_w[j] : 0.f;
    float ds = __fsub_rn(__fsub_rn(sum, G), __fmul_rn(G, expm1f(lp)));
    if (kEntropy) ds = __fmaf_rn(-gh, __fmul_rn(expf(lp), __fadd_rn(lp, H)), ds);
    return __fmul_rn(a.s, ds);
}
template <Dt D>
__device__ __forceinline__ void topk_bwd_put(char* dr, int64_t col, float d) {
    if constexpr (D == Dt::F32) reinterpret_cast<float*>(dr)[col] = d;
    else if constexpr (D == Dt::BF16)
        reinterpret_cast<uint16_t*>(dr)[col] = (uint16_t)(pack_bf16x2(d, d) & 0xffffu);
    else reinterpret_cast<uint16_t*>(dr)[col] = (uint16_t)(pack_f16x2(d, d) & 0xffffu);
}

// Rows of a large |LSE| (and of one without a number): beside it neither LSE nor its rounding residual
// holds log S, and a floor below it may be LSE itself.  One CTA takes the row, finds its
// maximum M and sum again and forms lp = s (x - M) - log S of each column.  Two passes more
// over rows that are rare: closed by a finite fill throughout, or of a temperature below
// 1e-5 or so.  One of 151936 BF16 takes 260 us, 256 of them 427 (ordinary rows 3.5 and 27).
constexpr float kTopkFarLse = 262144.f;
// Below the floor p is 0.
__device__ __forceinline__ float topk_bwd_floor(const TopkBwdArgs& a, float l) {
    return __fmul_rn(__fsub_rn(l, 200.f), a.inv_s);
}
__device__ __forceinline__ bool topk_bwd_far(float l, float fl) { return !(fabsf(l) < kTopkFarLse && fl > -3e38f); }
// An active row's target, -1 without targets; -2: not active.
__device__ __forceinline__ int64_t topk_bwd_target(const TopkBwdArgs& a, int64_t t) {
    if (a.mask != nullptr && __ldg(a.mask + t) == 0) return -2;
    if (a.y == nullptr) return -1;
    const int64_t y = __ldg(a.y + t);
    return y >= 0 && y < a.v && y != a.ignore_index ? y : -2;
}
template <Dt D, bool kEntropy>
__device__ __noinline__ void topk_bwd_far_row(const TopkBwdArgs& a, int64_t t, int64_t* sh_col, float* sh_w) {
    const int64_t yt = topk_bwd_target(a, t);
    const float l = __ldg(a.lse + t);
    if (yt == -2 || !topk_bwd_far(l, topk_bwd_floor(a, l))) return;   // the same for the whole CTA
    constexpr int EB = Unit<D>::kElemBytes, NW = Unit<D>::kWords, kWarps = kBwdThreads / kWarp, kB = D == Dt::F32 ? 1 : 2;
    __shared__ float sh_max[kWarps];
    __shared__ double sh_sum[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const char* xr = static_cast<const char*>(a.x) + t * a.ld * EB;   // dx may be x: plain loads
    char* dr = static_cast<char*>(a.dx) + t * a.ld_out * EB;
    const bool vec_out = (reinterpret_cast<uintptr_t>(dr) & 15u) == 0;
    // f(c, u) for the units of this thread, kB loaded together: the same wherever the row lies
    auto each = [&](auto&& f) {
#pragma unroll 1
        for (int64_t c0 = 8 * tid; c0 < a.v; c0 += kB * 8 * kBwdThreads) {
            Unit<D> u[kB];
#pragma unroll
            for (int b = 0; b < kB; ++b) {
                const int64_t c = c0 + b * 8 * kBwdThreads;
                if (c + 8 <= a.v) topk_load_any<D, true, false>(xr + c * EB, u[b]);
                else if (c < a.v) bwd_load<D, false, true>(xr, c, a.v, u[b]);
            }
#pragma unroll
            for (int b = 0; b < kB; ++b) {
                const int64_t c = c0 + b * 8 * kBwdThreads;
                if (c < a.v) f(c, u[b]);
            }
        }
    };
    const int64_t col = topk_bwd_columns(a, t, yt, sh_col, sh_w);
    float M = -INFINITY;
    each([&](int64_t c, const Unit<D>& u) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < a.v) M = f_max_nan(M, topk_element<D>(u.w, e));
    });
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = f_max_nan(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) sh_max[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = f_max_nan(M, sh_max[w]);
    double S = 0.0;
    each([&](int64_t c, const Unit<D>& u) {
        float p = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < a.v) p += expf(__fmul_rn(a.s, __fsub_rn(topk_element<D>(u.w, e), M)));
        S += (double)p;
    });
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) S += __shfl_xor_sync(0xffffffffu, S, off);
    if (lane == 0) sh_sum[warp] = S;
    __syncthreads();
    S = 0.0;
    for (int w = 0; w < kWarps; ++w) S += sh_sum[w];
    const float log_s = (float)log(S), G = topk_bwd_total(sh_w, lane);
    const float gh = kEntropy ? __ldg(a.gh + t) : 0.f, H = kEntropy ? __ldg(a.entropy + t) : 0.f;
    auto logp = [&](float x) {   // at -200 p is 0, and times a number
        return f_max_nan(__fsub_rn(__fmul_rn(a.s, __fsub_rn(x, M)), log_s), -200.f);
    };
    float ds = 0.f;
    if (col >= 0) {
        const float lp = logp(bits_value<D>(elem_bits_plain<D>(xr, col)));
        ds = topk_bwd_special<kEntropy>(a, col, sh_col, sh_w, lp, G, gh, H);
    }
    __syncthreads();   // the logits of the columns apart are read
    each([&](int64_t c, const Unit<D>& u) {
        uint32_t out[NW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float lp = logp(topk_element<D>(u.w, 2 * k + e));
                const float q = kEntropy ? __fmaf_rn(gh, __fadd_rn(lp, H), G) : G;
                d[e] = __fmul_rn(-a.s, __fmul_rn(expf(lp), q));
            }
            put_pair<D>(out, k, d[0], d[1]);
        }
        if (vec_out) bwd_store<D, true>(dr, c, a.v, out);
        else bwd_store<D, false>(dr, c, a.v, out);
    });
    __syncthreads();   // the row is stored; sh_col and sh_w are read
    if (col >= 0) topk_bwd_put<D>(dr, col, ds);
}

// One CTA per (segment of kBwdSegCols columns, row), elementwise; exp as in k_logp_bwd.
// The columns with a one-hot term (target and alternatives, at most 65) that lie in the
// segment are computed apart by a thread each, from logits read before any store (dx may be
// x), and stored after the segment: for the target alone w = G and nothing cancels.
//
// kShift: rows of any alignment.  A thread's units then lie on the 16-byte pieces of dx's row (the
// first starts up to 7 columns before it), x's are shifted out of two pieces.  (By elements, 2048 x
// 151936 BF16 in rows 151937 apart took 709 us, 275 so; aligned rows 179.)
template <Dt D, bool kShift, bool kInPlace, bool kEntropy>
__global__ void __launch_bounds__(kBwdThreads, kBwdMinBlocks<D>)
k_logp_topk_bwd(const __grid_constant__ TopkBwdArgs a) {
    constexpr int EB = Unit<D>::kElemBytes, NW = Unit<D>::kWords;
    constexpr int kBatch = kShift ? kBwdUnitsPerThread / 2 : kBwdUnitsPerThread;   // units loaded together
    __shared__ int64_t sh_col[kTopkMax + 1];
    __shared__ float sh_w[kTopkMax + 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t cs = (int64_t)kBwdThreads * 8;
    bool far = false;   // one of the rows is left to topk_bwd_far_row
#pragma unroll 1
    for (int64_t t = blockIdx.y; t < a.n; t += gridDim.y) {
        const char* xr = static_cast<const char*>(a.x) + t * a.ld * EB;
        char* dr = static_cast<char*>(a.dx) + t * a.ld_out * EB;
        const int64_t seg0 = (int64_t)blockIdx.x * kBwdSegCols -
                             (kShift ? (int64_t)(reinterpret_cast<uintptr_t>(dr) & 15u) / EB : 0);
        const int64_t col0 = seg0 + (int64_t)tid * 8;
        // unit at column c (kShift: it may begin before the row)
        auto load = [&](int64_t c, Unit<D>& u) {
            if constexpr (!kShift) {
                bwd_load<D, true, kInPlace>(xr, c, a.v, u);
            } else if (c >= 0 && c + 8 <= a.v) {
                topk_load_any<D, kInPlace, kInPlace>(xr + c * EB, u);   // in place the units are whole pieces
            } else {
#pragma unroll
                for (int k = 0; k < NW; ++k) u.w[k] = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j >= 0 && c + j < a.v) {
                        const uint32_t b = kInPlace ? elem_bits_plain<D>(xr, c + j) : elem_bits<D>(xr, c + j);
                        if constexpr (D == Dt::F32) u.w[j] = b;
                        else u.w[j >> 1] |= b << (16 * (j & 1));
                    }
            }
        };
        auto store = [&](int64_t c, const uint32_t (&o)[NW]) {
            if (!kShift || c >= 0) {
                bwd_store<D, true>(dr, c, a.v, o);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j >= 0 && c + j < a.v) {
                        if constexpr (D == Dt::F32) reinterpret_cast<uint32_t*>(dr)[c + j] = o[j];
                        else reinterpret_cast<uint16_t*>(dr)[c + j] =
                            (uint16_t)((j & 1) ? (o[j >> 1] >> 16) : (o[j >> 1] & 0xffffu));
                    }
            }
        };
        const float l = __ldg(a.lse + t);
        const int64_t yt = topk_bwd_target(a, t);
        if (yt == -2) {   // the same for the whole CTA
            uint32_t z[NW];
#pragma unroll
            for (int j = 0; j < NW; ++j) z[j] = 0u;
#pragma unroll
            for (int u = 0; u < kBwdUnitsPerThread; ++u)
                if (col0 + u * cs < a.v) store(col0 + u * cs, z);
            continue;
        }
        const float fl = topk_bwd_floor(a, l);
        if (topk_bwd_far(l, fl)) {   // the same for the whole CTA, and the row
            far = true;
            continue;
        }
        Unit<D> w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (col0 + u * cs < a.v) load(col0 + u * cs, w[u]);

        const int64_t col = topk_bwd_columns(a, t, yt, sh_col, sh_w);
        const bool special = col >= 0 && col >= seg0 && col < seg0 + kBwdSegCols;   // (seg0 may lie before the row)
        float xs = 0.f;
        if (special) xs = bits_value<D>(kInPlace ? elem_bits_plain<D>(xr, col) : elem_bits<D>(xr, col));
        const bool any = __syncthreads_or(special);   // also: the logits of the columns apart are read
        const float G = topk_bwd_total(sh_w, lane);

        const float l_lo = a.lse_lo ? __ldg(a.lse_lo + t) : 0.f;
        const float gh = kEntropy ? __ldg(a.gh + t) : 0.f, H = kEntropy ? __ldg(a.entropy + t) : 0.f;
        BwdRow r;
        r.s = a.s;
        r.gs = __fmul_rn(a.s, G);
        r.lr = (fabsf(l) < 8388608.f) ? __fmul_rn(rintf(__fmul_rn(l, 65536.f)), 1.f / 65536.f) : l;
        r.delta = __fadd_rn(__fsub_rn(l, r.lr), l_lo);   // l - lr is exact
        r.floor_f = fl;
        r.floor_w = 0xff80ff80u;
        if constexpr (D == Dt::BF16) {
            const uint32_t b = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(fl));
            r.floor_w = b | (b << 16);
        }
        r.neg_lr = f2(-r.lr, -r.lr);
        r.s2 = f2(a.s, a.s);
        // -s (e^-delta + b), with b for the bias of ex2; times G, or times G + gh (lp + H)
        const float base = kEntropy ? a.s : r.gs;
        const float coef = __fmaf_rn(base, __fsub_rn(bwd_rest(r.delta), kEx2BiasComp), -base);
        r.coef2 = f2(coef, coef);
        const float g0 = __fmaf_rn(gh, __fsub_rn(H, r.delta), G);
        const u64 g02 = f2(g0, g0), gh2 = f2(gh, gh), l2e = f2(kLog2e, kLog2e);
        const u64 nln2hi = f2(-kLn2Hi, -kLn2Hi), nln2lo = f2(-kLn2Lo, -kLn2Lo);

        float ds = 0.f;
        if (special) {
            const float lp = __fsub_rn(__fmaf_rn(a.s, fmaxf(xs, fl), -r.lr), r.delta);
            ds = topk_bwd_special<kEntropy>(a, col, sh_col, sh_w, lp, G, gh, H);
        }
#pragma unroll
        for (int half = 0; half < kBwdUnitsPerThread / kBatch; ++half) {
            if (half > 0) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (col0 + (half * kBatch + u) * cs < a.v) load(col0 + (half * kBatch + u) * cs, w[u]);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int64_t c = col0 + (half * kBatch + u) * cs;
                if (c < a.v) {
                    uint32_t out[NW];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const u64 tt = f2_fma(bwd_pair<D>(w[u], k, r), r.s2, r.neg_lr);
                        const u64 e = f2_mul(tt, l2e);
                        const u64 lost = f2_fma(e, nln2lo, f2_fma(e, nln2hi, tt));
                        float a0, a1;
                        f2_split(e, a0, a1);
                        u64 q = f2_mul(f2(ex2_ftz(a0), ex2_ftz(a1)), r.coef2);
                        if (kEntropy) q = f2_mul(q, f2_fma(tt, gh2, g02));
                        float d0, d1;
                        f2_split(f2_fma(q, lost, q), d0, d1);
                        put_pair<D>(out, k, d0, d1);
                    }
                    store(c, out);
                }
            }
        }
        __syncthreads();   // the segment is stored; sh_col and sh_w are read
        if (any && special) topk_bwd_put<D>(dr, col, ds);
    }
    if (far && blockIdx.x == 0) {
#pragma unroll 1
        for (int64_t t = blockIdx.y; t < a.n; t += gridDim.y) topk_bwd_far_row<D, kEntropy>(a, t, sh_col, sh_w);
    }
}

}  // namespace flp
