// Product of e4m3 matrices with FP32 scales on the tcgen05 tensor cores of sm_103a:
//   C[m, n] = sum over K blocks b of  sa[b, m] sb[b, n] sum_k A[m, k] B[n, k],  k in block b
// for A [M, K] with one scale for each 128 columns of a row and B [N, K] with one for each
// 128 columns of a row or for each 128 x 128 block.  Rows of A and B are contiguous.
//
// The sum of a block is 4 MMAs (kind::f8f6f4, K = 32) into an accumulator of its own in
// tensor memory; the epilogue warps read it while the next block's MMAs run and add it,
// scaled, to FP32 sums in registers: C's only long sum, one rounding a block.
//
// k_fp8_pair, for more rows than a few: CTA pairs (a cluster of 2) on 256 x 256 tiles with
// cta_group::2, as the bf16 products (gemm_bf16.cuh): each CTA copies 128 rows of A and of B
// a K block (32 KB a stage, 5 stages, 4 with B's scales a row beside them) and the even CTA
// issues M = 256, N = 256 MMAs.  Two accumulators of 256 columns take all of tensor memory.
// Eight epilogue warps a CTA: a thread has one row and 128 columns, which is what its registers
// hold.  The MMAs of a K block alone take 550 cycles; the epilogue bounds it at 750: 360 of 128
// multiply-adds by two warps a scheduler, the rest the latencies of loads, signals and scales, which
// two warps cannot hide from each other and more have no registers for.  4096 x 8192 x 4096 103 us, 2.7
// PFLOP/s; B's scales a row are one more multiply a value and reads of shared memory, 160 us.
//
// k_fp8_tokens, for a few rows of A (tokens): the operands change places, 128 rows of B a
// tile and the tokens the MMA's N, so that B is streamed once at the memory's rate; with few
// tiles a cluster of CTAs shares one tile's K blocks and adds the sums in a fixed order
// through distributed shared memory.
//
// Every wait is bounded: one that runs out sets the error word and the CTA's abort flag, the
// copies and MMAs in flight are waited for, tensor memory is freed and the kernel returns.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tc_prims.cuh"

namespace flp {

constexpr long long kFp8WaitCycles = 4000000000LL;
static __device__ int g_fp8_error;   // 1 = a bounded wait ran out

constexpr int kFp8BK = 128;          // K of a scale's block: one 128-byte swizzle row

struct Fp8Args {
    int64_t M, N;
    int nkb;                  // K blocks
    const float *sa, *sb;     // [nkb, lda], [nkb, ldb]
    int64_t lda, ldb;
    int b_shift;              // B's scale of row n is sb[b ldb + (n >> b_shift)]
    void* c;                  // [M, ldc]
    int64_t ldc;
    int out_dtype;            // FLP_DTYPE_*
    int vec;                  // rows of C start on 16-byte boundaries
    int64_t tiles_m, tiles_n, group;
};

__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (mbar_try(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > kFp8WaitCycles) {
                *abort_flag = 1;
                atomicExch(&g_fp8_error, 1);
                return false;
            }
        }
    }
}
// The same for the epilogue, where the other's clock costs registers (4096 x 8192 x 4096 114 us, 102 so):
// by the clock's upper half alone, of which a tick is 2^32 cycles, about 2 s; it gives up with tick
// kTicks.
__device__ __forceinline__ uint32_t fp8_clock_hi() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%clock_hi;" : "=r"(t));
    return t;
}
template <uint32_t kTicks = 2>
__device__ __forceinline__ bool fp8_wait_short(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    const uint32_t t0 = fp8_clock_hi();
#pragma unroll 1
    while (!mbar_try(bar, parity)) {
        const bool late = fp8_clock_hi() - t0 >= kTicks;
        if (late || *abort_flag != 0) {
            *abort_flag = 1;
            if (late) atomicExch(&g_fp8_error, 1);
            return false;
        }
    }
    return true;
}
// The signal of a read accumulator to the even CTA: what it orders is tensor memory (the fences
// beside it do that), no other memory. With release and acquire at cluster scope each arrival
// waited for the warp's copies of scales in flight: 4096 x 8192 x 4096 took 273 us, 153 without.
__device__ __forceinline__ void fp8_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool fp8_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool fp8_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    if (fp8_try_cluster(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (fp8_try_cluster(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > kFp8WaitCycles) {
                *abort_flag = 1;
                atomicExch(&g_fp8_error, 1);
                return false;
            }
        }
    }
}

// K-major operand in rows of 128 bytes with 128-byte swizzle; a K step of 32 values is 32
// bytes further.
__device__ __forceinline__ uint64_t fp8_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f8f6f4 with e4m3 operands (type fields 0), FP32 accumulators, both K-major.
template <int kBM, int kBN>
__host__ __device__ constexpr uint32_t fp8_idesc() {
    return (1u << 4) | ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}
template <bool kPair>
__device__ __forceinline__ void umma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}
// One lane of a converged warp, the same one every time.  The MMA warp runs its loop with all lanes
// and issues by this one: addresses and descriptors then stay in uniform registers.
__device__ __forceinline__ bool fp8_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}
// Arrive on the barrier at this place of both CTAs of the pair when this thread's MMAs so far are done.
__device__ __forceinline__ void fp8_commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
// 16 consecutive binary32 columns of this thread's lane, not waited for: the registers hold them
// after tmem_wait_ld alone, and what reads them is volatile too and stands behind it.
__device__ __forceinline__ void tmem_ld_ahead(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// sum += s t, and sums += s (t b) of two columns at once.  Measured (sums and t in registers, cycles
// per FMA and scheduler): single 1.4, pairs 1.0; where pairs have to be formed of what comes
// from tensor memory the single form is as fast, but not where b multiplies first.
__device__ __forceinline__ void fp8_add(float& sum, float s, uint32_t t) {
    asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(sum) : "f"(s), "f"(__uint_as_float(t)));
}
__device__ __forceinline__ void fp8_add(u64& sum, u64 s, uint32_t lo, uint32_t hi, uint32_t b_lo, uint32_t b_hi) {
    asm volatile(
        "{\n\t.reg .b64 t, b;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 t, t, b;\n\tfma.rn.f32x2 %0, %1, t, %0;\n\t}"
        : "+l"(sum)
        : "l"(s), "r"(lo), "r"(hi), "r"(b_lo), "r"(b_hi));
}

__device__ __forceinline__ void fp8_cp4(uint32_t dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fp8_cp16(uint32_t dst, const float* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fp8_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fp8_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float fp8_lds(uint32_t a) {
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
    return r;
}

__device__ __forceinline__ void fp8_put_one(const Fp8Args& p, int64_t at, float v) {
    if (p.out_dtype == 2) static_cast<float*>(p.c)[at] = v;
    else static_cast<uint16_t*>(p.c)[at] =
        (uint16_t)((p.out_dtype == 0 ? pack_bf16x2(v, v) : pack_f16x2(v, v)) & 0xffffu);
}
// FP32 sums of a row, single or in pairs.
template <int kN, bool kPairs>
struct Fp8Sums {
    float s[kN];
    __device__ __forceinline__ float get(int j) const { return s[j]; }
};
template <int kN>
struct Fp8Sums<kN, true> {
    u64 s[kN / 2];
    __device__ __forceinline__ float get(int j) const {
        float lo, hi;
        f2_split(s[j >> 1], lo, hi);
        return j & 1 ? hi : lo;
    }
};

// 32 rows of kN sums (a row a lane) to rows [m, m + 32), columns [n, n + kN) of C, by way of boxes
// of 32 rows x 128 bytes in shared memory: chunk j of 16 bytes of row r at place j ^ (r mod 8), as
// the tensor map's 128-byte swizzle has it.  With p.vec the boxes (two by turns) go out by TMA, rows
// past C left out, columns by whole 16 bytes: a box that C's last column cuts inside such a piece would
// reach behind it, and goes as without p.vec, a row a turn, by elements.  (Each lane storing its own
// row took 6700 cycles a 128 x 256 tile, 32 lines an instruction; the warps' own stores of
// whole lines out of the boxes 3500, 16 us of 122 at 4096 x 8192 x 4096; by TMA 13.)
constexpr uint32_t kFp8Box = 32 * 128;
template <int kN, bool kPairs>
__device__ __forceinline__ void fp8_put_rows(const Fp8Args& p, const CUtensorMap* tm_c, int64_t m, int64_t n,
                                             const Fp8Sums<kN, kPairs>& sum, uint32_t boxes, int lane) {
    const bool wide = p.out_dtype == 2;
    const int cols = wide ? 32 : 64;   // of a box
#pragma unroll
    for (int part = 0; part < kN / 32; ++part) {
        if (!wide && (part & 1)) continue;
        const int64_t n0 = n + part * 32;
        if (n0 >= p.N || m >= p.M) break;   // the same for the warp
        const uint32_t box = boxes + (wide ? part & 1 : (part >> 1) & 1) * kFp8Box;
        // the copy that last used this box has read it; at a tile's start both boxes', of which a ragged
        // tile before may have left the first one last
        if (lane == 0) {
            if (part == 0) bulk_wait_read<0>();
            else bulk_wait_read<1>();
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
            if (wide) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(sum.get(part * 32 + 4 * j + k));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = (part * 32 + 8 * j + 2 * k) % kN;   // of a 16-bit box: kN is a multiple of 64
                    w[k] = p.out_dtype == 0 ? pack_bf16x2(sum.get(c), sum.get(c + 1))
                                            : pack_f16x2(sum.get(c), sum.get(c + 1));
                }
            }
            sts_v4(box + (uint32_t)(lane * 128 + ((j ^ (lane & 7)) * 16)), w[0], w[1], w[2], w[3]);
        }
        if (p.vec && (n0 + cols <= p.N || p.N % (wide ? 4 : 8) == 0)) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(tm_c, (int32_t)n0, (int32_t)m, box);
                bulk_commit_group();
            }
        } else {
            __syncwarp();
            const int eb = wide ? 4 : 2;
            const int64_t have = p.N - n0 < cols ? p.N - n0 : cols;
            for (int r = 0; r < 32 && m + r < p.M; ++r)
                for (int c = lane; c < have; c += 32) {
                    const int b = c * eb, at = (((b >> 4) ^ (r & 7)) << 4) | (b & 15);
                    const int64_t to = (m + r) * p.ldc + n0 + c;
                    if (wide) {
                        static_cast<float*>(p.c)[to] = fp8_lds(box + (uint32_t)(r * 128 + at));
                    } else {
                        unsigned short h;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(box + (uint32_t)(r * 128 + at)) : "memory");
                        static_cast<uint16_t*>(p.c)[to] = h;
                    }
                }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- CTA pairs

constexpr int kFp8EpiWarps = 8;
// three warpgroups: copies and MMAs, and two of the epilogue, which take registers from the
// first (the launch has 168 a thread: 3 x 168 = 504 >= 40 + 2 x 232)
constexpr int kFp8PairThreads = 128 + 32 * kFp8EpiWarps;
constexpr int kFp8FewRegs = 40, kFp8ManyRegs = 232;
constexpr uint32_t kFp8PairHalf = 128 * kFp8BK;                  // 16 KB: this CTA's rows of A, or of B
constexpr uint32_t kFp8PairStage = 2 * kFp8PairHalf;
constexpr int kFp8Chunk = 16;                                    // columns a load
constexpr int kFp8AheadCols = 4;                                 // K blocks of B's scales on their way
constexpr uint32_t kFp8ColScales = kFp8AheadCols * kFp8EpiWarps * 128 * 4;     // 128 a warp
template <bool kColVec>
constexpr int kFp8PairStages = kColVec ? 4 : 5;
// the ring, two boxes per epilogue warp, B's scales, barriers
template <bool kColVec>
constexpr size_t kFp8PairSmem = 1024 + (size_t)kFp8PairStages<kColVec> * kFp8PairStage + 2 * kFp8EpiWarps * kFp8Box +
                                (kColVec ? kFp8ColScales : 0) + 256;
static_assert(kFp8PairSmem<true> <= 232448 && kFp8PairSmem<false> <= 232448, "shared memory per CTA");

struct Fp8Tile {
    int64_t m, n;
};
// Tile u: groups of `group` row blocks, inside a group the row block is the fast index.
__device__ __forceinline__ Fp8Tile fp8_tile(int64_t u, const Fp8Args& p) {
    const int64_t per = p.group * p.tiles_n, g = u / per, r = u - g * per;
    const int64_t rows = (g + 1) * p.group <= p.tiles_m ? p.group : p.tiles_m - g * p.group;
    return Fp8Tile{g * p.group + r % rows, r / rows};
}

// B has a scale per 128 x 128 block (kB 0) or per row (1); per row, on 16-byte boundaries and a multiple
// of 4 rows (2): a lane then copies four at once (4096 x 8192 x 4096 160 us, by single ones 176; both
// in one kernel 176).
template <int kB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFp8PairThreads, 1)
k_fp8_pair(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
           const __grid_constant__ CUtensorMap tm_c, Fp8Args p) {
    constexpr bool kColVec = kB != 0;
    extern __shared__ __align__(1024) unsigned char fp8_smem[];
    const uint32_t raw = smem_u32(fp8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;   // the same offset in both CTAs
    constexpr int kStages = kFp8PairStages<kColVec>;
    const uint32_t boxes = base + kStages * kFp8PairStage, col_scales = boxes + 2 * kFp8EpiWarps * kFp8Box;
    const uint32_t bars = col_scales + (kColVec ? kFp8ColScales : 0);
    // full: a stage's copies are there; done: its MMAs are, so that it may be filled again and its
    // accumulator read; tempty: an accumulator has been read by both CTAs
    const uint32_t full0 = bars, done0 = bars + 8 * kStages, tempty0 = bars + 16 * kStages;
    const uint32_t drain = tempty0 + 16, slot = drain + 8;
    unsigned char* slot_gen = fp8_smem + (slot - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(slot_gen);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_gen + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int64_t tiles = p.tiles_m * p.tiles_n, cid = cluster_id_x(), ncl = cluster_count_x();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(done0 + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) mbar_init(tempty0 + 8 * a, 2 * kFp8EpiWarps);   // both CTAs' epilogue warps
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
        if (p.vec) prefetch_tmap(&tm_c);
    }
    if (warp == 1) {
        tmem_alloc_pair(slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();   // both CTAs' barriers initialised and tensor memory allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFp8FewRegs));
    if (warp == 0) {
        // ---------------- copies: each CTA its own halves; both complete on the even CTA's barrier
        if (lane == 0) {
            const uint32_t full_leader = map_to_rank(full0, 0);
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            for (int64_t u = cid; ok && u < tiles; u += ncl) {
                const Fp8Tile w = fp8_tile(u, p);
                const int m0 = (int)(w.m * 256) + (int)rank * 128, n0 = (int)(w.n * 256) + (int)rank * 128;
                for (int kb = 0; kb < p.nkb; ++kb) {
                    if (!fp8_wait(done0 + 8 * stage, phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + stage * kFp8PairStage, bar = full_leader + 8 * stage;
                    if (leader) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * kFp8PairStage);
                    tma_load_2d_pair(dst, &tm_a, kb * kFp8BK, m0, bar);
                    tma_load_2d_pair(dst + kFp8PairHalf, &tm_b, kb * kFp8BK, n0, bar);
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
                    if (issued & (1u << s)) mbar_wait(full0 + 8 * s, (last_par >> s) & 1u, kFp8WaitCycles);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMAs (even CTA); one commit a K block, to both CTAs
        if (leader) {
            constexpr uint32_t idesc = fp8_idesc<256, 256>();
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = cid; ok && u < tiles; u += ncl) {
                for (int kb = 0; kb < p.nkb; ++kb) {
                    ok = fp8_wait(full0 + 8 * stage, phase, abort_flag) &&
                         fp8_wait_cluster(tempty0 + 8 * acc, acc_phase ^ 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t addr = base + stage * kFp8PairStage;
                    const uint64_t da = fp8_desc(addr), db = fp8_desc(addr + kFp8PairHalf);
                    if (fp8_elect()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_fp8<true>(tmem + (uint32_t)acc * 256, da + 2 * k, db + 2 * k, idesc, k != 0 ? 1u : 0u);
                        fp8_commit_both(done0 + 8 * stage);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++acc == 2) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
            }
            if (fp8_elect()) umma_commit_pair(drain);
            __syncwarp();
            mbar_wait(drain, 0, kFp8WaitCycles);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------- epilogue: this CTA's 128 rows, 128 of the 256 columns a warp
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFp8ManyRegs));
        const int q = warp & 3, half = (warp - 4) >> 2, e = warp - 4;
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)half * 128;
        const uint32_t tempty_leader = map_to_rank(tempty0, 0);
        const uint32_t box = boxes + (uint32_t)e * 2 * kFp8Box, my_col = col_scales + (uint32_t)e * 512;
        constexpr uint32_t kColStep = 512 * kFp8EpiWarps;
        int acc = 0, stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t u = cid; ok && u < tiles; u += ncl) {
            const Fp8Tile w = fp8_tile(u, p);
            const int64_t mw = w.m * 256 + (int64_t)rank * 128 + q * 32, m = mw + lane, n0 = w.n * 256 + half * 128;
            // scales of rows and columns past the end are those of the last: what they scale is not
            // stored.  A row's (and a block's of B) are loaded two K blocks ahead.
            const float* sa = p.sa + (m < p.M ? m : p.M - 1);
            const float* sb = p.sb + ((n0 < p.N ? n0 : p.N - 1) >> p.b_shift);
            float sa_next = __ldg(sa), sb_next = kColVec ? 1.f : __ldg(sb), sa_then = sa_next, sb_then = sb_next;
            if (p.nkb > 1) {
                sa_then = __ldg(sa += p.lda);
                if (!kColVec) sb_then = __ldg(sb += p.ldb);
            }
            auto fetch = [&](int kb) {   // B's scales of a row each, to shared memory
                if (kb < p.nkb) {
                    const uint32_t to = my_col + (uint32_t)(kb % kFp8AheadCols) * kColStep;
                    const float* from = p.sb + kb * p.ldb;
                    if constexpr (kB == 2) {
                        const int64_t c = n0 + 4 * lane;
                        fp8_cp16(to + lane * 16, from + (c < p.N ? c : p.N - 4));
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int64_t c = n0 + lane + 32 * k;
                            fp8_cp4(to + (lane + 32 * k) * 4, from + (c < p.N ? c : p.N - 1));
                        }
                    }
                }
                fp8_cp_commit();
            };
            if constexpr (kColVec)
                for (int k = 0; k < kFp8AheadCols - 1; ++k) fetch(k);
            Fp8Sums<128, kColVec> sum;
#pragma unroll
            for (int j = 0; j < (kColVec ? 64 : 128); ++j) sum.s[j] = 0;
            // the next columns, of this or the next block, are on their way while kFp8Chunk are added
            // (by 32 columns 114 us where 16 take 105, by 8 111: registers).  What a lane's wait gave is
            // voted on at the block's end: all lanes go on or none (a vote in the wait took 105 us for 102)
            auto ready = [&]() {
                ok = fp8_wait_short(done0 + 8 * stage, phase, abort_flag);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                tc_fence_after();
                __syncwarp();
                return ok;
            };
            uint32_t r[2][kFp8Chunk];
            ok = __all_sync(0xffffffffu, ready());
            tmem_ld_ahead(lane_addr + (uint32_t)acc * 256, r[0]);
#pragma unroll 1
            for (int kb = 0; ok && kb < p.nkb; ++kb) {
                const float s = kColVec ? sa_next : __fmul_rn(sa_next, sb_next);
                sa_next = sa_then;
                sb_next = sb_then;
                if (kb + 2 < p.nkb) {
                    sa_then = __ldg(sa += p.lda);
                    if (!kColVec) sb_then = __ldg(sb += p.ldb);
                }
                if constexpr (kColVec) {
                    fetch(kb + kFp8AheadCols - 1);
                    fp8_cp_wait<kFp8AheadCols - 1>();
                    __syncwarp();
                }
                [[maybe_unused]] const u64 s2 = f2(s, s);
                const uint32_t scales = my_col + (uint32_t)(kb % kFp8AheadCols) * kColStep;
#pragma unroll
                for (int c = 0; c < 128 / kFp8Chunk; ++c) {
                    tmem_wait_ld();
                    if (c + 1 < 128 / kFp8Chunk) {
                        tmem_ld_ahead(lane_addr + (uint32_t)(acc * 256 + (c + 1) * kFp8Chunk), r[(c + 1) & 1]);
                    } else {   // all of the accumulator is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) fp8_arrive_cluster(tempty_leader + 8 * acc);
                        acc ^= 1;
                        if (kb + 1 < p.nkb) ready();
                        tmem_ld_ahead(lane_addr + (uint32_t)acc * 256, r[0]);   // the last time unused
                    }
#pragma unroll
                    for (int j = 0; j < kFp8Chunk / 4; ++j) {
                        const uint32_t* t = &r[c & 1][4 * j];
                        if constexpr (kColVec) {
                            const uint4 b = lds_v4(scales + (uint32_t)(c * kFp8Chunk + 4 * j) * 4);
                            u64* to = &sum.s[c * (kFp8Chunk / 2) + 2 * j];
                            fp8_add(to[0], s2, t[0], t[1], b.x, b.y);
                            fp8_add(to[1], s2, t[2], t[3], b.z, b.w);
                        } else {
                            float* to = &sum.s[c * kFp8Chunk + 4 * j];
#pragma unroll
                            for (int k = 0; k < 4; ++k) fp8_add(to[k], s, t[k]);
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, ok);   // this place's scales are read, and all lanes go on or none
            }
            tmem_wait_ld();   // the last load, which nothing reads, before its registers serve again
            if (ok) fp8_put_rows(p, &tm_c, mw, n0, sum, box, lane);
            if constexpr (kColVec) fp8_cp_wait<0>();
        }
        if (lane == 0) bulk_wait_read<0>();   // the boxes have been read
        __syncwarp();
    }
    tc_fence_before();
    cluster_sync_all();   // the peer's MMAs and copies reach into this CTA until it is done
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- a few tokens

// Epilogue warps: two a scheduler from 64 tokens on, half of the tokens each (128 x 151936 x 4096
// 159 us; 179 by one a scheduler).
template <int kBN>
constexpr int kFp8TokEpi = kBN >= 64 ? 8 : 4;
template <int kBN>
constexpr int kFp8TokThreads = 64 + 32 * kFp8TokEpi<kBN>;
constexpr int kFp8TokAccs = 4;
constexpr int kFp8TokAhead = 8;
template <int kBN>
constexpr uint32_t kFp8TokStage = 128 * kFp8BK + kBN * kFp8BK;
template <int kBN>
constexpr int kFp8TokStages = kBN <= 32 ? 9 : kBN <= 64 ? 8 : 6;
// barriers, row scales (one a thread), column scales (those of its tokens a warp)
template <int kBN>
constexpr size_t kFp8TokSmem = 1024 + (size_t)kFp8TokStages<kBN> * kFp8TokStage<kBN> + 512 +
                               kFp8TokAhead * 32 * kFp8TokEpi<kBN> * 4 + kFp8TokAhead * 4 * kBN * 4;
static_assert(kFp8TokSmem<128> <= 232448 && kFp8TokSmem<16> <= 232448, "shared memory per CTA");

// Rows of the MMA: 128 rows of B a tile (tile u mod tiles_n), its columns: kBN rows of A.  Cluster
// rank r of S takes K blocks [r nkb / S, (r + 1) nkb / S); with S > 1 a cluster has one tile.
template <int kBN>
__global__ void __launch_bounds__(kFp8TokThreads<kBN>, 1)
k_fp8_tokens(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, Fp8Args p, int split) {
    constexpr int kStages = kFp8TokStages<kBN>;
    constexpr uint32_t kStage = kFp8TokStage<kBN>, kCols = kFp8TokAccs * kBN < 32 ? 32 : kFp8TokAccs * kBN;
    extern __shared__ __align__(1024) unsigned char fp8_smem[];
    const uint32_t raw = smem_u32(fp8_smem);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + kStages * kStage;
    const uint32_t full0 = bars, empty0 = bars + 8 * kStages;
    const uint32_t tfull0 = bars + 16 * kStages, tempty0 = tfull0 + 8 * kFp8TokAccs;
    const uint32_t drain = tempty0 + 8 * kFp8TokAccs, slot = drain + 8;
    constexpr int kEpi = kFp8TokEpi<kBN>, kCols1 = kBN * 4 / kEpi;   // tokens of a warp
    const uint32_t row_scales = bars + 512, col_scales = row_scales + kFp8TokAhead * 32 * kEpi * 4;
    unsigned char* slot_gen = fp8_smem + (slot - raw);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(slot_gen);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot_gen + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = split > 1 ? cluster_rank() : 0u;
    const int kb0 = (int)((int64_t)rank * p.nkb / split), kb1 = (int)((int64_t)(rank + 1) * p.nkb / split);
    const int64_t tiles = p.tiles_m * p.tiles_n, first = blockIdx.x / split, step = gridDim.x / split;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int a = 0; a < kFp8TokAccs; ++a) {
            mbar_init(tfull0 + 8 * a, 1);
            mbar_init(tempty0 + 8 * a, kEpi);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_a);
        prefetch_tmap(&tm_b);
    }
    if (warp == 1) {
        tmem_alloc(slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0, last_par = 0;
            bool ok = true;
            for (int64_t u = first; ok && u < tiles; u += step) {
                const int m0 = (int)(u % p.tiles_m) * kBN, n0 = (int)(u / p.tiles_m) * 128;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!fp8_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = base + stage * kStage;
                    mbar_arrive_expect_tx(full0 + 8 * stage, kStage);
                    tma_load_2d(dst, &tm_b, kb * kFp8BK, n0, full0 + 8 * stage);
                    tma_load_2d(dst + 128 * kFp8BK, &tm_a, kb * kFp8BK, m0, full0 + 8 * stage);
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
                    if (issued & (1u << s)) mbar_wait(full0 + 8 * s, (last_par >> s) & 1u, kFp8WaitCycles);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = fp8_idesc<128, kBN>();
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = first; ok && u < tiles; u += step) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!fp8_wait(full0 + 8 * stage, phase, abort_flag) ||
                        !fp8_wait(tempty0 + 8 * acc, acc_phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t addr = base + stage * kStage;
                    const uint64_t da = fp8_desc(addr), db = fp8_desc(addr + 128 * kFp8BK);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_fp8<false>(tmem + (uint32_t)(acc * kBN), da + 2 * k, db + 2 * k, idesc, k != 0 ? 1u : 0u);
                    umma_commit(empty0 + 8 * stage);
                    umma_commit(tfull0 + 8 * acc);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++acc == kFp8TokAccs) {
                        acc = 0;
                        acc_phase ^= 1u;
                    }
                }
            }
            umma_commit(drain);
            mbar_wait(drain, 0, kFp8WaitCycles);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, e = warp - 2, row = q * 32 + lane, part = e >> 2, t0 = part * kCols1;
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)t0;
        const uint32_t my_row = row_scales + (uint32_t)(e * 32 + lane) * 4;
        const uint32_t my_col = col_scales + (uint32_t)e * (kCols1 * 4);
        constexpr uint32_t kRowStep = 32 * kEpi * 4, kColStep = 4 * kBN * 4;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int64_t u = first; ok && u < tiles; u += step) {
            const int64_t m0 = u % p.tiles_m * kBN + t0, n = u / p.tiles_m * 128 + row;
            const float* sb = p.sb + ((n < p.N ? n : p.N - 1) >> p.b_shift);
            auto fetch = [&](int kb) {
                if (kb < kb1) {
                    const uint32_t at = (uint32_t)(kb % kFp8TokAhead);
                    fp8_cp4(my_row + at * kRowStep, sb + kb * p.ldb);
#pragma unroll
                    for (int k = 0; k < (kCols1 + 31) / 32; ++k) {
                        const int c = lane + 32 * k;
                        if (c < kCols1)
                            fp8_cp4(my_col + at * kColStep + c * 4,
                                    p.sa + kb * p.lda + (m0 + c < p.M ? m0 + c : p.M - 1));
                    }
                }
                fp8_cp_commit();
            };
            for (int k = 0; k < kFp8TokAhead - 1; ++k) fetch(kb0 + k);
            Fp8Sums<kCols1, true> sum;
#pragma unroll
            for (int j = 0; j < kCols1 / 2; ++j) sum.s[j] = 0;
#pragma unroll 1
            for (int kb = kb0; kb < kb1; ++kb) {
                fetch(kb + kFp8TokAhead - 1);
                fp8_cp_wait<kFp8TokAhead - 1>();
                __syncwarp();
                const uint32_t at = (uint32_t)(kb % kFp8TokAhead);
                const float s = fp8_lds(my_row + at * kRowStep);
                const u64 s2 = f2(s, s);
                ok = __all_sync(0xffffffffu, fp8_wait(tfull0 + 8 * acc, acc_phase, abort_flag));
                if (!ok) break;   // all lanes, or none
                tc_fence_after();
                uint32_t r[2][16];
                tmem_ld_ahead(lane_addr + (uint32_t)(acc * kBN), r[0]);
#pragma unroll
                for (int c = 0; c < kCols1 / 16; ++c) {
                    tmem_wait_ld();
                    if (c < kCols1 / 16 - 1) {
                        tmem_ld_ahead(lane_addr + (uint32_t)(acc * kBN + (c + 1) * 16), r[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t* t = &r[c & 1][4 * j];
                        u64* to = &sum.s[c * 8 + 2 * j];
                        const uint4 b = lds_v4(my_col + at * kColStep + (uint32_t)(c * 16 + 4 * j) * 4);
                        fp8_add(to[0], s2, t[0], t[1], b.x, b.y);
                        fp8_add(to[1], s2, t[2], t[3], b.z, b.w);
                    }
                }
                __syncwarp();   // this place's scales are read
                if (++acc == kFp8TokAccs) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            fp8_cp_wait<0>();
            if (split > 1) {
                // this rank's sums, [column][row], over the ring: its copies have all been read
                // (the last MMA is committed to the accumulator that was just waited for)
                if (ok) {
                    float* at = reinterpret_cast<float*>(fp8_smem + (base - raw)) + t0 * 128 + row;
#pragma unroll
                    for (int j = 0; j < kCols1; ++j) at[j * 128] = sum.get(j);
                }
            } else if (ok && n < p.N) {
#pragma unroll
                for (int j = 0; j < kCols1; ++j)
                    if (m0 + j < p.M) fp8_put_one(p, (m0 + j) * p.ldc + n, sum.get(j));
            }
        }
    }
    if (split > 1) {
        tc_fence_before();
        cluster_sync_all();   // every rank's sums are there
        if (warp >= 2) {
            // a warp has a column of its rank's part, a lane four rows, all ranks' loads in flight
            // (by single values and one warp a column's part 256 x 4096 x 4096 took 24 us, 17 so)
            const int64_t m0 = first % p.tiles_m * kBN, n = first / p.tiles_m * 128 + 4 * lane;
            const int c0 = (int)rank * kBN / split, c1 = ((int)rank + 1) * kBN / split;
#pragma unroll 2
            for (int c = c0 + warp - 2; c < c1; c += kEpi) {
                float4 v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < split)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                                     : "r"(map_to_rank(base, (uint32_t)r) + (uint32_t)(c * 128 + 4 * lane) * 4));
                float4 s = v[0];   // in the order of the K blocks
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < split) {
                        s.x = __fadd_rn(s.x, v[r].x);
                        s.y = __fadd_rn(s.y, v[r].y);
                        s.z = __fadd_rn(s.z, v[r].z);
                        s.w = __fadd_rn(s.w, v[r].w);
                    }
                if (m0 + c < p.M) {
                    const int64_t at = (m0 + c) * p.ldc + n;
                    if (n < p.N) fp8_put_one(p, at, s.x);
                    if (n + 1 < p.N) fp8_put_one(p, at + 1, s.y);
                    if (n + 2 < p.N) fp8_put_one(p, at + 2, s.z);
                    if (n + 3 < p.N) fp8_put_one(p, at + 3, s.w);
                }
            }
        }
        cluster_sync_all();   // and read
    } else {
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// Self-test of the waits: a warp waits for what nothing does, with the CTA's abort flag set from the
// start or not (then by the short wait alone, until the clock's next tick).
static __device__ int g_fp8_selftest;
static __global__ void __launch_bounds__(32) k_fp8_wait_selftest(int aborted) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int flag;
    const uint32_t b = smem_u32(&bar);
    if (threadIdx.x == 0) {
        mbar_init(b, 1);
        fence_mbar_init();
        flag = aborted;
    }
    __syncwarp();
    bool done = fp8_wait_short<1>(b, 0, &flag);
    if (aborted) done = fp8_wait(b, 0, &flag) || fp8_wait_cluster(b, 0, &flag) || done;
    done = __any_sync(0xffffffffu, done);
    if (threadIdx.x == 0) g_fp8_selftest = done ? 0 : 1;
}

}  // namespace flp
