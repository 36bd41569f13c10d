// Preference loss on pairs of packed sequences of selected-token logp.
//
// With r_s = sum over the active tokens of sequence s of (logp - ref)
// (divided by their number n_s when averaging), h = r_chosen - r_rejected,
// u = beta h - margin and sigma the logistic function, the loss of a pair is
//   sigmoid  -(1 - e) log sigma(u) - e log sigma(-u)   (label smoothing e)
//   hinge    max(0, 1 - u)
//   ipo      (h - 1/(2 beta))^2
// and the batch's the sum over the live pairs (both sides have an active
// token) divided by their number D.  The gradient of token t of sequence s is
// +-(dl/dh) / D, divided by n_s when averaging.
//
// One cooperative launch (all CTAs are resident, so every barrier ends), three phases
// with a barrier of the grid between them.
// Sums: the batch is cut into fixed chunks of 512 tokens; a warp takes a run of
// consecutive chunks and writes, for every sequence that a chunk meets, the sum and
// the active count into slot (chunk + sequence).  Along the packed batch each next
// piece moves to the next chunk, the next sequence or both, so slots never collide and
// a sequence's pieces lie side by side.  Pairs: 8 (or 32) lanes per pair add both
// sides' slots as two-float sums and form the loss and the sequences' coefficients;
// the loss and D are folded in a fixed order.  Grad: the warps write their chunks'
// gradients.  Nothing depends on timing.
//
// A run's window holds the bounds (and coefficients) of 31 sequences, one a lane, so
// that a chunk reads no bounds from memory.  The whole warp takes a long piece, one
// after the other; short ones (32 tokens at most) are taken by a lane each, all at
// once, out of shared memory.  The next chunk's tokens are copied into shared memory
// while this one's are summed.
//
// What bounds it: at 16.8 M tokens in 16384 sequences (218 MB in 50 us, 4.4 TB/s) the
// sums 28 us, by instructions and memory alike, the pairs 7, a chain of latencies, the
// gradients 16, out of L2; small batches take 13 us, latencies.  As three dependent
// launches these took 49.5 and 11, but a caller's queue of calls was bound by the
// launches (31 us a call on 2.5 M tokens, now 25).
#pragma once

#include <cooperative_groups.h>
#include <math.h>
#include <stdint.h>

namespace flp {

constexpr int kPrefChunk = 512;        // tokens per warp and step
constexpr int kPrefQuads = kPrefChunk / 128;   // groups of four neighbouring tokens a lane holds of it
constexpr int kPrefThreads = 256;
constexpr int kPrefCtas = 3;           // per SM
constexpr int kPrefMaxCtas = 608;      // most CTAs of a launch
// A window with at least kPrefBriefs pieces of at most kPrefShort tokens has them taken
// by a lane each (8192 pairs x 4 tokens: 113 us by whole warps, now 21; taking every short
// piece so, the odd cut end of a long sequence too, cost 3 us on long batches).
constexpr int kPrefShort = 32, kPrefBriefs = 4;

enum PrefKind { kPrefSigmoid = 0, kPrefHinge = 1, kPrefIpo = 2 };

struct PrefSlot {
    float sum;
    int count;
};

// An unevaluated sum of two FP32 numbers: about 48 bits.  (FP64 adds, at 1/64 of
// the FP32 rate, took most of the pair phase.)
struct PrefTwo {
    float hi, lo;
};
__device__ __forceinline__ PrefTwo pref_add(PrefTwo x, float y) {   // Knuth's TwoSum
    const float s = __fadd_rn(x.hi, y), b = __fsub_rn(s, x.hi);
    return {s, __fadd_rn(x.lo, __fadd_rn(__fsub_rn(x.hi, __fsub_rn(s, b)), __fsub_rn(y, b)))};
}
__device__ __forceinline__ PrefTwo pref_add(PrefTwo x, PrefTwo y) {
    PrefTwo r = pref_add(x, y.hi);
    r.lo = __fadd_rn(r.lo, y.lo);
    return r;
}
// An infinite or NaN hi makes lo meaningless (inf - inf): keep hi alone.
__device__ __forceinline__ PrefTwo pref_settle(PrefTwo x) { return isfinite(x.hi) ? x : PrefTwo{x.hi, 0.f}; }
__device__ __forceinline__ float pref_value(PrefTwo x) {
    x = pref_settle(x);
    return x.hi + x.lo;
}

struct PrefArgs {
    const float *logp, *ref;      // ref nullable
    const uint8_t* mask;          // nullable
    const int64_t* cu;            // [nseq + 1]
    int64_t n, nseq, nchunks;
    int kind, average, halves;
    float beta, smooth, margin, normalizer;
    float target_hi, target_lo;   // 1 / (2 beta) as two floats
    float *loss, *grad, *rewards;
    // workspace
    int* live;                    // live pairs
    PrefTwo* part_loss;           // [kPrefMaxCtas]
    PrefSlot* slots;              // [nchunks + nseq]
    float* coef;                  // [nseq] dl/dr before the division by D
};

// Sequence bounds, clamped to the batch.
__device__ __forceinline__ int64_t pref_cu(const PrefArgs& a, int64_t i) {
    const int64_t v = __ldg(a.cu + i);
    return v < 0 ? 0 : (v > a.n ? a.n : v);
}

// Number of sequences that end at or before `pos` (32 probes a step).
__device__ __forceinline__ int64_t pref_first_seq(const PrefArgs& a, int64_t pos) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = a.nseq;   // the answer lies in [lo, hi]
    while (hi > lo) {
        const int64_t step = (hi - lo + 31) / 32;
        const int64_t i = lo + (int64_t)lane * step + step - 1;   // the lane's last sequence
        const bool before = i < hi && pref_cu(a, i + 1) <= pos;
        const int k = __popc(__ballot_sync(0xffffffffu, before));   // leading segments wholly before
        lo += (int64_t)k * step;
        const int64_t top = lo + step - 1;
        hi = top < hi ? top : hi;
        if (lo > hi) lo = hi;
    }
    return lo;
}

// The bounds of the sequences s0 .. s0 + 30 that a run of tokens [base, base + len)
// meets, relative to base and clamped to [-1, len + 1].
struct PrefWindow {
    int64_t s0;
    int32_t bound;    // lane l: start of sequence s0 + l
    float coef;       // lane l: coefficient of sequence s0 + l (grad phase)
};
template <bool kCoef>
__device__ __forceinline__ void pref_window(const PrefArgs& a, int64_t base, int64_t len, int64_t s, float inv_den,
                                            PrefWindow& c) {
    const int lane = threadIdx.x & 31;
    const int64_t i = s + lane;
    int64_t v = (a.nseq > 0 && i <= a.nseq ? pref_cu(a, i) : a.n) - base;   // no sequences: cu may be null
    v = v < -1 ? -1 : (v > len + 1 ? len + 1 : v);
    c.s0 = s;
    c.bound = (int32_t)v;
    c.coef = kCoef && i < a.nseq ? __ldcg(a.coef + i) * inv_den : 0.f;
}
// The pieces of the chunk [t, t + kPrefChunk) of the run, bounds relative to the chunk:
// every lane with a short one calls brief(sequence, lo, hi, coefficient) at the same
// time, the whole warp calls piece(sequence, lo, hi, coefficient) for every long one.
// `any_brief` runs in the whole warp before the lanes' calls.
template <bool kCoef, class A, class B, class F>
__device__ __forceinline__ void pref_walk(const PrefArgs& a, int64_t base, int64_t len, float inv_den, PrefWindow& c,
                                          int32_t t, A any_brief, B brief, F piece) {
    const int lane = threadIdx.x & 31;
    for (;;) {
        const int32_t end = __shfl_down_sync(0xffffffffu, c.bound, 1);
        const int32_t lo = c.bound > t ? c.bound - t : 0, hi = end < t + kPrefChunk ? end - t : kPrefChunk;
        const bool real = lane < 31 && c.s0 + lane < a.nseq && hi > lo;
        uint32_t left = __ballot_sync(0xffffffffu, real);
        const uint32_t briefs = __ballot_sync(0xffffffffu, real && hi - lo <= kPrefShort);
        if (__popc(briefs) >= kPrefBriefs) {
            any_brief();
            if ((briefs >> lane) & 1u) brief(c.s0 + lane, lo, hi, c.coef);
            __syncwarp();
            left &= ~briefs;
        }
        for (; left != 0; left &= left - 1) {
            const int k = __ffs(left) - 1;
            piece(c.s0 + k, __shfl_sync(0xffffffffu, lo, k), __shfl_sync(0xffffffffu, hi, k),
                  kCoef ? __shfl_sync(0xffffffffu, c.coef, k) : 0.f);
        }
        // on to the next window while this one ends inside the chunk
        const int32_t last = __shfl_sync(0xffffffffu, c.bound, 31);
        if (last >= t + kPrefChunk || c.s0 + 31 >= a.nseq) break;
        pref_window<kCoef>(a, base, len, c.s0 + 31, inv_den, c);
    }
}

// A lane's tokens of a chunk: quad h holds tokens h 128 + 4 lane .. + 3.
struct PrefRaw {
    float p[4 * kPrefQuads], q[4 * kPrefQuads];
    uint32_t m[kPrefQuads];   // mask bytes; 0 for tokens past the batch's end
};
__device__ __forceinline__ bool pref_active(const uint32_t (&m)[kPrefQuads], int j) {
    return (m[j >> 2] & (0xffu << (8 * (j & 3)))) != 0;
}
template <bool kVec>
__device__ __forceinline__ void pref_mask(const PrefArgs& a, int64_t t0, uint32_t (&m)[kPrefQuads]) {
    const int64_t i0 = t0 + (threadIdx.x & 31) * 4;
    if (kVec && t0 + kPrefChunk <= a.n) {
#pragma unroll
        for (int h = 0; h < kPrefQuads; ++h)
            m[h] = a.mask ? __ldg(reinterpret_cast<const uint32_t*>(a.mask + i0) + 32 * h) : 0x01010101u;
    } else {
#pragma unroll
        for (int h = 0; h < kPrefQuads; ++h) {
            m[h] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t i = i0 + h * 128 + k;
                if (i < a.n) m[h] |= (a.mask ? (uint32_t)__ldg(a.mask + i) : 1u) << (8 * k);
            }
        }
    }
}
__device__ __forceinline__ void pref_tokens(const float* x, int64_t t0, int64_t n, float (&v)[4 * kPrefQuads]) {
    const int64_t i0 = t0 + (threadIdx.x & 31) * 4;
#pragma unroll
    for (int j = 0; j < 4 * kPrefQuads; ++j) {
        const int64_t i = i0 + (j >> 2) * 128 + (j & 3);
        v[j] = i < n ? __ldcs(x + i) : 0.f;
    }
}
// A chunk that the ring does not hold: the batch's last, or any of unaligned arrays.
__device__ __forceinline__ void pref_load(const PrefArgs& a, int64_t t0, PrefRaw& r) {
    pref_tokens(a.logp, t0, a.n, r.p);
    if (a.ref) pref_tokens(a.ref, t0, a.n, r.q);
    pref_mask<false>(a, t0, r.m);
}

// Chunks [c0, c1) of warp `w` of `warps`.
__device__ __forceinline__ void pref_run(const PrefArgs& a, int64_t w, int64_t warps, int64_t& c0, int64_t& c1) {
    c0 = a.nchunks / warps * w + a.nchunks % warps * w / warps;
    c1 = a.nchunks / warps * (w + 1) + a.nchunks % warps * (w + 1) / warps;
}

// This lane's places in its warp's ring of kPrefStages chunks (thread-private:
// a lane copies and reads back only its own tokens, so no barrier is needed).
constexpr int kPrefStages = 2;
constexpr uint32_t kPrefStageBytes = kPrefThreads * kPrefQuads * (16 + 16 + 4);
// logp and ref are read once: first out of the L2 cache, so that the mask stays for
// the gradients' pass.
__device__ __forceinline__ uint64_t pref_read_once() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void pref_ring_issue(const PrefArgs& a, int64_t t0, uint32_t stage, uint64_t once) {
    const int lane = threadIdx.x & 31;
    const float *p = a.logp + t0 + lane * 4, *q = a.ref + t0 + lane * 4;
    const uint8_t* m = a.mask + t0 + lane * 4;
#pragma unroll
    for (int h = 0; h < kPrefQuads; ++h) {
        const uint32_t at = stage + (h * kPrefThreads + threadIdx.x) * 16;
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(at), "l"(p + 128 * h), "l"(once)
                     : "memory");
        if (a.ref)
            asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(
                             at + kPrefQuads * kPrefThreads * 16), "l"(q + 128 * h), "l"(once) : "memory");
        if (a.mask)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                             stage + kPrefQuads * kPrefThreads * 32 + (h * kPrefThreads + threadIdx.x) * 4),
                         "l"(m + 128 * h) : "memory");
    }
}
__device__ __forceinline__ void pref_ring_read(const PrefArgs& a, uint32_t stage, PrefRaw& r) {
#pragma unroll
    for (int h = 0; h < kPrefQuads; ++h) {
        const uint32_t at = stage + (h * kPrefThreads + threadIdx.x) * 16;
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(r.p[4 * h]), "=f"(r.p[4 * h + 1]), "=f"(r.p[4 * h + 2]), "=f"(r.p[4 * h + 3]) : "r"(at)
                     : "memory");
        if (a.ref)
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(r.q[4 * h]), "=f"(r.q[4 * h + 1]), "=f"(r.q[4 * h + 2]), "=f"(r.q[4 * h + 3])
                         : "r"(at + kPrefQuads * kPrefThreads * 16) : "memory");
        r.m[h] = 0x01010101u;
        if (a.mask)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.m[h])
                         : "r"(stage + kPrefQuads * kPrefThreads * 32 + (h * kPrefThreads + threadIdx.x) * 4)
                         : "memory");
    }
}
__device__ __forceinline__ int pref_bytes_set(uint32_t m) {
    return __popc((m | ((m & 0x7f7f7f7fu) + 0x7f7f7f7fu)) & 0x80808080u);
}
// Addresses in a stage of the warp's token q of a chunk (its value) and of its mask byte.
__device__ __forceinline__ uint32_t pref_token_at(uint32_t stage, int q) {
    return stage + ((q >> 7) * kPrefThreads + (threadIdx.x & ~31u) + ((q >> 2) & 31)) * 16 + (q & 3) * 4;
}
__device__ __forceinline__ uint32_t pref_mask_at(uint32_t stage, int q) {
    return stage + kPrefQuads * kPrefThreads * 32 + ((q >> 7) * kPrefThreads + (threadIdx.x & ~31u) + ((q >> 2) & 31)) * 4 +
           (q & 3);
}
// This lane's tokens to the stage, at their places.
__device__ __forceinline__ void pref_stage_tokens(uint32_t stage, const float (&v)[4 * kPrefQuads]) {
#pragma unroll
    for (int h = 0; h < kPrefQuads; ++h)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + (h * kPrefThreads + threadIdx.x) * 16),
                     "f"(v[4 * h]), "f"(v[4 * h + 1]), "f"(v[4 * h + 2]), "f"(v[4 * h + 3]) : "memory");
}

template <bool kVec>
__device__ __forceinline__ void pref_sums(const PrefArgs& a, int64_t w, int64_t warps, uint32_t ring) {
    const int lane = threadIdx.x & 31;
    int64_t c0, c1;
    pref_run(a, w, warps, c0, c1);
    if (c0 >= c1) return;
    const int64_t base = c0 * kPrefChunk, len = (c1 - c0) * kPrefChunk;
    const int64_t full = kVec ? a.n / kPrefChunk : 0;   // chunks before this are whole and copied ahead
    const uint64_t once = pref_read_once();
#pragma unroll
    for (int k = 0; k < kPrefStages - 1; ++k) {
        if (c0 + k < c1 && c0 + k < full) pref_ring_issue(a, base + k * kPrefChunk, ring + k * kPrefStageBytes, once);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    PrefWindow cur;
    pref_window<false>(a, base, len, pref_first_seq(a, base), 0.f, cur);
    int stage = 0;
    for (int64_t c = c0; c < c1; ++c) {
        PrefRaw r;
        const int64_t ahead = c + kPrefStages - 1;
        const int into = stage == 0 ? kPrefStages - 1 : stage - 1;
        if (ahead < c1 && ahead < full) pref_ring_issue(a, ahead * kPrefChunk, ring + into * kPrefStageBytes, once);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group %0;" ::"n"(kPrefStages - 1) : "memory");
        const uint32_t slot = ring + stage * kPrefStageBytes;
        if (c < full) pref_ring_read(a, slot, r);
        else pref_load(a, c * kPrefChunk, r);
        stage = stage == kPrefStages - 1 ? 0 : stage + 1;
        // a masked value is not used
        float v[4 * kPrefQuads], quad[kPrefQuads];
#pragma unroll
        for (int h = 0; h < kPrefQuads; ++h) {
#pragma unroll
            for (int j = 4 * h; j < 4 * h + 4; ++j)
                v[j] = pref_active(r.m, j) ? (a.ref ? r.p[j] - r.q[j] : r.p[j]) : 0.f;
            quad[h] = (v[4 * h] + v[4 * h + 1]) + (v[4 * h + 2] + v[4 * h + 3]);
        }
        bool staged = false;
        pref_walk<false>(
            a, base, len, 0.f, cur, (int32_t)((c - c0) * kPrefChunk),
            [&] {
                if (staged) return;
                staged = true;
                pref_stage_tokens(slot, v);
#pragma unroll
                for (int h = 0; h < kPrefQuads; ++h)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot + kPrefQuads * kPrefThreads * 32 +
                                                                 (h * kPrefThreads + threadIdx.x) * 4),
                                 "r"(r.m[h]) : "memory");
                __syncwarp();
            },
            [&](int64_t s, int32_t lo, int32_t hi, float) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                int cnt = 0;
                for (int q = lo; q < hi; q += 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (q + j < hi) {
                            float x;
                            unsigned short m;
                            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(pref_token_at(slot, q + j)) : "memory");
                            asm volatile("ld.shared.u8 %0, [%1];" : "=h"(m) : "r"(pref_mask_at(slot, q + j)) : "memory");
                            part[j] += x;
                            cnt += m != 0 ? 1 : 0;
                        }
                    }
                }
                a.slots[c + s] = PrefSlot{(part[0] + part[1]) + (part[2] + part[3]), cnt};
            },
            [&](int64_t s, int32_t lo, int32_t hi, float) {
                float sum = 0.f;
                int cnt = 0;
#pragma unroll
                for (int h = 0; h < kPrefQuads; ++h) {
                    const int q = h * 128 + lane * 4;
                    if (q >= lo && q + 4 <= hi) {
                        sum += quad[h];
                        cnt += pref_bytes_set(r.m[h]);
                    } else if (q + 4 > lo && q < hi) {   // a bound inside the quad: one lane or two
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (q + j >= lo && q + j < hi) {
                                sum += v[4 * h + j];
                                cnt += pref_active(r.m, 4 * h + j) ? 1 : 0;
                            }
                    }
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                cnt = __reduce_add_sync(0xffffffffu, cnt);
                if (lane == 0) a.slots[c + s] = PrefSlot{sum, cnt};
            });
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int kLanes, class T>
__device__ __forceinline__ T pref_group_sum(T v) {
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int kLanes>
__device__ __forceinline__ PrefTwo pref_group_sum(PrefTwo v) {
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) {
        // the same order in both lanes of an exchange, so that they get the same bits
        const PrefTwo w{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
        v = threadIdx.x & o ? pref_add(w, v) : pref_add(v, w);
    }
    return v;
}

// This lane's share of the sum and active tokens (a sequence may have more than 2^31)
// of the sequence [b, e).
template <int kLanes>
__device__ __forceinline__ void pref_sequence(const PrefArgs& a, int64_t s, int64_t b, int64_t e, PrefTwo& sum,
                                              int64_t& cnt) {
    sum = {0.f, 0.f};
    cnt = 0;
    if (e > b) {
        const int64_t c1 = (e - 1) / kPrefChunk;
        for (int64_t c = b / kPrefChunk + (threadIdx.x & (kLanes - 1)); c <= c1; c += kLanes) {
            const float2 q = __ldcg(reinterpret_cast<const float2*>(a.slots + c + s));
            sum = pref_add(sum, q.x);
            cnt += __float_as_int(q.y);
        }
    }
}

// Pairs `first`, first + step, ... (one per group of kLanes lanes): coefficients and
// rewards; this thread's share of the loss and of the live pairs.
template <int kLanes>
__device__ __forceinline__ void pref_pairs(const PrefArgs& a, int64_t first, int64_t step, PrefTwo& loss, int& live) {
    const int64_t pairs = a.nseq / 2;
    loss = {0.f, 0.f};
    live = 0;
    // every lane of the warp takes every turn (the sums are warp-wide shuffles)
    for (int64_t p0 = first; __any_sync(0xffffffffu, p0 < pairs); p0 += step) {
        const bool real = p0 < pairs;
        const int64_t p = real ? p0 : pairs - 1;
        const int64_t sc = a.halves ? p : 2 * p, sj = a.halves ? p + pairs : 2 * p + 1;
        const int64_t bc = pref_cu(a, sc), ec = pref_cu(a, sc + 1), bj = pref_cu(a, sj), ej = pref_cu(a, sj + 1);
        PrefTwo rc, rj;
        int64_t nc, nj;
        pref_sequence<kLanes>(a, sc, bc, ec, rc, nc);
        pref_sequence<kLanes>(a, sj, bj, ej, rj, nj);
        rc = pref_settle(pref_group_sum<kLanes>(rc));
        rj = pref_settle(pref_group_sum<kLanes>(rj));
        nc = pref_group_sum<kLanes>(nc);
        nj = pref_group_sum<kLanes>(nj);
        if (real && (threadIdx.x & (kLanes - 1)) == 0) {
            float wc = 1.f, wj = 1.f;
            if (a.average) {
                wc = nc > 0 ? __frcp_rn((float)nc) : 0.f;
                wj = nj > 0 ? __frcp_rn((float)nj) : 0.f;
                rc = {nc > 0 ? __fdiv_rn(rc.hi + rc.lo, (float)nc) : 0.f, 0.f};
                rj = {nj > 0 ? __fdiv_rn(rj.hi + rj.lo, (float)nj) : 0.f, 0.f};
            }
            float each = 0.f, dh = 0.f;
            if (nc > 0 && nj > 0) {
                PrefTwo h = pref_settle(pref_add(rc, PrefTwo{-rj.hi, -rj.lo}));
                if (a.kind == kPrefIpo) {
                    const float t = pref_value(pref_add(h, PrefTwo{-a.target_hi, -a.target_lo}));
                    each = t * t;
                    dh = 2.f * t;
                } else {
                    const float u = fmaf(a.beta, h.hi, fmaf(a.beta, h.lo, -a.margin));
                    if (a.kind == kPrefHinge) {
                        each = u != u ? u : fmaxf(0.f, 1.f - u);
                        dh = u != u ? u : (u < 1.f ? -a.beta : 0.f);
                    } else {
                        const float tail = log1pf(expf(-fabsf(u))), e = a.smooth;
                        // a weight of zero takes its side out (no 0 * inf)
                        each = tail + (e < 1.f && !(u >= 0.f) ? (1.f - e) * -u : 0.f) +
                               (e > 0.f && !(u <= 0.f) ? e * u : 0.f);
                        dh = a.beta * (e / (1.f + expf(-u)) - (1.f - e) / (1.f + expf(u)));
                    }
                }
                ++live;
                loss = pref_add(loss, each);
            }
            a.coef[sc] = dh * wc;
            a.coef[sj] = -dh * wj;
            a.rewards[2 * p] = a.beta * (rc.hi + rc.lo);
            a.rewards[2 * p + 1] = a.beta * (rj.hi + rj.lo);
        }
    }
}

// Sum of (l, k) over a CTA of kThreads, in thread 0, in a fixed order.
template <int kThreads>
__device__ __forceinline__ void pref_cta_sum(PrefTwo& l, int& k, PrefTwo* sl, int* sk) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    l = pref_group_sum<32>(l);
    k = pref_group_sum<32>(k);
    __syncthreads();
    if (lane == 0) {
        sl[warp] = l;
        sk[warp] = k;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        l = {0.f, 0.f};
        k = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            l = pref_add(l, sl[w]);
            k += sk[w];
        }
    }
}
__device__ __forceinline__ float pref_inv_den(const PrefArgs& a, int live) {
    return live > 0 ? __frcp_rn(a.normalizer > 0.f ? a.normalizer : (float)live) : 0.f;
}
__device__ __forceinline__ float pref_loss(const PrefArgs& a, PrefTwo loss, int live) {
    return live > 0 ? __fdiv_rn(pref_value(loss), a.normalizer > 0.f ? a.normalizer : (float)live) : 0.f;
}

// The gradients of warp w's chunks; `wait` returns 1 / D once it and the
// coefficients are there.
template <bool kVec, class F>
__device__ __forceinline__ void pref_grad(const PrefArgs& a, int64_t w, int64_t warps, uint32_t slot, F wait) {
    const int lane = threadIdx.x & 31;
    int64_t c0, c1;
    pref_run(a, w, warps, c0, c1);
    const int64_t base = c0 * kPrefChunk, len = (c1 - c0) * kPrefChunk;
    uint32_t next[kPrefQuads];
    int64_t s = 0;
    if (c0 < c1) {
        pref_mask<kVec>(a, base, next);
        s = pref_first_seq(a, base);
    }
    const float inv_den = wait();
    if (c0 >= c1) return;
    PrefWindow cur;
    pref_window<true>(a, base, len, s, inv_den, cur);
    for (int64_t c = c0; c < c1; ++c) {
        const int64_t t0 = c * kPrefChunk;
        uint32_t m[kPrefQuads];
#pragma unroll
        for (int h = 0; h < kPrefQuads; ++h) m[h] = next[h];
        if (c + 1 < c1) pref_mask<kVec>(a, t0 + kPrefChunk, next);
        float v[4 * kPrefQuads] = {};
        bool staged = false;
        pref_walk<true>(
            a, base, len, inv_den, cur, (int32_t)((c - c0) * kPrefChunk),
            [&] {
                if (staged) return;
                staged = true;
                const float zeros[4 * kPrefQuads] = {};
                pref_stage_tokens(slot, zeros);
                __syncwarp();
            },
            [&](int64_t, int32_t lo, int32_t hi, float g) {
                for (int q = lo; q < hi; ++q)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(pref_token_at(slot, q)), "f"(g) : "memory");
            },
            [&](int64_t, int32_t lo, int32_t hi, float g) {
#pragma unroll
                for (int h = 0; h < kPrefQuads; ++h) {
                    const int q = h * 128 + lane * 4;
                    if (q >= lo && q + 4 <= hi) {
                        v[4 * h] = v[4 * h + 1] = v[4 * h + 2] = v[4 * h + 3] = g;
                    } else if (q + 4 > lo && q < hi) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (q + j >= lo && q + j < hi) v[4 * h + j] = g;
                    }
                }
            });
        if (staged) {   // a token is in a short piece, a long one or none
#pragma unroll
            for (int h = 0; h < kPrefQuads; ++h) {
                float x[4];
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                             : "r"(slot + (h * kPrefThreads + threadIdx.x) * 16) : "memory");
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] += x[j];
            }
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 4 * kPrefQuads; ++j) v[j] = pref_active(m, j) ? v[j] : 0.f;
        const int64_t i0 = t0 + lane * 4;
        if (kVec && t0 + kPrefChunk <= a.n) {
#pragma unroll
            for (int h = 0; h < kPrefQuads; ++h)
                __stcs(reinterpret_cast<float4*>(a.grad + i0) + 32 * h,
                       make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4 * kPrefQuads; ++j) {
                const int64_t i = i0 + (j >> 2) * 128 + (j & 3);
                if (i < a.n) a.grad[i] = v[j];
            }
        }
    }
}

template <bool kVec>
__global__ void __launch_bounds__(kPrefThreads, kPrefCtas)
k_pref(PrefArgs a, int narrow) {
    __shared__ PrefTwo sl[kPrefThreads / 32];
    __shared__ int sk[kPrefThreads / 32];
    extern __shared__ __align__(16) unsigned char pref_smem[];
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(pref_smem);
    const auto grid = cooperative_groups::this_grid();
    const int64_t w = (int64_t)blockIdx.x * (kPrefThreads / 32) + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)gridDim.x * (kPrefThreads / 32);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.live = 0;
    pref_sums<kVec>(a, w, warps, ring);
    grid.sync();
    PrefTwo l;
    int k;
    if (narrow) {
        constexpr int kGroups = kPrefThreads / 8;
        pref_pairs<8>(a, (int64_t)blockIdx.x * kGroups + threadIdx.x / 8, (int64_t)gridDim.x * kGroups, l, k);
    } else {
        pref_pairs<32>(a, w, warps, l, k);
    }
    pref_cta_sum<kPrefThreads>(l, k, sl, sk);
    if (threadIdx.x == 0) {
        a.part_loss[blockIdx.x] = l;
        if (k > 0) atomicAdd(a.live, k);   // whole numbers: any order gives the same sum
    }
    pref_grad<kVec>(a, w, warps, ring, [&] {
        grid.sync();
        return pref_inv_den(a, __ldcg(a.live));
    });
    if (blockIdx.x == gridDim.x - 1) {   // the loss, in an order fixed by the grid
        l = {0.f, 0.f};
        for (int i = threadIdx.x; i < (int)gridDim.x; i += kPrefThreads) {
            const float2 q = __ldcg(reinterpret_cast<const float2*>(a.part_loss + i));
            l = pref_add(l, PrefTwo{q.x, q.y});
        }
        k = 0;
        pref_cta_sum<kPrefThreads>(l, k, sl, sk);
        if (threadIdx.x == 0) *a.loss = pref_loss(a, l, __ldcg(a.live));
    }
}

}  // namespace flp
