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
// Three launches.  Sums: the batch is cut into fixed chunks of 256 tokens, one
// warp each; a chunk writes the sum and the active count of every sequence it
// meets into slot (chunk + sequence).  Along the packed batch each next piece
// moves to the next chunk, the next sequence or both, so slots never collide
// and a sequence's pieces lie side by side.  Pairs: a warp per pair adds both
// sides' slots in FP64 and forms the loss and the sequences' coefficients; the
// last CTA folds the loss and D.  Grad: a warp per chunk writes the gradients.
// Nothing depends on timing.
#pragma once

#include <math.h>
#include <stdint.h>

namespace flp {

constexpr int kPrefChunk = 256;        // tokens per warp and step
constexpr int kPrefThreads = 256;
constexpr int kPrefPairCtas = 1024;    // most CTAs of the pair kernel (the fold's shape)

enum PrefKind { kPrefSigmoid = 0, kPrefHinge = 1, kPrefIpo = 2 };

struct PrefSlot {
    float sum;
    int count;
};

struct PrefArgs {
    const float *logp, *ref;      // ref nullable
    const uint8_t* mask;          // nullable
    const int64_t* cu;            // [nseq + 1]
    int64_t n, nseq, nchunks;
    int kind, average, halves;
    float beta, smooth, margin, normalizer;
    float *loss, *grad, *rewards;
    // workspace
    unsigned* ticket;
    float* inv_den;
    double* part_loss;            // [kPrefPairCtas]
    int64_t* part_live;           // [kPrefPairCtas]
    PrefSlot* slots;              // [nchunks + nseq]
    int32_t* first_seq;           // [nchunks] first sequence that ends after the chunk's start
    float* coef;                  // [nseq] dl/dr before the division by D
};

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// Token j of lane in a chunk: four neighbours in each half.
__device__ __forceinline__ int pref_tok(int lane, int j) { return (j >> 2) * 128 + lane * 4 + (j & 3); }

__device__ __forceinline__ void pref_load4(const float* p, int64_t i, int64_t n, bool vec, float (&v)[4]) {
    if (vec && i + 4 <= n) {
        const float4 q = __ldcs(reinterpret_cast<const float4*>(p + i));
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < n ? __ldcs(p + i + k) : 0.f;
    }
}
// Bit k: token i + k exists and is active.
__device__ __forceinline__ uint32_t pref_mask4(const uint8_t* m, int64_t i, int64_t n, bool vec) {
    uint32_t bits = 0;
    if (m != nullptr && vec && i + 4 <= n) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(m + i));
#pragma unroll
        for (int k = 0; k < 4; ++k) bits |= ((w >> (8 * k)) & 0xffu) ? (1u << k) : 0u;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n && (m == nullptr || __ldg(m + i + k) != 0)) bits |= 1u << k;
    }
    return bits;
}

template <bool kVec>
__global__ void __launch_bounds__(kPrefThreads)
k_pref_sums(PrefArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kPrefThreads / 32);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    for (int64_t c = (int64_t)blockIdx.x * (kPrefThreads / 32) + (threadIdx.x >> 5); c < a.nchunks; c += warps) {
        const int64_t t0 = c * kPrefChunk, t1 = t0 + kPrefChunk < a.n ? t0 + kPrefChunk : a.n;
        float v[8];
        uint32_t bits = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = t0 + h * 128 + lane * 4;
            float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
            pref_load4(a.logp, i, a.n, kVec, p);
            if (a.ref) pref_load4(a.ref, i, a.n, kVec, q);
            const uint32_t m = pref_mask4(a.mask, i, a.n, kVec);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * h + k] = (m >> k) & 1u ? p[k] - q[k] : 0.f;   // a masked value is not read
            bits |= m << (4 * h);
        }
        int64_t s = pref_first_seq(a, t0);
        if (lane == 0) a.first_seq[c] = (int32_t)s;
        int64_t b = s < a.nseq ? pref_cu(a, s) : t1;
        while (s < a.nseq && b < t1) {
            const int64_t e = pref_cu(a, s + 1);
            if (e > b && e > t0) {
                float sum = 0.f;
                int cnt = 0;
                const int lo = b > t0 ? (int)(b - t0) : 0, hi = e < t1 ? (int)(e - t0) : kPrefChunk;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = pref_tok(lane, j);
                    if (k >= lo && k < hi) {
                        sum += v[j];
                        cnt += (bits >> j) & 1u;
                    }
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
                }
                if (lane == 0) a.slots[c + s] = PrefSlot{sum, cnt};
            }
            b = e;
            ++s;
        }
    }
}

// (sum, active tokens) of sequence s, in every lane.
__device__ __forceinline__ void pref_sequence(const PrefArgs& a, int64_t s, double& sum, int64_t& cnt) {
    const int lane = threadIdx.x & 31;
    const int64_t b = pref_cu(a, s), e = pref_cu(a, s + 1);
    sum = 0.0;
    cnt = 0;
    if (e > b) {
        const int64_t c1 = (e - 1) / kPrefChunk;
        for (int64_t c = b / kPrefChunk + lane; c <= c1; c += 32) {
            const PrefSlot q = a.slots[c + s];
            sum += (double)q.sum;
            cnt += q.count;
        }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
    }
}

__global__ void __launch_bounds__(kPrefThreads)
k_pref_pairs(PrefArgs a) {
    __shared__ double s_loss[kPrefThreads / 32];
    __shared__ int64_t s_live[kPrefThreads / 32];
    __shared__ bool s_last;
    grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t pairs = a.nseq / 2;
    double loss = 0.0;
    int64_t live = 0;
    for (int64_t p = (int64_t)blockIdx.x * (kPrefThreads / 32) + warp; p < pairs;
         p += (int64_t)gridDim.x * (kPrefThreads / 32)) {
        const int64_t sc = a.halves ? p : 2 * p, sj = a.halves ? p + pairs : 2 * p + 1;
        double rc, rj;
        int64_t nc, nj;
        pref_sequence(a, sc, rc, nc);
        pref_sequence(a, sj, rj, nj);
        if (lane == 0) {
            float wc = 1.f, wj = 1.f;
            if (a.average) {
                rc = nc > 0 ? rc / (double)nc : 0.0;
                rj = nj > 0 ? rj / (double)nj : 0.0;
                wc = nc > 0 ? 1.f / (float)nc : 0.f;
                wj = nj > 0 ? 1.f / (float)nj : 0.f;
            }
            float each = 0.f, dh = 0.f;
            if (nc > 0 && nj > 0) {
                const double h = rc - rj;
                if (a.kind == kPrefIpo) {
                    const float t = (float)(h - 0.5 / (double)a.beta);
                    each = t * t;
                    dh = 2.f * t;
                } else {
                    const float u = (float)((double)a.beta * h - (double)a.margin);
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
                loss += (double)each;
            }
            a.coef[sc] = dh * wc;
            a.coef[sj] = -dh * wj;
            a.rewards[2 * p] = (float)((double)a.beta * rc);
            a.rewards[2 * p + 1] = (float)((double)a.beta * rj);
        }
    }
    if (lane == 0) {
        s_loss[warp] = loss;
        s_live[warp] = live;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double l = 0.0;
        int64_t k = 0;
        for (int w = 0; w < kPrefThreads / 32; ++w) {
            l += s_loss[w];
            k += s_live[w];
        }
        a.part_loss[blockIdx.x] = l;
        a.part_live[blockIdx.x] = k;
        __threadfence();
        s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (!s_last) return;
    // the last CTA: fold in an order fixed by the grid
    double l = 0.0;
    int64_t k = 0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += kPrefThreads) {
        l += __ldcg(a.part_loss + i);
        k += __ldcg(a.part_live + i);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        k += __shfl_xor_sync(0xffffffffu, k, o);
    }
    if (lane == 0) {
        s_loss[warp] = l;
        s_live[warp] = k;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        l = 0.0;
        k = 0;
        for (int w = 0; w < kPrefThreads / 32; ++w) {
            l += s_loss[w];
            k += s_live[w];
        }
        const double den = a.normalizer > 0.f ? (double)a.normalizer : (double)k;
        *a.inv_den = k > 0 ? (float)(1.0 / den) : 0.f;
        *a.loss = k > 0 ? (float)(l / den) : 0.f;
    }
}

template <bool kVec>
__global__ void __launch_bounds__(kPrefThreads)
k_pref_grad(PrefArgs a) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kPrefThreads / 32);
    const float inv_den = __ldcg(a.inv_den);
    for (int64_t c = (int64_t)blockIdx.x * (kPrefThreads / 32) + (threadIdx.x >> 5); c < a.nchunks; c += warps) {
        const int64_t t0 = c * kPrefChunk, t1 = t0 + kPrefChunk < a.n ? t0 + kPrefChunk : a.n;
        uint32_t bits = pref_mask4(a.mask, t0 + lane * 4, a.n, kVec);
        bits |= pref_mask4(a.mask, t0 + 128 + lane * 4, a.n, kVec) << 4;
        float v[8] = {};
        int64_t s = a.first_seq[c];
        int64_t b = s < a.nseq ? pref_cu(a, s) : t1;
        while (s < a.nseq && b < t1) {
            const int64_t e = pref_cu(a, s + 1);
            if (e > b && e > t0) {
                const float g = __ldcg(a.coef + s) * inv_den;
                const int lo = b > t0 ? (int)(b - t0) : 0, hi = e < t1 ? (int)(e - t0) : kPrefChunk;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = pref_tok(lane, j);
                    if (k >= lo && k < hi && ((bits >> j) & 1u)) v[j] = g;
                }
            }
            b = e;
            ++s;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = t0 + h * 128 + lane * 4;
            if (kVec && i + 4 <= a.n) {
                __stcs(reinterpret_cast<float4*>(a.grad + i),
                       make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k < a.n) a.grad[i + k] = v[4 * h + k];
            }
        }
    }
}

}  // namespace flp
