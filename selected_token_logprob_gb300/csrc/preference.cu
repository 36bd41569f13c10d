// Host side of the preference loss (logp_preference_loss): argument checks,
// workspace layout and launches.
#include <math.h>

#include "host_common.h"
#include "preference_kernels.cuh"

using namespace flp_host;

namespace {

// Byte offsets of the workspace's parts; false when they overflow.
struct PrefLayout {
    int64_t part_loss, slots, coef, total;
};

bool pref_layout(int64_t n, int64_t nseq, PrefLayout* l) {
    const int64_t nchunks = n / flp::kPrefChunk + (n % flp::kPrefChunk != 0);
    int64_t slots, b;
    if (__builtin_add_overflow(nchunks, nseq, &slots) || slots > INT64_MAX / 32) return false;
    l->part_loss = 256;   // the live pairs
    l->slots = l->part_loss + 8 * flp::kPrefMaxCtas;
    l->coef = l->slots + 8 * slots;
    if (__builtin_add_overflow(l->coef, 4 * nseq + 255, &b)) return false;
    l->total = b / 256 * 256;
    return true;
}

flp_status check_pref_counts(int64_t n, int64_t num_seqs) {
    if (n < 0) return fail(FLP_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (num_seqs < 0 || num_seqs >= INT32_MAX || num_seqs % 2 != 0)
        return fail(FLP_EINVAL, "num_seqs must be even and in [0, 2^31 - 1) (got %lld)", (long long)num_seqs);
    return FLP_OK;
}

}  // namespace

extern "C" {

flp_status logp_preference_loss_workspace_size(int64_t n, int64_t num_seqs, int64_t* bytes) {
    if (bytes == nullptr) return fail(FLP_EINVAL, "bytes is a null pointer");
    flp_status st;
    if ((st = check_pref_counts(n, num_seqs)) != FLP_OK) return st;
    PrefLayout l;
    if (!pref_layout(n, num_seqs, &l)) return fail(FLP_EINVAL, "workspace size overflows int64");
    *bytes = l.total;
    return ok();
}

flp_status logp_preference_loss(const float* logp, const float* ref_logp, const uint8_t* active_mask,
                                const int64_t* cu_seqlens, int64_t num_seqs, int64_t n, int kind, int layout,
                                int average, float beta, float label_smoothing, float margin, float normalizer,
                                void* workspace, int64_t workspace_bytes, float* loss, float* grad, float* rewards,
                                flp_stream_t stream) {
    flp_status st;
    if ((st = check_pref_counts(n, num_seqs)) != FLP_OK) return st;
    if (kind < FLP_PREF_SIGMOID || kind > FLP_PREF_IPO) return fail(FLP_EINVAL, "kind must be 0, 1 or 2 (got %d)", kind);
    if (layout != FLP_PREF_INTERLEAVED && layout != FLP_PREF_HALVES)
        return fail(FLP_EINVAL, "layout must be 0 or 1 (got %d)", layout);
    if (!(beta > 0.f) || !isfinite(beta)) return fail(FLP_EINVAL, "beta must be finite and > 0 (got %g)", (double)beta);
    if (!(label_smoothing >= 0.f && label_smoothing <= 1.f) || (kind != FLP_PREF_SIGMOID && label_smoothing != 0.f))
        return fail(FLP_EINVAL, "label_smoothing must be in [0, 1], and 0 unless the kind is sigmoid (got %g)",
                    (double)label_smoothing);
    if (!isfinite(margin) || (kind == FLP_PREF_IPO && margin != 0.f))
        return fail(FLP_EINVAL, "margin must be finite, and 0 for the ipo kind (got %g)", (double)margin);
    if (!(normalizer >= 0.f) || !isfinite(normalizer))
        return fail(FLP_EINVAL, "normalizer must be finite and >= 0 (got %g)", (double)normalizer);
    PrefLayout l;
    if (!pref_layout(n, num_seqs, &l)) return fail(FLP_EINVAL, "workspace size overflows int64");
    if (workspace_bytes < l.total)
        return fail(FLP_EINVAL, "workspace_bytes (%lld) is below the %lld bytes needed", (long long)workspace_bytes,
                    (long long)l.total);
    if (!aligned16(workspace)) return fail(FLP_EINVAL, "workspace must start on a 16-byte boundary");
    const bool tokens = n > 0, seqs = num_seqs > 0;
    const void* ptrs[] = {loss, workspace, tokens ? logp : nullptr, tokens ? grad : nullptr,
                          seqs ? cu_seqlens : nullptr, seqs ? rewards : nullptr, tokens ? ref_logp : nullptr,
                          tokens ? active_mask : nullptr};
    const char* names[] = {"loss", "workspace", "logp", "grad", "cu_seqlens", "rewards", "ref_logp", "active_mask"};
    const bool optional[] = {false, false, !tokens, !tokens, !seqs, !seqs, true, true};
    int dev;
    if ((st = common_device(8, ptrs, names, optional, &dev)) != FLP_OK) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(FLP_ECUDA, "device index %d out of range", dev);
    DeviceGuard guard;
    if ((st = guard.enter(dev)) != FLP_OK) return st;
    const int sms = sm_count(dev);
    if (sms <= 0) return fail(FLP_ECUDA, "could not read the SM count of device %d", dev);
    flp::PrefArgs a;
    a.logp = logp;
    a.ref = ref_logp;
    a.mask = active_mask;
    a.cu = cu_seqlens;
    a.n = n;
    a.nseq = num_seqs;
    a.nchunks = ceil_div(n, flp::kPrefChunk);
    a.kind = kind;
    a.average = average != 0;
    a.halves = layout == FLP_PREF_HALVES;
    a.beta = beta;
    a.smooth = label_smoothing;
    a.margin = margin;
    a.normalizer = normalizer;
    const double target = 0.5 / (double)beta;
    a.target_hi = (float)target;
    a.target_lo = isfinite(a.target_hi) ? (float)(target - (double)a.target_hi) : 0.f;
    a.loss = loss;
    a.grad = grad;
    a.rewards = rewards;
    char* base = static_cast<char*>(workspace);
    a.live = reinterpret_cast<int*>(base);
    a.part_loss = reinterpret_cast<flp::PrefTwo*>(base + l.part_loss);
    a.slots = reinterpret_cast<flp::PrefSlot*>(base + l.slots);
    a.coef = reinterpret_cast<float*>(base + l.coef);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = aligned16(logp) && aligned16(ref_logp) && aligned16(grad) &&
                     (reinterpret_cast<uintptr_t>(active_mask) & 3u) == 0;
    // 8 lanes per pair while a sequence has a few slots, a warp beyond that (8192 pairs
    // x 1024 tokens: 50 and 60 us; 501 x 5000: 22 and 21; 64 x 60000: 32 and 28)
    const bool narrow = a.nchunks <= 16 * num_seqs;
    // A chunk a warp, a pair a group of lanes, up to the CTAs that can be resident.
    constexpr int kRing = flp::kPrefStages * (int)flp::kPrefStageBytes;
    const auto kern = vec ? flp::k_pref<true> : flp::k_pref<false>;
    static std::atomic<int> fits[2][kMaxDevices];
    int fit = fits[vec][dev].load(std::memory_order_acquire);
    if (fit == 0) {
        int per_sm = 0;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, flp::kPrefThreads, kRing);
        if (e != cudaSuccess) return fail(FLP_ECUDA, "preference setup: %s", cudaGetErrorString(e));
        if (per_sm < 1) return fail(FLP_ECUDA, "preference setup: device %d cannot hold the kernel", dev);
        fit = per_sm * sms < flp::kPrefMaxCtas ? per_sm * sms : flp::kPrefMaxCtas;
        fits[vec][dev].store(fit, std::memory_order_release);
    }
    const int64_t by_tokens = ceil_div(a.nchunks, flp::kPrefThreads / 32);
    const int64_t by_pairs = ceil_div(num_seqs / 2, flp::kPrefThreads / (narrow ? 8 : 32));
    int64_t ctas = by_tokens > by_pairs ? by_tokens : by_pairs;
    ctas = ctas < 1 ? 1 : (ctas > fit ? fit : ctas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(flp::kPrefThreads);
    cfg.dynamicSmemBytes = kRing;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, narrow ? 1 : 0);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "preference launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
