// Host side of the norm's backward (fused_layer_norm_backward): argument checks and
// launches.
#include <math.h>

#include "norm_host.h"

using namespace flp_host;

namespace {

// Where a call's launches go: `sms` sizes the grid of the rows (kNormSms but in the
// self-test).
struct NormTo {
    int dev, sms;
    cudaStream_t s;
};

template <class T, class G, bool kCenter>
flp_status launch_bwd_any(const flp::NormBwdArgs& a, const NormTo& to, int* parts) {
    const cudaStream_t s = to.s;
    flp::k_norm_dx_any<T, G, kCenter><<<row_ctas(a.n, 1, to.sms * 8), flp::kNormAnyThreads, 0, s>>>(a);
    if (a.part_w || a.part_b) {
        *parts = row_ctas(a.n, 1, flp::kNormAnyParts);
        const dim3 grid((unsigned)ceil_div(a.d, flp::kNormAnyThreads), (unsigned)*parts);
        flp::k_norm_dw_any<T, G, kCenter><<<grid, flp::kNormAnyThreads, 0, s>>>(a);
    }
    return check_launch("norm backward");
}

// Launches the row kernel.  *parts = its CTAs, one partial row each, that are left
// to fold; 0 where the kernel folds them itself.
template <class T, class G, int kTpr, bool kFull, bool kAligned>
flp_status launch_bwd_rows(const flp::NormBwdArgs& a, const NormTo& to, int* parts) {
    const int dev = to.dev;
    static std::atomic<bool> ready[kMaxDevices];
    static std::atomic<int> fits[kMaxDevices];   // CTAs that can be resident at once + 1, with the most shared memory
    constexpr int kThreads = flp::kNormThreads<kTpr>, kRows = kThreads / kTpr;
    static_assert(kNormSms * flp::kNormBwdCtas<kTpr> <= flp::kNormParts, "a partial row per CTA");
    const auto kern = flp::k_norm_bwd<T, G, kTpr, kFull, kAligned>;
    constexpr int kStages = flp::kNormBwdStages<T, G>;
    constexpr auto bytes = [](int64_t d) {
        return kAligned ? (size_t)kThreads * flp::kNormElems * (sizeof(T) + sizeof(G)) * kStages
                        : ((size_t)(flp::norm_pitch<T>(d) + flp::norm_pitch<G>(d)) * kStages + flp::norm_pitch<T>(d)) *
                              kRows;
    };
    // for the widest row of this kernel, so that one number serves all its calls
    constexpr size_t top = bytes((int64_t)kTpr * flp::kNormElems);
    static_assert(top <= kNormMaxSmem, "the widest row of this kernel fits");
    const size_t smem = bytes(a.d);
    flp_status st;
    if ((st = norm_setup(kern, dev, ready)) != FLP_OK) return st;
    const int rows = row_ctas(a.n, kRows, to.sms * flp::kNormBwdCtas<kTpr>);
    int fit = fits[dev].load(std::memory_order_acquire);
    if (fit == 0) {
        int per_sm = 0;
        const int sms = sm_count(dev);
        if (sms <= 0 ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, top) != cudaSuccess) {
            (void)cudaGetLastError();
            per_sm = 0;
        }
        fit = per_sm * sms + 1;
        fits[dev].store(fit, std::memory_order_release);
    }
    const bool sums = a.part_w != nullptr || a.part_b != nullptr, grid_fold = sums && rows < fit;
    // with a few rows more CTAs than take any, so that the fold takes one turn
    int grid = rows;
    if (grid_fold) {
        const int teams = kThreads / 32 / flp::norm_fold_team(rows, kThreads / 32);
        const int64_t want = ceil_div(ceil_div(a.d, 8) * ((a.part_w != nullptr) + (a.part_b != nullptr)), teams);
        if (grid < want) grid = (int)(want < fit - 1 ? want : fit - 1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = to.s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = grid_fold ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, rows, grid_fold ? 1 : 0);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "norm backward launch: %s", cudaGetErrorString(e));
    *parts = grid_fold || !sums ? 0 : rows;
    return ok();
}

template <class T, class G, bool kFull, bool kAligned>
flp_status launch_bwd_v(const flp::NormBwdArgs& a, const NormTo& to, int* parts) {
    // As in the forward, the fewest threads that hold a row (2 M rows of 64 BF16: by a warp
    // each 515 us, 160 here; 65536 x 512 with 128 threads 69, 42 here; 32768 x 2048 with 256
    // 83, 69 here), but for two warps a row (131072 x 1024: 168 us, with four 153).
    constexpr int E = flp::kNormElems;
    if (a.d <= 8 * E) return launch_bwd_rows<T, G, 8, kFull, kAligned>(a, to, parts);
    if (a.d <= 16 * E) return launch_bwd_rows<T, G, 16, kFull, kAligned>(a, to, parts);
    if (a.d <= 32 * E) return launch_bwd_rows<T, G, 32, kFull, kAligned>(a, to, parts);
    if (a.d <= 128 * E) return launch_bwd_rows<T, G, 128, kFull, kAligned>(a, to, parts);
    if (a.d <= 256 * E) return launch_bwd_rows<T, G, 256, kFull, kAligned>(a, to, parts);
    return launch_bwd_rows<T, G, 512, kFull, kAligned>(a, to, parts);
}

template <class T, class G>
flp_status launch_norm_bwd(const flp::NormBwdArgs& a, bool vec, const NormTo& to, int* parts) {
    const bool center = a.mean != nullptr, full = center || a.part_b != nullptr;
    if (a.d > 512 * flp::kNormElems)
        return center ? launch_bwd_any<T, G, true>(a, to, parts) : launch_bwd_any<T, G, false>(a, to, parts);
    if (vec)
        return full ? launch_bwd_v<T, G, true, true>(a, to, parts) : launch_bwd_v<T, G, false, true>(a, to, parts);
    return full ? launch_bwd_v<T, G, true, false>(a, to, parts) : launch_bwd_v<T, G, false, false>(a, to, parts);
}

// Most partial rows of n rows: a CTA that has one has a row.
int64_t norm_parts(int64_t n) { return n < flp::kNormParts ? n : flp::kNormParts; }

bool norm_workspace_bytes(int64_t n, int64_t d, int64_t* out) {
    int64_t b;
    if (d > INT64_MAX - 4 || __builtin_mul_overflow((d + 3) / 4 * 4, 8 * norm_parts(n), &b) || b > INT64_MAX - 256)
        return false;
    *out = ceil_div(b, 256) * 256;
    return true;
}

flp_status norm_backward(int sms, const void* dy, int dy_dtype, int64_t ld_dy, const void* x, int dtype, int64_t n,
                         int64_t d, int64_t ld_x, const void* weight, int weight_dtype, const float* mean,
                         const float* rstd, int center, void* workspace, int64_t workspace_bytes, void* dx,
                         int64_t ld_dx, float* dweight, float* dbias, int accumulate, flp_stream_t stream) {
    flp_status st;
    if ((st = check_norm_shape(n, d, dtype)) != FLP_OK) return st;
    if ((st = check_side_dtype("weight", weight_dtype, dtype)) != FLP_OK) return st;
    if ((st = check_side_dtype("dy", dy_dtype, dtype)) != FLP_OK) return st;
    if (ld_x < d || ld_dy < d || ld_dx < d)
        return fail(FLP_EINVAL, "ld_x (%lld), ld_dy (%lld) and ld_dx (%lld) must be >= d (%lld)", (long long)ld_x,
                    (long long)ld_dy, (long long)ld_dx, (long long)d);
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (n == 0 && !sums) return ok();
    int64_t need = 0;
    if (!norm_workspace_bytes(n, d, &need)) return fail(FLP_EINVAL, "workspace size overflows int64");
    if (sums && n > 0) {
        if (workspace_bytes < need)
            return fail(FLP_EINVAL, "workspace_bytes (%lld) is below the %lld bytes needed",
                        (long long)workspace_bytes, (long long)need);
        if (!aligned16(workspace)) return fail(FLP_EINVAL, "workspace must start on a 16-byte boundary");
    }
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int dev;
    if (n == 0) {
        // no rows: the sums are empty
        const void* ptrs[] = {dweight, dbias};
        const char* names[] = {"dweight", "dbias"};
        const bool optional[] = {true, true};
        if ((st = common_device(2, ptrs, names, optional, &dev)) != FLP_OK) return st;
        DeviceGuard guard;
        if ((st = guard.enter(dev)) != FLP_OK) return st;
        cudaError_t e = cudaSuccess;
        if (!accumulate && dweight) e = cudaMemsetAsync(dweight, 0, (size_t)d * 4, s);
        if (e == cudaSuccess && !accumulate && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)d * 4, s);
        if (e != cudaSuccess) return fail(FLP_ECUDA, "norm backward: %s", cudaGetErrorString(e));
        return ok();
    }
    const int eb = elem_bytes(dtype), gb = elem_bytes(dy_dtype);
    int64_t bx, bg, bd;
    if (!span_bytes(n, d, ld_x, eb, &bx) || !span_bytes(n, d, ld_dy, gb, &bg) || !span_bytes(n, d, ld_dx, eb, &bd))
        return fail(FLP_EINVAL, "x, dy or dx extent overflows int64");
    const Extent ed{"dx", dx, bd};
    if ((st = check_apart(ed, {"x", x, bx}, false)) != FLP_OK) return st;
    if ((st = check_apart(ed, {"dy", dy, bg}, false)) != FLP_OK) return st;
    const void* ptrs[] = {dy, x, rstd, dx, mean, weight, dweight, dbias, workspace};
    const char* names[] = {"dy", "x", "rstd", "dx", "mean", "weight", "dweight", "dbias", "workspace"};
    const bool optional[] = {false, false, false, false, center == 0, true, true, true, !sums};
    if ((st = common_device(9, ptrs, names, optional, &dev)) != FLP_OK) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(FLP_ECUDA, "device index %d out of range", dev);
    DeviceGuard guard;
    if ((st = guard.enter(dev)) != FLP_OK) return st;
    float* ws = static_cast<float*>(workspace);
    const int64_t dp = ceil_div(d, 4) * 4;
    const flp::NormBwdArgs a{dy, ld_dy, x, n, d, ld_x, {weight, weight_dtype}, center ? mean : nullptr, rstd,
                             1.f / (float)d, dx, ld_dx, dp, dweight ? ws : nullptr,
                             dbias ? ws + norm_parts(n) * dp : nullptr, dweight, dbias, accumulate != 0};
    const bool wide = dy_dtype == FLP_DTYPE_F32;
    const bool vec = (d * eb) % 16 == 0 && rows_aligned16(x, ld_x, dtype) && rows_aligned16(dx, ld_dx, dtype) &&
                     rows_aligned16(dy, ld_dy, dy_dtype) && aligned16(weight);
    const NormTo to{dev, sms, s};
    int parts = 0;
    if (dtype == FLP_DTYPE_BF16)
        st = wide ? launch_norm_bwd<__nv_bfloat16, float>(a, vec, to, &parts)
                  : launch_norm_bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, to, &parts);
    else if (dtype == FLP_DTYPE_F16)
        st = wide ? launch_norm_bwd<__half, float>(a, vec, to, &parts)
                  : launch_norm_bwd<__half, __half>(a, vec, to, &parts);
    else
        st = launch_norm_bwd<float, float>(a, vec, to, &parts);
    if (st != FLP_OK || parts == 0) return st;
    return launch_dependent("norm fold", flp::k_norm_fold<flp::kNormFoldThreads>, dim3((unsigned)(2 * ceil_div(d, 8))), flp::kNormFoldThreads,
                            (size_t)0, s, a, parts);
}

}  // namespace

extern "C" {

flp_status fused_layer_norm_backward_workspace_size(int64_t d, int64_t* bytes) {
    if (bytes == nullptr) return fail(FLP_EINVAL, "bytes is a null pointer");
    if (d < 1) return fail(FLP_EINVAL, "d must be >= 1 (got %lld)", (long long)d);
    if (!norm_workspace_bytes(flp::kNormParts, d, bytes)) return fail(FLP_EINVAL, "workspace size overflows int64");
    return ok();
}

flp_status fused_layer_norm_backward_rows_workspace_size(int64_t n, int64_t d, int64_t* bytes) {
    if (bytes == nullptr) return fail(FLP_EINVAL, "bytes is a null pointer");
    if (n < 0) return fail(FLP_EINVAL, "n must be >= 0 (got %lld)", (long long)n);
    if (d < 1) return fail(FLP_EINVAL, "d must be >= 1 (got %lld)", (long long)d);
    if (!norm_workspace_bytes(n, d, bytes)) return fail(FLP_EINVAL, "workspace size overflows int64");
    return ok();
}

flp_status fused_layer_norm_backward(const void* dy, int dy_dtype, int64_t ld_dy, const void* x, int dtype, int64_t n,
                                     int64_t d, int64_t ld_x, const void* weight, int weight_dtype, const float* mean,
                                     const float* rstd, int center, void* workspace, int64_t workspace_bytes, void* dx,
                                     int64_t ld_dx, float* dweight, float* dbias, int accumulate,
                                     flp_stream_t stream) {
    return norm_backward(kNormSms, dy, dy_dtype, ld_dy, x, dtype, n, d, ld_x, weight, weight_dtype, mean, rstd, center,
                         workspace, workspace_bytes, dx, ld_dx, dweight, dbias, accumulate, stream);
}

flp_status flp_selftest_norm_backward(int sms, const void* dy, int dy_dtype, int64_t ld_dy, const void* x, int dtype,
                                      int64_t n, int64_t d, int64_t ld_x, const void* weight, int weight_dtype,
                                      const float* mean, const float* rstd, int center, void* workspace,
                                      int64_t workspace_bytes, void* dx, int64_t ld_dx, float* dweight, float* dbias,
                                      int accumulate, flp_stream_t stream) {
    if (sms < 1 || sms > kNormSms) return fail(FLP_EINVAL, "sms must be in [1, %d] (got %d)", kNormSms, sms);
    return norm_backward(sms, dy, dy_dtype, ld_dy, x, dtype, n, d, ld_x, weight, weight_dtype, mean, rstd, center,
                         workspace, workspace_bytes, dx, ld_dx, dweight, dbias, accumulate, stream);
}

}  // extern "C"
