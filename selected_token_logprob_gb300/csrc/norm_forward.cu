// Host side of the norm's forward (fused_layer_norm_forward): argument checks and
// launches.
#include <math.h>

#include "norm_host.h"

using namespace flp_host;

namespace {

template <class T, bool kCenter>
flp_status launch_fwd_any(const flp::NormFwdArgs& a, cudaStream_t s) {
    flp::k_norm_fwd_any<T, kCenter><<<row_ctas(a.n, 1, kNormSms * 8), flp::kNormAnyThreads, 0, s>>>(a);
    return check_launch("norm forward");
}

template <class T, class W, int kTpr, bool kCenter, bool kAligned>
flp_status launch_fwd_rows(const flp::NormFwdArgs& a, int dev, cudaStream_t s) {
    static std::atomic<bool> ready[kMaxDevices];
    constexpr int kThreads = flp::kNormThreads<kTpr>, kRows = kThreads / kTpr;
    constexpr int kStages = flp::kNormFwdStages<T, kTpr, kAligned>;
    static_assert((size_t)flp::norm_pitch<T>(kTpr * flp::kNormElems) * kRows * (kStages + 1) <= kNormMaxSmem || kAligned,
                  "the widest row of this kernel fits");
    const auto kern = flp::k_norm_fwd<T, W, kTpr, kCenter, kAligned>;
    const size_t smem = kAligned ? (size_t)kThreads * flp::kNormElems * sizeof(T) * kStages
                                 : (size_t)flp::norm_pitch<T>(a.d) * kRows * (kStages + 1);
    flp_status st;
    if ((st = norm_setup(kern, dev, ready)) != FLP_OK) return st;
    kern<<<row_ctas(a.n, kRows, kNormSms * flp::kNormFwdCtas<kTpr>), kThreads, smem, s>>>(a);
    return check_launch("norm forward");
}

template <class T, class W, bool kCenter, bool kAligned>
flp_status launch_fwd_v(const flp::NormFwdArgs& a, int dev, cudaStream_t s) {
    // The fewest threads that hold a row: with the next form up, 2 M rows of 64 BF16 take
    // 393 us by a warp each (103 here), 65536 x 512 49 (26), 131072 x 1024 112 (101),
    // 32768 x 2048 60 (47), 16384 x 4096 64 (48).  Wider rows than these are read once per
    // sum (8192 x 8192 that way: 82 us, 50 here).
    constexpr int E = flp::kNormElems;
    if (a.d <= 8 * E) return launch_fwd_rows<T, W, 8, kCenter, kAligned>(a, dev, s);
    if (a.d <= 16 * E) return launch_fwd_rows<T, W, 16, kCenter, kAligned>(a, dev, s);
    if (a.d <= 32 * E) return launch_fwd_rows<T, W, 32, kCenter, kAligned>(a, dev, s);
    if (a.d <= 64 * E) return launch_fwd_rows<T, W, 64, kCenter, kAligned>(a, dev, s);
    if (a.d <= 128 * E) return launch_fwd_rows<T, W, 128, kCenter, kAligned>(a, dev, s);
    if (a.d <= 256 * E) return launch_fwd_rows<T, W, 256, kCenter, kAligned>(a, dev, s);
    if (a.d <= 512 * E) return launch_fwd_rows<T, W, 512, kCenter, kAligned>(a, dev, s);
    if (a.d <= 1024 * E) return launch_fwd_rows<T, W, 1024, kCenter, kAligned>(a, dev, s);
    return launch_fwd_any<T, kCenter>(a, s);
}

template <class T, class W>
flp_status launch_fwd_w(const flp::NormFwdArgs& a, bool center, bool vec, int dev, cudaStream_t s) {
    if (vec) return center ? launch_fwd_v<T, W, true, true>(a, dev, s) : launch_fwd_v<T, W, false, true>(a, dev, s);
    return center ? launch_fwd_v<T, W, true, false>(a, dev, s) : launch_fwd_v<T, W, false, false>(a, dev, s);
}

template <class T>
flp_status launch_norm_fwd(const flp::NormFwdArgs& a, bool center, bool vec, int dev, cudaStream_t s) {
    return a.w.dtype == FLP_DTYPE_F32 ? launch_fwd_w<T, float>(a, center, vec, dev, s)
                                      : launch_fwd_w<T, T>(a, center, vec, dev, s);
}

}  // namespace

extern "C" {

flp_status fused_layer_norm_forward(const void* x, int dtype, int64_t n, int64_t d, int64_t ld_x,
                                    const void* weight, const void* bias, int weight_dtype, float eps, int center,
                                    void* y, int64_t ld_y, float* mean, float* rstd, flp_stream_t stream) {
    flp_status st;
    if ((st = check_norm_shape(n, d, dtype)) != FLP_OK) return st;
    if ((st = check_side_dtype("weight", weight_dtype, dtype)) != FLP_OK) return st;
    if (ld_x < d || ld_y < d)
        return fail(FLP_EINVAL, "ld_x (%lld) and ld_y (%lld) must be >= d (%lld)", (long long)ld_x, (long long)ld_y,
                    (long long)d);
    if (!(eps >= 0.f) || !isfinite(eps)) return fail(FLP_EINVAL, "eps must be finite and >= 0 (got %g)", (double)eps);
    if (n == 0) return ok();
    const int eb = elem_bytes(dtype);
    int64_t bx, by;
    if (!span_bytes(n, d, ld_x, eb, &bx) || !span_bytes(n, d, ld_y, eb, &by))
        return fail(FLP_EINVAL, "x or y extent overflows int64");
    const Extent ey{"y", y, by};
    if ((st = check_apart(ey, {"x", x, bx}, ld_x == ld_y)) != FLP_OK) return st;
    const void* ptrs[] = {x, y, weight, bias, mean, rstd};
    const char* names[] = {"x", "y", "weight", "bias", "mean", "rstd"};
    const bool optional[] = {false, false, true, true, true, true};
    int dev;
    if ((st = common_device(6, ptrs, names, optional, &dev)) != FLP_OK) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(FLP_ECUDA, "device index %d out of range", dev);
    DeviceGuard guard;
    if ((st = guard.enter(dev)) != FLP_OK) return st;
    const flp::NormFwdArgs a{x, n, d, ld_x, {weight, weight_dtype}, {bias, weight_dtype}, eps, 1.f / (float)d,
                             y, ld_y, mean, rstd};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // 16-byte vectors need whole, aligned ones in every row and vector
    const bool vec = (d * eb) % 16 == 0 && rows_aligned16(x, ld_x, dtype) && rows_aligned16(y, ld_y, dtype) &&
                     aligned16(weight) && aligned16(bias);
    if (dtype == FLP_DTYPE_BF16) return launch_norm_fwd<__nv_bfloat16>(a, center != 0, vec, dev, s);
    if (dtype == FLP_DTYPE_F16) return launch_norm_fwd<__half>(a, center != 0, vec, dev, s);
    return launch_norm_fwd<float>(a, center != 0, vec, dev, s);
}

}  // extern "C"
