// Host side of the Newton-Schulz orthogonalisation (flp_orthogonalize):
// argument checks, workspace layout, tensor maps and launches.
#include <math.h>

#include "host_common.h"
#include "ortho_cluster.cuh"
#include "ortho_kernels.cuh"

using namespace flp_host;

namespace {

struct OrthLayout {
    int64_t m, n, mp, np;              // of X: the matrix or its transpose, m <= n
    int64_t parts, d, e, f, hi0, hi1, lo, a0, b0, total;   // byte offsets
};

bool orth_layout(int64_t batch, int64_t rows, int64_t cols, OrthLayout* l) {
    l->m = rows < cols ? rows : cols;
    l->n = rows < cols ? cols : rows;
    l->mp = ceil_div(l->m, 64) * 64;
    l->np = ceil_div(l->n, 64) * 64;
    int64_t all_rows, x, a;
    if (__builtin_mul_overflow(batch, l->mp, &all_rows) || __builtin_mul_overflow(all_rows, l->np * 2, &x) ||
        __builtin_mul_overflow(all_rows, l->mp * 2, &a))
        return false;
    if (x > INT64_MAX / 16 || a > INT64_MAX / 16) return false;
    auto up = [](int64_t v) { return ceil_div(v, 1024) * 1024; };
    l->parts = 0;
    l->d = up(batch * flp::kOrthParts * (int64_t)sizeof(flp::OrthSum));
    l->e = l->d + up(all_rows * 4);
    l->f = l->e + up(all_rows * 4);
    l->hi0 = l->f + up(all_rows * 4);
    l->hi1 = l->hi0 + up(x);
    l->lo = l->hi1 + up(x);
    l->a0 = l->lo + up(x);
    l->b0 = l->a0 + up(a);
    l->total = l->b0 + up(a);
    return true;
}

flp_status check_orth_shape(int64_t batch, int64_t rows, int64_t cols) {
    if (batch < 0 || rows < 0 || cols < 0)
        return fail(FLP_EINVAL, "batch, rows and cols must be >= 0 (got %lld, %lld, %lld)", (long long)batch,
                    (long long)rows, (long long)cols);
    const int64_t lo = rows < cols ? rows : cols, hi = rows < cols ? cols : rows;
    const int64_t kMax = ((int64_t)1 << 31) - 1;
    // tensor-map coordinates and launch grids are 32-bit
    if (hi > kMax - 512 || lo > 65536 || (lo > 0 && batch > (kMax - 512) / (ceil_div(lo, 64) * 64)) ||
        batch > kMax / flp::kOrthParts)
        return fail(FLP_EUNSUPPORTED, "the smaller side must be <= 65536 and batch times it below 2^31");
    if (hi > 0 && batch > 0 &&
        (long double)batch * ceil_div(lo, 64) * 2.0L * ceil_div(hi, 64) * 2.0L > (long double)kMax)
        return fail(FLP_EUNSUPPORTED, "batch * rows * cols is too large");
    return FLP_OK;
}

// Tensor map of an FP16 row-major [rows, cols] matrix without padding between
// rows: boxes of box_cols (64: 128-byte swizzle, 32: 64-byte swizzle) x box_rows,
// zero fill.
flp_status orth_tmap(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, uint32_t box_rows,
                     uint32_t box_cols = 64) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(FLP_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FLP_EINVAL, "tensor map rejected by the driver (error %d)", (int)r);
    return FLP_OK;
}

// A launch of one product: its kernel for this shape, once per device allowed
// its shared memory.
struct OrthMaps {
    CUtensorMap a, b, in, lo, out;   // operands, what the epilogue reads and writes
};

template <int kMode, int kBN, bool kPair>
flp_status orth_launch(int dev, int fit, const OrthMaps& t, const flp::OrthArgs& p, cudaStream_t s) {
    static std::atomic<bool> ready[kMaxDevices];
    const auto kern = flp::k_orth_product<kMode, kBN, kPair>;
    constexpr size_t smem = flp::kOrthSmemBytes<kBN, kPair, kMode == flp::kOrthGram || kMode == flp::kOrthPoly>;
    static_assert(smem <= 232448, "shared memory per CTA");
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return fail(FLP_ECUDA, "orthogonalize setup: %s", cudaGetErrorString(e));
        ready[dev].store(true, std::memory_order_release);
    }
    const int64_t ctas = (p.units < fit ? p.units : fit) * (kPair ? 2 : 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(flp::kOrthProductThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kPair ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, t.a, t.b, t.in, t.lo, t.out, p);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "orthogonalize product launch: %s", cudaGetErrorString(e));
    return FLP_OK;
}

// Output tiles of one matrix.
int64_t orth_tiles(bool sym, int64_t rows, int64_t cols, int bm, int bn) {
    const int64_t tm = ceil_div(rows, bm), tn = ceil_div(cols, bn);
    if (!sym) return tm * tn;
    int64_t t = 0;
    for (int64_t mb = 0; mb < tm; ++mb) t += tn - mb * bm / bn;
    return t;
}

// A product whose 128 x 128 tiles leave SMs idle: a cluster of `split` CTAs a tile.
template <int kMode>
flp_status orth_split_launch(int dev, int split, const OrthMaps& t, const flp::OrthArgs& p, cudaStream_t s) {
    static std::atomic<bool> ready[kMaxDevices];
    const auto kern = flp::k_orth_split<kMode>;
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)flp::kOrthSplitSmem);
        if (e != cudaSuccess) return fail(FLP_ECUDA, "orthogonalize setup: %s", cudaGetErrorString(e));
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.units * split));
    cfg.blockDim = dim3(flp::kOrthThreads);
    cfg.dynamicSmemBytes = flp::kOrthSplitSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, t.a, t.b, p);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "orthogonalize product launch: %s", cudaGetErrorString(e));
    return FLP_OK;
}

// CTA pairs that can be resident at once on `dev` (cached; 0 if the query fails).
int orth_pairs(int dev) {
    static std::atomic<int> count[kMaxDevices];
    int c = count[dev].load(std::memory_order_acquire);
    if (c == 0) {
        const auto kern = flp::k_orth_product<flp::kOrthGram, 256, true>;
        constexpr size_t smem = flp::kOrthSmemBytes<256, true, true>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(flp::kOrthProductThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&c, (void*)kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            return 0;
        }
        count[dev].store(c, std::memory_order_release);
    }
    return c;
}

// The form of a product of matrices of mp x np (both padded) on `sms` SMs that hold
// `pairs` CTA pairs at once.
enum OrthFormKind { kOrthFormSplit = 0, kOrthFormCta = 1, kOrthFormPair = 2 };
OrthFormKind orth_form(bool sym, int64_t batch, int64_t mp, int64_t np, int sms, int pairs) {
    const int64_t cols = sym ? mp : np, units = batch * orth_tiles(sym, mp, cols, 128, 128);
    // Fewer 128 x 128 tiles than SMs: a tile a cluster, its K loop and its epilogue
    // split over up to 4 CTAs (a call on 1024 x 1024: 135 us with the tiles below, 152
    // unsplit, 117 split; 200 x 400: 90, 117, 89; 512 x 4096: 188, 193, 128).
    if (units <= sms) return kOrthFormSplit;
    // Else by the waves: 256 x 256 tiles a pair or 128 x 128 a CTA.  A wave of pairs weighs
    // 540 : 420 of one of CTAs: fitted to whole calls, with what a wave costs beside its K
    // blocks (which alone take 585 and 490 cycles).  Symmetric products by CTAs and by pairs:
    // 3008 x 3104 616 and 657 us in all, 8 x 1024 x 4096 687 and 745, 5 x 1000 x 1100 271 and
    // 250, 4096 x 4096 1312 and 1025; those with X: 20 x 300 x 310 134 and 164, 3008 x 3104
    // 648 and 616, 4096 x 4096 1218 and 1025.
    const int64_t small = ceil_div(units, sms) * 420;
    const int64_t wide = batch * orth_tiles(sym, mp, cols, 256, 256);
    return pairs <= 0 || small <= ceil_div(wide, pairs) * 540 ? kOrthFormCta : kOrthFormPair;
}

template <int kMode>
flp_status orth_product(int dev, int sms, int pairs, int64_t batch, const OrthMaps& t, flp::OrthArgs p, cudaStream_t s) {
    constexpr bool kSym = kMode == flp::kOrthGram || kMode == flp::kOrthPoly;
    const int64_t cols = kSym ? p.mp : p.np;
    p.nkb = (int)((kMode == flp::kOrthGram ? p.np : p.mp) / flp::kOrthBK);
    const OrthFormKind form = orth_form(kSym, batch, p.mp, p.np, sms, pairs);
    auto shape = [&](int bm, int bn) {
        p.tiles_m = (int)ceil_div(p.mp, bm);
        p.tiles_n = (int)ceil_div(cols, bn);
        p.per = orth_tiles(kSym, p.mp, cols, bm, bn);
        p.units = batch * p.per;
    };
    shape(128, 128);
    if (form == kOrthFormSplit) {
        int split = 1;
        while (split < 4 && p.units * split * 2 <= sms && p.nkb >= 4) split *= 2;
        return orth_split_launch<kMode>(dev, split, t, p, s);
    }
    if (form == kOrthFormCta) return orth_launch<kMode, 128, false>(dev, sms, t, p, s);
    shape(256, 256);
    return orth_launch<kMode, 256, true>(dev, pairs, t, p, s);
}

cudaLaunchConfig_t orth_cluster_config(int ctas, int64_t batch, cudaStream_t s, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * ctas));
    cfg.blockDim = dim3(flp::kOrthCluThreads);
    cfg.dynamicSmemBytes = flp::kOrthCluSmem;
    cfg.stream = s;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)ctas;
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of `ctas` CTAs (a power of two) that can be resident at once (0: none).
template <class T>
int orth_cluster_fit(int dev, int ctas) {
    static std::atomic<int> fits[kMaxDevices][5];   // by log2 of the CTAs; + 1
    const auto kern = flp::k_orth_cluster<T>;
    int log = 0;
    while ((1 << log) < ctas) ++log;
    int f = fits[dev][log].load(std::memory_order_acquire);
    if (f == 0) {
        cudaLaunchAttribute attr;
        const cudaLaunchConfig_t cfg = orth_cluster_config(ctas, 1, nullptr, &attr);
        int n = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)flp::kOrthCluSmem) !=
                cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, (void*)kern, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;
        }
        f = n + 1;
        fits[dev][log].store(f, std::memory_order_release);
    }
    return f - 1;
}

// CTAs of the cluster that holds a matrix with m <= 128 in one launch (0: the tiled
// kernels).
template <class T>
int orth_cluster_ctas(int dev, int64_t batch, int64_t m, int64_t blocks) {
    if (m > 128) return 0;
    auto fewest = [&](int per) {   // CTAs that hold `per` blocks of 64 columns each
        for (int c = 1; c <= flp::kOrthCluMaxCtas; c *= 2)
            if (ceil_div(blocks, c) <= per) return c;
        return 0;
    };
    // Few columns: one CTA, without exchanges (64 x 128: 19.6 us, in 2 CTAs 25.0; 128 x 256:
    // 37.6, in 4 41.6; 76 x 64 x 256: 26.9, in 4 70.0; a few of 64 x 256 alone the other
    // way round, 26.6 and 24.2).
    if (blocks <= 4) return orth_cluster_fit<T>(dev, 1) > 0 ? 1 : 0;
    // Two blocks a CTA while all clusters run at once (64 x 512: 27.3 us, four blocks
    // 35.1; 128 x 512: 45.8, 61.1; 64 x 1024: 29.0, 34.3), else four, or six with the most
    // CTAs (16 x 128 x 1024: two 93.7, four 56.0).
    int c = fewest(2);
    if (c == 0 || batch > orth_cluster_fit<T>(dev, c)) {
        c = fewest(4);
        if (c == 0) c = ceil_div(blocks, flp::kOrthCluMaxCtas) <= flp::kOrthCluMaxBlocks ? flp::kOrthCluMaxCtas : 0;
        if (c == 0) return 0;
    }
    const int fit = orth_cluster_fit<T>(dev, c);
    if (fit <= 0) return 0;
    // Large clusters leave SMs idle: over 64 rows the tiled kernels win from the third
    // wave on (128 x 4096, 16 CTAs: a batch of 12 128 against 139 us, of 16 190 against
    // 158; 128 x 2048, 8 CTAs: of 24 115 against 132, of 32 171 against 151); smaller
    // clusters and fewer rows stay ahead (200 x 64 x 1024: 206 against 279).
    if (m > 64 && c >= 8 && batch > 2 * (int64_t)fit) return 0;
    return c;
}

// The one-cluster form; *done = false where the tiled kernels have to serve.
template <class T>
flp_status orth_cluster_launch(int dev, int64_t batch, const flp::OrthCluArgs& p, cudaStream_t s, bool* done) {
    const int ctas = orth_cluster_ctas<T>(dev, batch, p.m, p.blocks);
    *done = ctas > 0 && batch * ctas < kMaxGrid;
    if (!*done) return FLP_OK;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = orth_cluster_config(ctas, batch, s, &attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, flp::k_orth_cluster<T>, p);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "orthogonalize cluster launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace

cudaError_t flp_take_orthogonalize_error(int* code) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, flp::g_orth_error, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(flp::g_orth_error, &zero, sizeof zero);
    *code = v;
    return e;
}

extern "C" {

flp_status flp_orthogonalize_workspace_size(int64_t batch, int64_t rows, int64_t cols, int64_t* bytes) {
    if (bytes == nullptr) return fail(FLP_EINVAL, "bytes is a null pointer");
    flp_status st;
    if ((st = check_orth_shape(batch, rows, cols)) != FLP_OK) return st;
    OrthLayout l;
    if (!orth_layout(batch, rows, cols, &l)) return fail(FLP_EINVAL, "workspace size overflows int64");
    *bytes = l.total;
    return ok();
}

flp_status flp_selftest_orthogonalize_form(int product, int64_t batch, int64_t rows, int64_t cols, int sms, int pairs,
                                           int* form) {
    if (form == nullptr) return fail(FLP_EINVAL, "form is a null pointer");
    if (product != 0 && product != 1) return fail(FLP_EINVAL, "product must be 0 or 1 (got %d)", product);
    if (sms < 1) return fail(FLP_EINVAL, "sms must be >= 1 (got %d)", sms);
    flp_status st;
    if ((st = check_orth_shape(batch, rows, cols)) != FLP_OK) return st;
    OrthLayout l;
    if (!orth_layout(batch, rows, cols, &l)) return fail(FLP_EINVAL, "workspace size overflows int64");
    *form = (int)orth_form(product == 0, batch, l.mp, l.np, sms, pairs);
    return ok();
}

flp_status flp_orthogonalize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ld_x,
                             int64_t stride_x, int steps, const float* coefficients, float eps, float scale,
                             void* workspace, int64_t workspace_bytes, void* out, int out_dtype, int64_t ld_out,
                             int64_t stride_out, flp_stream_t stream) {
    flp_status st;
    if ((st = check_dtype(dtype)) != FLP_OK) return st;
    if (out_dtype != FLP_DTYPE_BF16 && out_dtype != FLP_DTYPE_F32)
        return fail(FLP_EINVAL, "out_dtype must be FLP_DTYPE_BF16 or FLP_DTYPE_F32 (got %d)", out_dtype);
    if ((st = check_orth_shape(batch, rows, cols)) != FLP_OK) return st;
    if (steps < 1 || steps > flp::kOrthMaxSteps)
        return fail(FLP_EINVAL, "steps must be in [1, %d] (got %d)", flp::kOrthMaxSteps, steps);
    if (coefficients == nullptr) return fail(FLP_EINVAL, "coefficients is a null pointer");
    for (int k = 0; k < 3 * steps; ++k)
        if (!isfinite(coefficients[k])) return fail(FLP_EINVAL, "coefficients must be finite");
    if (!(eps >= 0.f) || !isfinite(eps) || !isfinite(scale))
        return fail(FLP_EINVAL, "eps must be finite and >= 0 and scale finite");
    if (ld_x < cols || ld_out < cols)
        return fail(FLP_EINVAL, "ld_x (%lld) and ld_out (%lld) must be >= cols (%lld)", (long long)ld_x,
                    (long long)ld_out, (long long)cols);
    if (batch == 0 || rows == 0 || cols == 0) return ok();
    int64_t bx, bo, span_x, span_o;
    if (!span_bytes(rows, cols, ld_x, 1, &bx) || !span_bytes(rows, cols, ld_out, 1, &bo) ||
        !span_bytes(batch, bx, stride_x, elem_bytes(dtype), &span_x) ||
        !span_bytes(batch, bo, stride_out, elem_bytes(out_dtype), &span_o))
        return fail(FLP_EINVAL, "x or out extent overflows int64");
    if (batch > 1 && (stride_x < 0 || stride_out < bo))
        return fail(FLP_EINVAL, "stride_x must be >= 0 and stride_out cover a matrix");
    // a matrix's x is read before its out is written, but matrices do not wait for
    // one another: out is x in place, or apart from it
    const uintptr_t xa = reinterpret_cast<uintptr_t>(x), oa = reinterpret_cast<uintptr_t>(out);
    const bool in_place = x == out && ld_x == ld_out && (batch == 1 || stride_x == stride_out) &&
                          elem_bytes(dtype) == elem_bytes(out_dtype);
    if (!in_place && x != nullptr && out != nullptr && xa < oa + (uintptr_t)span_o && oa < xa + (uintptr_t)span_x)
        return fail(FLP_EINVAL, "out overlaps x");
    OrthLayout l;
    if (!orth_layout(batch, rows, cols, &l)) return fail(FLP_EINVAL, "workspace size overflows int64");
    if (workspace_bytes < l.total)
        return fail(FLP_EINVAL, "workspace_bytes (%lld) is below the %lld bytes needed", (long long)workspace_bytes,
                    (long long)l.total);
    if ((reinterpret_cast<uintptr_t>(workspace) & 127u) != 0)
        return fail(FLP_EINVAL, "workspace must start on a 128-byte boundary");
    const void* ptrs[] = {x, workspace, out};
    const char* names[] = {"x", "workspace", "out"};
    int dev;
    if ((st = common_device(3, ptrs, names, nullptr, &dev)) != FLP_OK) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(FLP_ECUDA, "device index %d out of range", dev);
    DeviceGuard guard;
    if ((st = guard.enter(dev)) != FLP_OK) return st;
    const int sms = sm_count(dev);
    if (sms <= 0) return fail(FLP_ECUDA, "could not read the SM count of device %d", dev);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int eb = elem_bytes(dtype), ob = elem_bytes(out_dtype);
    const bool vec_in = (cols * eb) % 16 == 0 && rows_aligned16(x, ld_x, dtype) &&
                        (batch == 1 || (stride_x * eb) % 16 == 0);
    const bool vec_out = aligned16(out) && (ld_out * ob) % 16 == 0 && (batch == 1 || (stride_out * ob) % 16 == 0);
    // by what the steps after it multiply a step's noise
    float stray[flp::kOrthMaxSteps];
    double grow = 1.0;
    for (int k = steps - 1; k >= 0; --k) {
        stray[k] = (float)(flp::kOrthStray / grow);
        grow *= (double)coefficients[3 * k] * (double)coefficients[3 * k];
    }
    if (l.m <= 128) {
        flp::OrthCluArgs c{};
        c.x = x;
        c.ld = ld_x;
        c.stride = stride_x;
        c.m = l.m;
        c.n = l.n;
        c.mp = (int)l.mp;
        c.blocks = (int)(l.np / 64);
        c.transposed = rows > cols ? 1 : 0;
        c.vec = vec_in;
        c.steps = steps;
        c.eps = eps;
        c.scale = scale;
        c.out = out;
        c.out_dtype = out_dtype;
        c.vec_out = vec_out;
        c.ld_out = ld_out;
        c.stride_out = stride_out;
        for (int k = 0; k < 3 * steps; ++k) c.coef[k] = coefficients[k];
        for (int k = 0; k < steps; ++k) c.stray[k] = stray[k];
        bool done = false;
        st = dtype == FLP_DTYPE_BF16 ? orth_cluster_launch<__nv_bfloat16>(dev, batch, c, s, &done)
             : dtype == FLP_DTYPE_F16 ? orth_cluster_launch<__half>(dev, batch, c, s, &done)
                                      : orth_cluster_launch<float>(dev, batch, c, s, &done);
        if (st != FLP_OK || done) return st;
    }
    const int pairs = orth_pairs(dev);
    char* ws = static_cast<char*>(workspace);
    __half* hi[2] = {reinterpret_cast<__half*>(ws + l.hi0), reinterpret_cast<__half*>(ws + l.hi1)};
    __half* lo = reinterpret_cast<__half*>(ws + l.lo);

    // operands in boxes of 128 rows (MN-major: 64), the epilogues' reads and writes of 32
    CUtensorMap op_x[2], op_x64[2], op_a0, op_b0, ep_x[2], ep_lo, ep_a0, ep_b0;
    const int64_t all_rows = batch * l.mp;
    for (int k = 0; k < 2; ++k) {
        if ((st = orth_tmap(&op_x[k], hi[k], all_rows, l.np, 128)) != FLP_OK) return st;
        if ((st = orth_tmap(&op_x64[k], hi[k], all_rows, l.np, 64)) != FLP_OK) return st;
        if ((st = orth_tmap(&ep_x[k], hi[k], all_rows, l.np, 32, 32)) != FLP_OK) return st;
    }
    if ((st = orth_tmap(&ep_lo, lo, all_rows, l.np, 32, 32)) != FLP_OK) return st;
    if ((st = orth_tmap(&op_a0, ws + l.a0, all_rows, l.mp, 128)) != FLP_OK) return st;
    if ((st = orth_tmap(&ep_a0, ws + l.a0, all_rows, l.mp, 32, 32)) != FLP_OK) return st;
    if ((st = orth_tmap(&op_b0, ws + l.b0, all_rows, l.mp, 128)) != FLP_OK) return st;
    if ((st = orth_tmap(&ep_b0, ws + l.b0, all_rows, l.mp, 32, 32)) != FLP_OK) return st;

    flp::OrthInput in{};
    in.x = x;
    in.rows = rows;
    in.cols = cols;
    in.ld = ld_x;
    in.stride = stride_x;
    in.tiles_m = l.mp / 64;
    in.tiles = in.tiles_m * (l.np / 64);
    in.all_tiles = batch * in.tiles;
    in.transposed = rows > cols ? 1 : 0;
    in.vec = vec_in;
    // parts of at least 16 K elements; their number must not depend on the batch
    int64_t parts = ceil_div(rows * cols, 16384);
    parts = parts < rows ? parts : rows;
    in.parts = (int)(parts < flp::kOrthParts ? parts : flp::kOrthParts);
    in.eps = eps;
    in.sums = reinterpret_cast<flp::OrthSum*>(ws + l.parts);
    in.hi = hi[0];
    in.lo = lo;
    in.mp = l.mp;
    in.np = l.np;
    const int64_t gs = batch * in.parts;
    const int64_t gl = in.all_tiles < 8 * (int64_t)sms ? in.all_tiles : 8 * (int64_t)sms;
    auto input = [&](auto sum, auto load) {
        sum<<<(unsigned)gs, flp::kOrthSumThreads, 0, s>>>(in);
        const flp_status e = check_launch("orthogonalize norm");
        return e != FLP_OK ? e
                           : launch_dependent("orthogonalize input", load, dim3((unsigned)gl), flp::kOrthLoadThreads,
                                              (size_t)0, s, in);
    };
    st = dtype == FLP_DTYPE_BF16 ? input(flp::k_orth_sumsq<__nv_bfloat16>, flp::k_orth_load<__nv_bfloat16>)
         : dtype == FLP_DTYPE_F16 ? input(flp::k_orth_sumsq<__half>, flp::k_orth_load<__half>)
                                  : input(flp::k_orth_sumsq<float>, flp::k_orth_load<float>);
    if (st != FLP_OK) return st;

    flp::OrthArgs p{};
    p.m = l.m;
    p.n = l.n;
    p.mp = l.mp;
    p.np = l.np;
    p.d = reinterpret_cast<float*>(ws + l.d);
    p.e = reinterpret_cast<float*>(ws + l.e);
    p.f = reinterpret_cast<float*>(ws + l.f);
    p.mat_in = reinterpret_cast<const __half*>(ws + l.a0);
    p.x_lo = lo;
    p.out = out;
    p.out_dtype = out_dtype;
    p.transposed = rows > cols ? 1 : 0;
    p.vec_out = vec_out;
    p.ld_out = ld_out;
    p.stride_out = stride_out;
    p.scale = scale;
    for (int k = 0; k < steps; ++k) {
        const int cur = k & 1;
        p.a = coefficients[3 * k];
        p.b = coefficients[3 * k + 1];
        p.c = coefficients[3 * k + 2];
        p.stray = stray[k];
        p.x_hi = hi[cur];
        p.x_out = hi[cur ^ 1];
        p.mat_out = reinterpret_cast<__half*>(ws + l.a0);
        OrthMaps t{op_x[cur], op_x[cur], ep_a0, ep_a0, ep_a0};   // Gram reads nothing beside its operands
        if ((st = orth_product<flp::kOrthGram>(dev, sms, pairs, batch, t, p, s)) != FLP_OK) return st;
        p.mat_out = reinterpret_cast<__half*>(ws + l.b0);
        t = OrthMaps{op_a0, op_a0, ep_a0, ep_a0, ep_b0};
        if ((st = orth_product<flp::kOrthPoly>(dev, sms, pairs, batch, t, p, s)) != FLP_OK) return st;
        t = OrthMaps{op_b0, op_x64[cur], ep_x[cur], ep_lo, ep_x[cur ^ 1]};
        if (k + 1 < steps) st = orth_product<flp::kOrthApply>(dev, sms, pairs, batch, t, p, s);
        else st = orth_product<flp::kOrthFinal>(dev, sms, pairs, batch, t, p, s);
        if (st != FLP_OK) return st;
    }
    return ok();
}

}  // extern "C"
