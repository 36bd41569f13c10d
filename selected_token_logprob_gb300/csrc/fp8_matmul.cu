// Host side of the 8-bit products and their quantiser (flp_quantize_fp8, flp_fp8_matmul):
// argument checks and launches.
#include "fp8_matmul.cuh"
#include "fp8_quantize.cuh"
#include "norm_host.h"

using namespace flp_host;

namespace {

constexpr int64_t kMaxSide = ((int64_t)1 << 31) - 1024;   // tensor-map coordinates are 32-bit

template <class T>
flp_status launch_quantize(const flp::QuantArgs& a, bool vec, cudaStream_t s) {
    const int64_t tiles = ceil_div(a.rows, 128) * a.tiles_c;
    if (tiles > kMaxGrid) return fail(FLP_EUNSUPPORTED, "rows * cols is too large");
    const int grid = (int)tiles;
    if (vec) flp::k_quantize_fp8<T, true><<<grid, flp::kQuantThreads, 0, s>>>(a);
    else flp::k_quantize_fp8<T, false><<<grid, flp::kQuantThreads, 0, s>>>(a);
    return check_launch("quantize");
}

// Rows of `cols` elements of eb bytes, boxes of 128 bytes (one swizzle row) x box_rows, zeros outside.
flp_status fp8_tmap(CUtensorMap* map, const char* name, CUtensorMapDataType type, int eb, const void* ptr,
                    int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(FLP_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * eb)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / eb), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(map, type, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FLP_EINVAL, "%s: tensor map rejected by the driver (error %d)", name, (int)r);
    return FLP_OK;
}

template <class K>
flp_status fp8_setup(K kern, int dev, size_t smem, std::atomic<bool>* ready) {
    if (ready[dev].load(std::memory_order_acquire)) return FLP_OK;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "fp8 product setup: %s", cudaGetErrorString(e));
    ready[dev].store(true, std::memory_order_release);
    return FLP_OK;
}

template <class... Args>
flp_status fp8_launch(void (*kern)(Args...), int64_t grid, int threads, size_t smem, int cluster, cudaStream_t s,
                      Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "fp8 product launch: %s", cudaGetErrorString(e));
    return ok();
}

template <int kB>
flp_status launch_pair(const flp::Fp8Args& p, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                       int dev, int sms, cudaStream_t s) {
    static std::atomic<bool> ready[kMaxDevices];
    const auto kern = flp::k_fp8_pair<kB>;
    flp_status st;
    if ((st = fp8_setup(kern, dev, flp::kFp8PairSmem<kB != 0>, ready)) != FLP_OK) return st;
    const int64_t tiles = p.tiles_m * p.tiles_n, pairs = tiles < sms / 2 ? tiles : sms / 2;
    return fp8_launch(kern, 2 * pairs, flp::kFp8PairThreads, flp::kFp8PairSmem<kB != 0>, 1, s, ta, tb, tc, p);
}

template <int kBN>
flp_status launch_tokens(flp::Fp8Args p, const CUtensorMap& ta, const CUtensorMap& tb, int dev, int sms, int split,
                         cudaStream_t s) {
    static std::atomic<bool> ready[kMaxDevices];
    const auto kern = flp::k_fp8_tokens<kBN>;
    flp_status st;
    if ((st = fp8_setup(kern, dev, flp::kFp8TokSmem<kBN>, ready)) != FLP_OK) return st;
    const int64_t tiles = p.tiles_m * p.tiles_n;
    const int64_t grid = split > 1 ? tiles * split : tiles < sms ? tiles : sms;
    return fp8_launch(kern, grid, flp::kFp8TokThreads<kBN>, flp::kFp8TokSmem<kBN>, split, s, ta, tb, p, split);
}

// Which kernel: 0 = pairs on 256 x 256 tiles, else the tokens' kernel with that many rows
// of A a tile (16 .. 128) and `split` CTAs a tile.
struct Fp8Form {
    int bn, split;
};

Fp8Form fp8_form(int64_t M, int64_t N, int64_t nkb, bool b_square, int sms) {
    int bn = 16;
    while (bn < 128 && bn < M) bn *= 2;
    const int64_t tiles = ceil_div(M, bn) * ceil_div(N, 128);
    // Clusters of 4 and 8 leave SMs over (36 and 15 of them fit into 152), and one that waits for
    // another costs more than its split saves: 256 x 1024 x 4096 with 16 clusters of 8 took 19 us,
    // with 16 of 4 11.
    int split = 1;
    while (split < 8 && tiles * split * 2 <= sms * (split == 4 ? 15 : 18) / 20 && nkb >= 4 * split) split *= 2;
    // Up to 64 rows B's bytes bound it, and pairs use a quarter of their tiles at most: 64 x 151936
    // x 4096 takes 119 us, pairs 124.
    if (M <= 64) return Fp8Form{bn, split};
    // The times of either in ns, a wave of tiles and a K block of a tile at the rates measured (B
    // with one scale a block, with one a row). In us, tokens and pairs: 128 x 4096 x 4096 12 and 18;
    // 128 x 151936 x 4096 159 and 128, 144 and 183; 256 x 4096 x 4096 17.5 and 18, 16 and 26; 512 x
    // 4096 x 4096 24 and 18, 21 and 26; 384 x 8192 x 8192 75 and 31, 66 and 47.
    const int64_t waves = ceil_div(ceil_div(M, 256) * ceil_div(N, 256), sms / 2);
    const int64_t pairs = waves * (nkb * (b_square ? 370 : 640) + 2500) + 3500;
    const int64_t tok = ceil_div(tiles * split, sms) * (ceil_div(nkb, split) * (b_square ? 570 : 500) + 1000) + 3500 +
                        (split > 1 ? 2500 : 0);
    return pairs <= tok ? Fp8Form{0, 1} : Fp8Form{bn, split};
}

}  // namespace

cudaError_t flp_take_fp8_error(int* code) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, flp::g_fp8_error, sizeof v);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(flp::g_fp8_error, &zero, sizeof zero);
    *code = v;
    return e;
}

extern "C" {

flp_status flp_quantize_fp8(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, int square, void* q,
                            int64_t ld_q, float* scale, int64_t ld_scale, void* qt, int64_t ld_qt, float* scale_t,
                            int64_t ld_scale_t, flp_stream_t stream) {
    flp_status st;
    if ((st = check_dtype(dtype)) != FLP_OK) return st;
    if (rows < 0 || cols < 0)
        return fail(FLP_EINVAL, "rows and cols must be >= 0 (got %lld, %lld)", (long long)rows, (long long)cols);
    if (rows > kMaxSide || cols > kMaxSide) return fail(FLP_EUNSUPPORTED, "rows and cols must be below 2^31 - 1024");
    if ((q == nullptr) != (scale == nullptr) || (qt == nullptr) != (scale_t == nullptr))
        return fail(FLP_EINVAL, "q and scale, and qt and scale_t, go together");
    if (q == nullptr && qt == nullptr) return fail(FLP_EINVAL, "give q, qt or both");
    if (ld_x < cols) return fail(FLP_EINVAL, "ld_x (%lld) must be >= cols (%lld)", (long long)ld_x, (long long)cols);
    const int64_t rb = ceil_div(rows, 128), cb = ceil_div(cols, 128);
    const int64_t sw = square ? rb : rows, stw = square ? cb : cols;   // scales in a row of either
    if (q != nullptr && (ld_q < cols || ld_scale < sw))
        return fail(FLP_EINVAL, "ld_q (%lld) must be >= %lld and ld_scale (%lld) >= %lld", (long long)ld_q,
                    (long long)cols, (long long)ld_scale, (long long)sw);
    if (qt != nullptr && (ld_qt < rows || ld_scale_t < stw))
        return fail(FLP_EINVAL, "ld_qt (%lld) must be >= %lld and ld_scale_t (%lld) >= %lld", (long long)ld_qt,
                    (long long)rows, (long long)ld_scale_t, (long long)stw);
    if (rows == 0 || cols == 0) return ok();
    int64_t bx, bq = 0, bs = 0, bqt = 0, bst = 0;
    if (!span_bytes(rows, cols, ld_x, elem_bytes(dtype), &bx) || (q && !span_bytes(rows, cols, ld_q, 1, &bq)) ||
        (q && !span_bytes(cb, sw, ld_scale, 4, &bs)) || (qt && !span_bytes(cols, rows, ld_qt, 1, &bqt)) ||
        (qt && !span_bytes(rb, stw, ld_scale_t, 4, &bst)))
        return fail(FLP_EINVAL, "an extent overflows int64");
    const Extent e[5] = {{"q", q, bq}, {"scale", scale, bs}, {"qt", qt, bqt}, {"scale_t", scale_t, bst}, {"x", x, bx}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 5; ++j)
            if ((st = check_apart(e[i], e[j], false)) != FLP_OK) return st;
    const void* ptrs[] = {x, q, scale, qt, scale_t};
    const char* names[] = {"x", "q", "scale", "qt", "scale_t"};
    const bool optional[] = {false, true, true, true, true};
    int dev;
    if ((st = common_device(5, ptrs, names, optional, &dev)) != FLP_OK) return st;
    DeviceGuard guard;
    if ((st = guard.enter(dev)) != FLP_OK) return st;
    const flp::QuantArgs a{x, rows, cols, ld_x, square != 0, static_cast<uint8_t*>(q), ld_q, scale, ld_scale,
                           static_cast<uint8_t*>(qt), ld_qt, scale_t, ld_scale_t, cb,
                           reinterpret_cast<uintptr_t>(q) % 8 == 0 && ld_q % 8 == 0,
                           aligned16(qt) && ld_qt % 16 == 0};
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = rows_aligned16(x, ld_x, dtype);
    if (dtype == FLP_DTYPE_BF16) return launch_quantize<__nv_bfloat16>(a, vec, s);
    if (dtype == FLP_DTYPE_F16) return launch_quantize<__half>(a, vec, s);
    return launch_quantize<float>(a, vec, s);
}

flp_status flp_fp8_matmul(const void* a, int64_t m, int64_t k, int64_t ld_a, const float* a_scale, int64_t ld_a_scale,
                          const void* b, int64_t n, int64_t ld_b, const float* b_scale, int64_t ld_b_scale,
                          int b_square, void* c, int out_dtype, int64_t ld_c, flp_stream_t stream) {
    flp_status st;
    if ((st = check_dtype(out_dtype)) != FLP_OK) return st;
    if (m < 0 || n < 0 || k < 1)
        return fail(FLP_EINVAL, "m and n must be >= 0 and k >= 1 (got %lld, %lld, %lld)", (long long)m, (long long)n,
                    (long long)k);
    if (m > kMaxSide || n > kMaxSide || k > kMaxSide)
        return fail(FLP_EUNSUPPORTED, "m, n and k must be below 2^31 - 1024");
    if (ld_a < k || ld_b < k)
        return fail(FLP_EINVAL, "ld_a (%lld) and ld_b (%lld) must be >= k (%lld)", (long long)ld_a, (long long)ld_b,
                    (long long)k);
    if (ld_c < n) return fail(FLP_EINVAL, "ld_c (%lld) must be >= n (%lld)", (long long)ld_c, (long long)n);
    const int64_t nkb = ceil_div(k, 128), bw = b_square ? ceil_div(n, 128) : n;
    if (ld_a_scale < m || ld_b_scale < bw)
        return fail(FLP_EINVAL, "ld_a_scale (%lld) must be >= %lld and ld_b_scale (%lld) >= %lld",
                    (long long)ld_a_scale, (long long)m, (long long)ld_b_scale, (long long)bw);
    if (m == 0 || n == 0) return ok();
    // a single row's stride is not used: any that the tensor map takes
    const int64_t step_a = m == 1 ? ceil_div(k, 16) * 16 : ld_a, step_b = n == 1 ? ceil_div(k, 16) * 16 : ld_b;
    if (!aligned16(a) || !aligned16(b) || step_a % 16 || step_b % 16)
        return fail(FLP_EINVAL, "rows of a and b must start on 16-byte boundaries (ld_a %lld, ld_b %lld)",
                    (long long)ld_a, (long long)ld_b);
    int64_t ba, bb, bc, bas, bbs;
    if (!span_bytes(m, k, ld_a, 1, &ba) || !span_bytes(n, k, ld_b, 1, &bb) ||
        !span_bytes(m, n, ld_c, elem_bytes(out_dtype), &bc) || !span_bytes(nkb, m, ld_a_scale, 4, &bas) ||
        !span_bytes(nkb, bw, ld_b_scale, 4, &bbs))
        return fail(FLP_EINVAL, "an extent overflows int64");
    const Extent ec{"c", c, bc};
    for (const Extent& i : {Extent{"a", a, ba}, Extent{"b", b, bb}, Extent{"a_scale", a_scale, bas},
                            Extent{"b_scale", b_scale, bbs}})
        if ((st = check_apart(ec, i, false)) != FLP_OK) return st;
    const void* ptrs[] = {a, a_scale, b, b_scale, c};
    const char* names[] = {"a", "a_scale", "b", "b_scale", "c"};
    int dev;
    if ((st = common_device(5, ptrs, names, nullptr, &dev)) != FLP_OK) return st;
    if (dev < 0 || dev >= kMaxDevices) return fail(FLP_ECUDA, "device index %d out of range", dev);
    DeviceGuard guard;
    if ((st = guard.enter(dev)) != FLP_OK) return st;
    const int sms = sm_count(dev);
    if (sms <= 0) return fail(FLP_ECUDA, "could not read the SM count of device %d", dev);

    const Fp8Form f = fp8_form(m, n, nkb, b_square != 0, sms);
    flp::Fp8Args p{m, n, (int)nkb, a_scale, b_scale, ld_a_scale, ld_b_scale, b_square ? 7 : 0, c, ld_c, out_dtype,
                   rows_aligned16(c, ld_c, out_dtype), 0, 0, 0};
    CUtensorMap ta, tb;
    if ((st = fp8_tmap(&ta, "a", CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a, m, k, step_a, (uint32_t)(f.bn ? f.bn : 128))) != FLP_OK) return st;
    if ((st = fp8_tmap(&tb, "b", CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, b, n, k, step_b, 128)) != FLP_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (f.bn == 0) {
        p.tiles_m = ceil_div(m, 256);
        p.tiles_n = ceil_div(n, 256);
        p.group = 16;
        CUtensorMap tc = ta;   // not read unless p.vec
        p.vec = p.vec && ld_c <= kMaxSide;   // the map's strides are below 2^40 bytes
        if (p.vec) {
            const CUtensorMapDataType type = out_dtype == FLP_DTYPE_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : out_dtype == FLP_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
            if ((st = fp8_tmap(&tc, "c", type, elem_bytes(out_dtype), c, m, n, ld_c, 32)) != FLP_OK) return st;
        }
        if (b_square) return launch_pair<0>(p, ta, tb, tc, dev, sms, s);
        const bool fours = aligned16(b_scale) && ld_b_scale % 4 == 0 && n % 4 == 0;
        return fours ? launch_pair<2>(p, ta, tb, tc, dev, sms, s) : launch_pair<1>(p, ta, tb, tc, dev, sms, s);
    }
    p.tiles_m = ceil_div(m, f.bn);
    p.tiles_n = ceil_div(n, 128);
    switch (f.bn) {
        case 16: return launch_tokens<16>(p, ta, tb, dev, sms, f.split, s);
        case 32: return launch_tokens<32>(p, ta, tb, dev, sms, f.split, s);
        case 64: return launch_tokens<64>(p, ta, tb, dev, sms, f.split, s);
        default: return launch_tokens<128>(p, ta, tb, dev, sms, f.split, s);
    }
}

flp_status flp_selftest_fp8_wait(int device, int aborted, int* gave_up) {
    if (gave_up == nullptr) return fail(FLP_EINVAL, "gave_up is a null pointer");
    DeviceGuard guard;
    flp_status st;
    if ((st = guard.enter(device)) != FLP_OK) return st;
    flp::k_fp8_wait_selftest<<<1, 32>>>(aborted != 0);
    if ((st = check_launch("fp8 wait self-test")) != FLP_OK) return st;
    const cudaError_t e = cudaMemcpyFromSymbol(gave_up, flp::g_fp8_selftest, sizeof *gave_up);
    if (e != cudaSuccess) return fail(FLP_ECUDA, "fp8 wait self-test: %s", cudaGetErrorString(e));
    return ok();
}

flp_status flp_selftest_fp8_form(int64_t m, int64_t n, int64_t k, int b_square, int sms, int* bn, int* split) {
    if (m < 1 || n < 1 || k < 1 || sms < 2 || bn == nullptr || split == nullptr)
        return fail(FLP_EINVAL, "m, n and k must be >= 1, sms >= 2 and the outputs not null");
    const Fp8Form f = fp8_form(m, n, ceil_div(k, 128), b_square != 0, sms);
    *bn = f.bn;
    *split = f.split;
    return ok();
}

}  // extern "C"
