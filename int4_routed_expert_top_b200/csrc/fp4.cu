// fp4.cu - C ABI of the 4-bit floating point operators (see include/coli_moe.h):
// the quantiser of rows and the grouped product with quantised weights.
#include <algorithm>

#include "coli_moe.h"
#include "common.cuh"
#include "fp4.cuh"
#include "host.cuh"

using namespace coli;

namespace {

bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool aligned16(const void* p) { return aligned_to(p, 16); }
int block_of(coli_fp4 fmt) { return fmt == COLI_NVFP4 ? 16 : 32; }
int words_of(coli_fp4 fmt, int K) { return (K / block_of(fmt) + 3) / 4; }

int fp4_ok(const char* what, coli_fp4 fmt, int64_t rows, int K) {
    if (fmt != COLI_MXFP4 && fmt != COLI_NVFP4) return fail(COLI_E_INVAL, "%s: bad format %d", what, (int)fmt);
    if (rows < 0 || rows > INT32_MAX) return fail(COLI_E_INVAL, "%s: %lld rows", what, (long long)rows);
    if (K < 32 || K % 32 || K > (1 << 20)) return fail(COLI_E_INVAL, "%s: K=%d is no multiple of 32 in [32, 2^20]", what, K);
    return COLI_OK;
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        sms = 148;
    return sms;
}

// Rows of an expert per tile: 32 for a CTA by itself, 224 for a pair of CTAs, whose
// weights then pass an SM once and not several times, at the price of a kernel that
// lays out the rows' scales and of longer starts and ends.  With experts of n = P / E rows
// on average (the counts are on the device), a stage of a tile of 32 takes 0.25 us and
// one of a pair as long as 1.6 of those, a row of tiles has E * R / 128 * K / 256 stages
// over 148 SMs, and pairs take some 5 us (20 stages) more to begin and end.  So pairs where
// (row tiles of 32) - 1.6 (row tiles of 224) of these rows take more than 20 stages an SM:
//                                          by itself, in pairs (us)
//   32 experts of 4096 x 6144, 16 rows         72.9   76.6
//                              33 rows         91.2   77.9
//                              97 rows          174   85.3
//                             385 rows          546    164
//   one matrix of 10240 x 6144, 33 rows        14.0   18.0
//                               65 rows        16.3   17.5
//                 10240 x 2048, 50 rows         8.8   10.8
//                              400 rows        22.5   15.2
//                 18944 x 6144, 193 rows       45.6   17.1
//   8 experts of 2048 x 2048, 50 rows           9.6   11.4
// and where that gives tiles for half of the 74 pairs at least; with fewer the cut tiles'
// joining takes more than it saves (one matrix of 4096 x 6144, 385 rows, 32 tiles: 22.9 and
// 28.2 us).  Once true it stays true for more rows (a tile of 224 begun counts for nothing
// until its rows make up for it), and with it the larger workspace.
constexpr int kFpSmallNT = 32, kFpLargeNT = 224;
bool pairs_apply(int64_t P, int K, int E, int R) {
    const int64_t n = (P + E - 1) / E;
    if (n <= kFpSmallNT) return false;
    const int64_t full = (n - 1) / kFpLargeNT, rest = (n - full * kFpLargeNT + 31) / 32;  // row tiles
    const int64_t tiles = (int64_t)E * ((R - 1) / 256 + 1) * (full + 1);
    const int64_t stages = (int64_t)E * ((R - 1) / 128 + 1) * ((K + 255) / 256);  // of a row of tiles
    const int64_t saved = 27 * full + std::max<int64_t>(0, 5 * rest - 8);         // rows of tiles, times 5
    constexpr int64_t enough = 20 * 5 * 148;
    return tiles >= 40 && (saved > enough || stages * saved > enough);
}

// bytes [rows][K/2], boxes of 128 bytes x box_rows, 128-byte swizzle
int encode_codes_map(CUtensorMap* m, const void* base, int64_t rows, int K, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(COLI_E_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)K / 2, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K / 2};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(COLI_E_CUDA, "codes tensor map encode failed (%d)", (int)r);
    return COLI_OK;
}

// scale tiles: rows of 512 bytes, boxes of box_rows
int encode_scales_map(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return fail(COLI_E_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {128, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {512};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(COLI_E_CUDA, "scales tensor map encode failed (%d)", (int)r);
    return COLI_OK;
}

// Row tiles of pairs at most, and the bytes of their scales (of a row: whole stages).
int64_t pair_row_tiles(int64_t P, int E) { return P / kFpLargeNT + E; }
size_t pair_scale_bytes(coli_fp4 fmt, int64_t P, int K, int E) {
    const int64_t words = (int64_t)((K + 255) / 256) * (fmt == COLI_NVFP4 ? 4 : 2);
    return (size_t)(pair_row_tiles(P, E) * words * ((kFpLargeNT + 127) / 128) * 512);
}
size_t partial_bytes(int NT) { return (size_t)kFpMaxGrid * 128 * NT * 4; }

template <typename T>
int launch_quantize(coli_fp4 fmt, coli_act act, dim3 grid, dim3 threads, const Fp4QuantArgs& a, int lg, const void* x, void* values, cudaStream_t st) {
    const bool nv = fmt == COLI_NVFP4, glu = act == COLI_ACT_SWIGLU;
    const auto kern = nv ? (glu ? fp4_quantize_kernel<T, true, true> : fp4_quantize_kernel<T, true, false>)
                         : (glu ? fp4_quantize_kernel<T, false, true> : fp4_quantize_kernel<T, false, false>);
    return launch_pdl(kern, grid, threads, 0, st, "fp4 quantize", a, lg, (const T*)x, (T*)values);
}

// what later products of this thread withhold (coli_moe_fp4_set_wait_test), -1: nothing
thread_local int32_t g_withhold = -1;

template <int NT, bool NV, bool PAIR, typename YT, bool TW = false>
int launch_product(const FpArgs& a, const void* x_codes, const void* w_codes, void* y, cudaStream_t st) {
    using C = FpShape<NT, NV, PAIR>;
    const auto kern = fp4_product_kernel<NT, NV, PAIR, YT, TW>;
    FpMaps<PAIR> maps;
    int rc;
    if ((rc = encode_codes_map(&maps.w, w_codes, (int64_t)a.E * a.R, a.K, 128))) return rc;
    if ((rc = encode_codes_map(&maps.x, x_codes, a.P, a.K, C::box))) return rc;
    if constexpr (PAIR) {
        const int64_t blocks = ((int64_t)a.E * a.R + 127) / 128, words = (int64_t)a.KS * C::atoms;
        if ((rc = encode_scales_map(&maps.ws, a.ws, blocks * a.wwords, C::atoms))) return rc;
        if ((rc = encode_scales_map(&maps.xs, a.xtiles, a.max_xtiles * words * C::nb, C::atoms * C::nb))) return rc;
        // a warp per two words of a tile, as many as the SMs hold at once
        const int64_t ctas = (a.max_xtiles * words / 2 + 7) / 8;
        if ((rc = launch_pdl(fp4_tile_scales_kernel<NT, C::M, C::nb>, dim3((unsigned)std::min<int64_t>(ctas, 8 * 148)),
                             kFpTileScaleThreads, 0, st, "fp4 product scales", a, (int)words)))
            return rc;
    }
    if ((rc = set_smem((const void*)kern, C::smem))) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(sm_count(), kFpMaxGrid) / C::ctas * C::ctas);
    cfg.blockDim = dim3(C::threads);
    cfg.dynamicSmemBytes = C::smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C::ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps, a, (YT*)y);
    if (e != cudaSuccess) return fail(COLI_E_CUDA, "fp4 product: %s", cudaGetErrorString(e));
    return check_launch("fp4 product");
}

template <int NT, bool PAIR>
int launch_product_t(coli_fp4 fmt, coli_dtype yt, const FpArgs& a, const void* x_codes, const void* w_codes, void* y,
                     cudaStream_t st) {
    if (a.withhold >= 0) {
        if (fmt != COLI_MXFP4 || yt != COLI_F32)
            return fail(COLI_E_UNSUPPORTED, "fp4_product: the wait test takes MXFP4 with f32 results");
        return launch_product<NT, false, PAIR, float, true>(a, x_codes, w_codes, y, st);
    }
    if (fmt == COLI_NVFP4)
        return yt == COLI_F32 ? launch_product<NT, true, PAIR, float>(a, x_codes, w_codes, y, st)
                              : launch_product<NT, true, PAIR, __nv_bfloat16>(a, x_codes, w_codes, y, st);
    return yt == COLI_F32 ? launch_product<NT, false, PAIR, float>(a, x_codes, w_codes, y, st)
                          : launch_product<NT, false, PAIR, __nv_bfloat16>(a, x_codes, w_codes, y, st);
}

}  // namespace

extern "C" {

int coli_moe_fp4_bytes(coli_fp4 fmt, int64_t rows, int32_t K, size_t* code_bytes, size_t* scale_bytes) {
    const int rc = fp4_ok("fp4_bytes", fmt, rows, K);
    if (rc) return rc;
    if (!code_bytes || !scale_bytes) return fail(COLI_E_INVAL, "fp4_bytes: NULL pointer");
    *code_bytes = (size_t)rows * (K / 2);
    *scale_bytes = (size_t)((rows + 127) / 128) * words_of(fmt, K) * 512;
    return COLI_OK;
}

int coli_moe_fp4_quantize(coli_fp4 fmt, const void* x, coli_dtype xt, int64_t n_src, int64_t rows, int32_t K,
                          coli_act act, const int32_t* src, const int32_t* count, const float* gscale, void* codes,
                          void* scales, void* values, coli_stream_t stream) {
    int rc = fp4_ok("fp4_quantize", fmt, rows, K);
    if (rc) return rc;
    if (xt != COLI_F32 && xt != COLI_BF16) return fail(COLI_E_INVAL, "fp4_quantize: bad dtype");
    if (act != COLI_ACT_NONE && act != COLI_ACT_SWIGLU) return fail(COLI_E_INVAL, "fp4_quantize: bad act %d", (int)act);
    if (gscale && fmt == COLI_MXFP4) return fail(COLI_E_INVAL, "fp4_quantize: MXFP4 has no f32 scale");
    if (n_src < 0 || (!src && n_src < rows))
        return fail(COLI_E_INVAL, "fp4_quantize: %lld source rows", (long long)n_src);
    if (rows == 0) return COLI_OK;
    if ((!x && n_src > 0) || !codes || !scales) return fail(COLI_E_INVAL, "fp4_quantize: NULL pointer");
    if (!aligned_to(x, 32) || !aligned_to(codes, 16) || !aligned_to(scales, 16) || !aligned_to(values, 32))
        return fail(COLI_E_INVAL, "fp4_quantize: x and values must be 32-byte aligned, codes and scales 16-byte");
    if ((rc = elements_ok("fp4_quantize", {{src, 4}, {count, 4}, {gscale, 4}}))) return rc;
    Fp4QuantArgs a;
    a.n_src = (uint32_t)std::min<int64_t>(n_src, (int64_t)1 << 31);  // src holds 31-bit indexes
    a.rows = (int)rows; a.K = K; a.words = words_of(fmt, K);
    a.src = src; a.count = count; a.gscale = gscale;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint32_t*>(scales);
    // a warp per chunk of a row, several rows to a CTA or a warp where they are short
    const int lg = K > 256 ? 5 : K > 128 ? 4 : 3;
    const int chunks = (K + kQuantCols - 1) / kQuantCols;
    const int parts = (chunks + kQuantWarps - 1) / kQuantWarps, warps = (chunks + parts - 1) / parts;
    const int rows_per = std::max(1, 8 / warps);
    const int cta_rows = rows_per << (5 - lg);
    const dim3 grid((unsigned)((rows + cta_rows - 1) / cta_rows), parts);
    const dim3 threads(32 * warps, rows_per);
    if (xt == COLI_F32)
        return launch_quantize<float>(fmt, act, grid, threads, a, lg, x, values, S(stream));
    return launch_quantize<__nv_bfloat16>(fmt, act, grid, threads, a, lg, x, values, S(stream));
}

int coli_moe_fp4_product_workspace_size(coli_fp4 fmt, int64_t P, int32_t K, int32_t E, int32_t R, size_t* bytes) {
    const int rc = fp4_ok("fp4_product", fmt, P, K);
    if (rc) return rc;
    if (!bytes) return fail(COLI_E_INVAL, "fp4_product_workspace_size: NULL pointer");
    if (E < 1 || E > kFpMaxE || R < 1 || (E > 1 && R % 128) || (int64_t)E * R > INT32_MAX)
        return fail(COLI_E_INVAL, "fp4_product: bad sizes E=%d R=%d", E, R);
    *bytes = kFpHeadBytes + (pairs_apply(P, K, E, R) ? partial_bytes(kFpLargeNT) + pair_scale_bytes(fmt, P, K, E)
                                                  : partial_bytes(kFpSmallNT));
    return COLI_OK;
}

int coli_moe_fp4_product(coli_fp4 fmt, const void* x_codes, const void* x_scales, int64_t P, int32_t K,
                         const void* w_codes, const void* w_scales, int32_t E, int32_t R, const int32_t* offsets,
                         const float* alpha, void* y, coli_dtype yt, void* ws, size_t ws_bytes, coli_stream_t stream) {
    size_t need;
    int rc = coli_moe_fp4_product_workspace_size(fmt, P, K, E, R, &need);
    if (rc) return rc;
    if (yt != COLI_F32 && yt != COLI_BF16) return fail(COLI_E_INVAL, "fp4_product: bad dtype");
    if (!offsets && E > 1) return fail(COLI_E_INVAL, "fp4_product: %d experts need offsets", E);
    if (P == 0) return COLI_OK;
    if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return fail(COLI_E_INVAL, "fp4_product: NULL pointer");
    if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales))
        return fail(COLI_E_INVAL, "fp4_product: codes and scales must be 16-byte aligned");
    if (!ws || ws_bytes < need || !aligned16(ws))
        return fail(COLI_E_WORKSPACE, "fp4_product: workspace of %zu bytes, %zu needed", ws ? ws_bytes : 0, need);
    if ((rc = elements_ok("fp4_product", {{offsets, 4}, {alpha, 4}, {y, yt == COLI_F32 ? 4 : 2}}))) return rc;
    FpArgs a;
    a.xs = static_cast<const uint32_t*>(x_scales);
    a.ws = static_cast<const uint8_t*>(w_scales);
    a.P = P;
    a.K = K; a.E = E; a.R = R;
    a.KS = (K + 255) / 256;
    a.xwords = a.wwords = words_of(fmt, K);
    a.offsets = offsets; a.alpha = alpha;
    a.err = static_cast<uint64_t*>(ws);
    a.withhold = g_withhold;
    a.flags = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + kFpFlagBytes);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kFpHeadBytes);
    a.xtiles = reinterpret_cast<uint4*>(static_cast<char*>(ws) + kFpHeadBytes + partial_bytes(kFpLargeNT));  // pairs
    a.max_xtiles = pair_row_tiles(P, E);
    if (pairs_apply(P, K, E, R)) return launch_product_t<kFpLargeNT, true>(fmt, yt, a, x_codes, w_codes, y, S(stream));
    return launch_product_t<kFpSmallNT, false>(fmt, yt, a, x_codes, w_codes, y, S(stream));
}

int coli_moe_fp4_product_status(const void* ws, int32_t* flags, coli_stream_t stream) {
    if (!ws || !flags) return fail(COLI_E_INVAL, "fp4_product_status: NULL pointer");
    uint64_t word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, ws, sizeof(word), cudaMemcpyDeviceToHost, S(stream));
    if (e == cudaSuccess) e = cudaStreamSynchronize(S(stream));
    if (e != cudaSuccess) return fail(COLI_E_CUDA, "fp4_product_status: %s", cudaGetErrorString(e));
    *flags = word == kFpBroken ? kErrWaitTimeout : 0;
    if (*flags) return fail(COLI_E_TIMEOUT, "fp4_product: a bounded wait gave up; the workspace has to be cleared");
    return COLI_OK;
}

int coli_moe_fp4_set_wait_test(int32_t withhold) {
    if (withhold > 1) return fail(COLI_E_INVAL, "fp4_set_wait_test: nothing to withhold named %d", withhold);
    g_withhold = withhold < 0 ? -1 : withhold;
    return COLI_OK;
}

}  // extern "C"
