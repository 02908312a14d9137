// block.cu - C ABI of the operators around the experts (see include/coli_moe.h):
// sort, dispatch and combine with their gradients, and the norms between blocks.
// Host code validates arguments and launches the kernels of rows.cuh and
// norm.cuh on the caller's stream.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <utility>

#include "coli_moe.h"
#include "common.cuh"
#include "host.cuh"
#include "norm.cuh"
#include "rows.cuh"

using namespace coli;

namespace {

bool type_ok(int t) { return t == COLI_F32 || t == COLI_BF16; }
int type_size(int t) { return t == COLI_F32 ? 4 : 2; }

bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// what every call on picks checks
int picks_ok(const char* what, int T, int k) {
    if (T < 0 || k < 1 || k > 32 || (int64_t)T * k > (1 << 30))
        return fail(COLI_E_INVAL, "%s: bad sizes T=%d k=%d", what, T, k);
    return COLI_OK;
}

int rows_ok(const char* what, int T, int H, int k) {
    const int rc = picks_ok(what, T, k);
    if (rc) return rc;
    if (H < 1 || H > (1 << 24) || (int64_t)T * ((H + 255) / 256) > INT32_MAX)  // one CTA per 256 columns at most
        return fail(COLI_E_INVAL, "%s: bad sizes T=%d H=%d", what, T, H);
    return COLI_OK;
}

int64_t sort_chunk(int64_t P) {
    const int64_t group = 32 * kSortWarps;
    return ((P + kSortMaxChunks - 1) / kSortMaxChunks + group - 1) / group * group;
}

template <typename V, int N>
int launch_dispatch(const void* x, int T, int nvec, int k, const int32_t* inv, void* xs, cudaStream_t st) {
    const int per = (nvec + 256 * N - 1) / (256 * N);
    return launch_pdl(dispatch_kernel<V, N>, dim3((unsigned)T * per), 256, 0, st, "dispatch", (const V*)x,
                      (int64_t)T * k, nvec, per, k, inv, (V*)xs);
}

// How many neighbouring elements an access may take: `most`, 2 or 1, by the row
// length and every pointer's alignment (sizes: of the elements behind them).
template <int most>
int chunk_of(int H, std::initializer_list<std::pair<const void*, int>> buffers) {
    for (int w : {most, 2}) {
        bool ok = H % w == 0;
        for (const auto& b : buffers) ok = ok && aligned(b.first, w * b.second);
        if (ok) return w;
    }
    return 1;
}

template <typename OT, typename YT>
int launch_rows_sum(const void* o, int T, int H, int k, const int32_t* inv, const float* w,
                    const void* residual, void* y, cudaStream_t st) {
    constexpr int N = 16 / sizeof(OT);  // columns of a lane: 16 bytes of o
    const int W = chunk_of<N>(H, {{o, (int)sizeof(OT)}, {residual, (int)sizeof(YT)}, {y, (int)sizeof(YT)}});
    const int64_t items = (int64_t)T * ((H + 32 * N - 1) / (32 * N));
    const auto kern = W == N ? rows_sum_kernel<OT, YT, N, N>
                             : W == 2 ? rows_sum_kernel<OT, YT, N, 2> : rows_sum_kernel<OT, YT, N, 1>;
    // as many CTAs as the SMs hold, and no more than there are warps of work
    const int grid = (int)std::min<int64_t>((items + 7) / 8, (W == N ? 3 : 2) * 148);
    return launch_pdl(kern, dim3(grid), 256, 0, st, "combine", (const OT*)o, (int64_t)T * k, T, H, k, inv, w,
                      (const YT*)residual, (YT*)y);
}

int rows_sum(const char* what, const void* o, coli_dtype ot, int T, int H, int k, const int32_t* inv, const float* w,
             const void* residual, void* y, coli_dtype yt, cudaStream_t st) {
    const int rc = rows_ok(what, T, H, k);
    if (rc) return rc;
    if (!type_ok(ot) || !type_ok(yt)) return fail(COLI_E_INVAL, "%s: bad dtype", what);
    if (T == 0) return COLI_OK;
    if (!o || !inv || !y) return fail(COLI_E_INVAL, "%s: NULL pointer", what);
    const int os = type_size(ot), ys = type_size(yt), el = elements_ok(what, {{o, os}, {inv, 4}, {w, 4}, {residual, ys}, {y, ys}});
    if (el) return el;
    if (ot == COLI_F32)
        return yt == COLI_F32 ? launch_rows_sum<float, float>(o, T, H, k, inv, w, residual, y, st)
                              : launch_rows_sum<float, __nv_bfloat16>(o, T, H, k, inv, w, residual, y, st);
    return yt == COLI_F32 ? launch_rows_sum<__nv_bfloat16, float>(o, T, H, k, inv, w, residual, y, st)
                          : launch_rows_sum<__nv_bfloat16, __nv_bfloat16>(o, T, H, k, inv, w, residual, y, st);
}

template <typename YT, typename OT>
int launch_rows_sum_backward(const void* dy, const void* o, int T, int H, int k, const int32_t* inv,
                             const float* w, void* d_o, float* dw, cudaStream_t st) {
    constexpr int N = 16 / sizeof(OT);
    const int W = chunk_of<N>(H, {{o, (int)sizeof(OT)}, {d_o, (int)sizeof(OT)}, {dy, (int)sizeof(YT)}});
    const auto kern = W == N ? rows_sum_backward_kernel<YT, OT, N, N>
                             : W == 2 ? rows_sum_backward_kernel<YT, OT, N, 2> : rows_sum_backward_kernel<YT, OT, N, 1>;
    return launch_pdl(kern, dim3((unsigned)(((int64_t)T * k + 7) / 8)), 256, 0, st, "combine backward",
                      (const YT*)dy, (const OT*)o, (int64_t)T * k, H, k, inv, w, (OT*)d_o, dw);
}

int norm_ok(const char* what, const coli_norm_desc* d, int T) {
    if (!d) return fail(COLI_E_INVAL, "%s: NULL descriptor", what);
    if (d->H < 1 || d->H > kNormMaxH || T < 0) return fail(COLI_E_INVAL, "%s: bad sizes T=%d H=%d", what, T, d->H);
    if (!type_ok(d->xt) || !type_ok(d->bt)) return fail(COLI_E_INVAL, "%s: bad dtype", what);
    if (d->xt == COLI_BF16 && d->bt == COLI_F32)
        return fail(COLI_E_UNSUPPORTED, "%s: f32 blocks on a bf16 stream", what);
    if (d->gate_kind < COLI_GATE_NONE || d->gate_kind > COLI_GATE_FULL)
        return fail(COLI_E_INVAL, "%s: bad gate_kind %d", what, d->gate_kind);
    if (!(d->eps > 0.0f) || !std::isfinite(d->eps) || !std::isfinite(d->alpha))
        return fail(COLI_E_INVAL, "%s: eps must be positive, eps and alpha finite", what);
    return COLI_OK;
}

NormArgs norm_args(const coli_norm_desc& d, const float* gate, int T) {
    NormArgs a;
    a.H = d.H; a.T = T;
    a.post_norm = d.post_norm != 0;
    a.gate_kind = d.gate_kind;
    a.alpha = d.alpha; a.eps = d.eps;
    a.post_gain = d.post_gain; a.pre_gain = d.pre_gain;
    a.gate = gate;
    return a;
}

// neighbours of an access, vectors of eight per thread and threads of a row
struct NormShape { int W, N, threads; };
// Forward, many tokens: about 256 threads a row, so that an SM holds several rows; few
// (less than two rows per SM): one vector a thread (the time of one row is what
// counts).  Rows without 16-byte access need more registers a vector, so fewer vectors
// (4000 x 6143, f32 stream: 85 us with two, 97 with three).  Backward: one vector a
// thread where a CTA can be that large (the same rows: 194 us, with three 356).
NormShape norm_shape(int H, int T, int W, bool backward) {
    NormShape s;
    s.W = W;
    const int vecs = (H + 7) / 8;
    if (vecs <= (backward ? 768 : T < 2 * 148 ? 1024 : 256))
        s.N = 1;
    else
        s.N = vecs <= (W == 8 ? 512 : 1024) ? 2 : vecs <= 3 * 512 ? 3 : 4;
    s.threads = ((vecs + s.N - 1) / s.N + 31) / 32 * 32;
    return s;
}

// calls the kernel with its type and shape parameters as template arguments
template <template <typename, typename, int, int> class K, typename XT, typename BT, int W, typename... A>
int norm_launch_w(const NormShape& s, A... args) {
    if (s.N == 1) return K<XT, BT, W, 1>::launch(s, args...);
    if (s.N == 2) return K<XT, BT, W, 2>::launch(s, args...);
    if (s.N == 3) return K<XT, BT, W, 3>::launch(s, args...);
    return K<XT, BT, W, 4>::launch(s, args...);
}
template <template <typename, typename, int, int> class K, typename XT, typename BT, typename... A>
int norm_launch(const NormShape& s, A... args) {
    if (s.W == 8) return norm_launch_w<K, XT, BT, 8>(s, args...);
    if (s.W == 2) return norm_launch_w<K, XT, BT, 2>(s, args...);
    return norm_launch_w<K, XT, BT, 1>(s, args...);
}
template <template <typename, typename, int, int> class K, typename... A>
int norm_dispatch(const coli_norm_desc& d, const NormShape& s, A... args) {
    if (d.bt == COLI_F32) return norm_launch<K, float, float>(s, args...);
    if (d.xt == COLI_F32) return norm_launch<K, float, __nv_bfloat16>(s, args...);
    return norm_launch<K, __nv_bfloat16, __nv_bfloat16>(s, args...);
}

template <typename XT, typename BT, int W, int N>
struct NormForward {
    static int launch(const NormShape& s, const NormArgs& a, const void* x, const void* o, void* x_out,
                      void* n_out, float* rstd_post, float* rstd_pre, cudaStream_t st) {
        return launch_pdl(block_norm_kernel<XT, BT, W, N>, dim3(a.T), s.threads, 0, st, "block norm", a,
                          (const XT*)x, (const BT*)o, (XT*)x_out, (BT*)n_out, rstd_post, rstd_pre);
    }
};

// The backward pass: with many tokens, CTAs whose rows come through a ring (their
// sums over tokens fill the registers: 8192 columns at 512 threads); else as many CTAs
// per SM as its registers hold.  Clusters of two add the sums over tokens before they
// leave an SM (clusters of four leave SMs without a CTA where a GPC's number of them is no
// multiple of four: the ring's 37 did not fit at once and took twice as long).
constexpr int kNormSms = 148;
constexpr int kNormRingMaxH = 8192;
constexpr int kNormRingBytes = 224 * 1024;   // of an SM
constexpr int kNormCluster = 2;
int norm_backward_cluster(int grid) { return grid >= kNormCluster ? kNormCluster : 1; }
// CTAs of the plain form: 768 threads per SM (80 registers each), at most 8 CTAs (4000
// tokens of 130: 19 us, with 16 27 us, for the sums of every CTA are added up), and
// their sums in 200 KB of shared memory
int norm_plain_ctas(const coli_norm_desc& d, int T) {
    const int threads = norm_shape(d.H, T, 1, true).threads;
    return kNormSms * std::max(1, std::min({8, 768 / threads, 200 * 1024 / (kNormKept * d.H * 4)}));
}
int norm_backward_grid(int T, int ctas) {
    const int grid = std::min(T, ctas);
    return grid / norm_backward_cluster(grid) * norm_backward_cluster(grid);
}
// CTAs of the ring form: as many per SM as have two stages with every input, at
// most six, and two rows or more for each; 0 where that leaves none
int norm_ring_ctas(const coli_norm_desc& d, int T) {
    const int need = 2 * d.H * 4 + 2 * 2 * d.H * (type_size(d.xt) + type_size(d.bt));
    const int per_sm = std::min({6, kNormRingBytes / need, T / (2 * kNormSms)});
    return d.H <= kNormRingMaxH && d.H % 8 == 0 ? per_sm * kNormSms : 0;
}

// the ring of a call: no stages where it does not apply
NormRing norm_ring(const coli_norm_desc& d, int ctas, bool wide, bool x_out, bool dx_out, bool o, bool dn) {
    NormRing r = {0, 0, {-1, -1, -1, -1}, {-1, -1}, 0};
    if (!wide || ctas < 1) return r;
    const bool vec[2] = {dn, o && d.gate_kind != COLI_GATE_FULL};
    for (int i = 0; i < 2; ++i) {
        if (!vec[i]) continue;
        r.gain[i] = r.first;
        r.first += d.H * 4;
    }
    const bool has[4] = {x_out, dx_out, o, dn};
    for (int i = 0; i < 4; ++i) {
        if (!has[i]) continue;
        r.off[i] = r.stage;
        r.stage += d.H * type_size(i < 2 ? d.xt : d.bt);
    }
    r.stages = std::min(kNormMaxStages, (kNormRingBytes / (ctas / kNormSms) - 1024 - r.first) / r.stage);
    // room for the sums at the end as well
    if (r.stages < 2 || kNormKept * d.H * 4 > r.first + r.stages * r.stage) r.stages = 0;
    return r;
}

// the row of CTA 0 that later gradients of this thread do not copy
// (coli_moe_block_norm_set_wait_test), -1: none
thread_local int32_t g_norm_withhold = -1;

template <typename XT, typename BT, int W, int N, bool RING, bool TW = false>
struct NormBackward {
    static int launch(const NormShape& s, const NormArgs& a, const NormSums& keep, const NormRing& ring,
                      const void* x_out, const void* o, const float* rstd_post, const float* rstd_pre,
                      const void* dx_out, const void* dn, void* dx, void* d_o, float* dgate, float* partial, int grid,
                      cudaStream_t st) {
        const auto kern = block_norm_backward_kernel<XT, BT, W, N, RING, TW>;
        const int smem = RING ? ring.first + ring.stages * ring.stage : std::min(keep.n, kNormKept) * a.H * 4;
        int rc = set_smem((const void*)kern, smem);
        if (rc) return rc;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(s.threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = norm_backward_cluster(grid);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, keep, ring, (const XT*)x_out, (const BT*)o, rstd_post,
                                                 rstd_pre, (const XT*)dx_out, (const BT*)dn, (XT*)dx, (BT*)d_o, dgate,
                                                 partial, (int)g_norm_withhold);
        if (e != cudaSuccess) return fail(COLI_E_CUDA, "block norm backward: %s", cudaGetErrorString(e));
        return check_launch("block norm backward");
    }
};
template <typename XT, typename BT, int W, int N> using NormBackwardPlain = NormBackward<XT, BT, W, N, false>;

// ring rows: one or two vectors of eight per thread
template <typename XT, typename BT, typename... A>
int norm_ring_launch(const NormShape& s, A... args) {
    if (s.N == 1) return NormBackward<XT, BT, 8, 1, true>::launch(s, args...);
    return NormBackward<XT, BT, 8, 2, true>::launch(s, args...);
}
template <typename... A>
int norm_ring_dispatch(const coli_norm_desc& d, const NormShape& s, A... args) {
    if (g_norm_withhold >= 0) return NormBackward<float, __nv_bfloat16, 8, 1, true, true>::launch(s, args...);
    if (d.bt == COLI_F32) return norm_ring_launch<float, float>(s, args...);
    if (d.xt == COLI_F32) return norm_ring_launch<float, __nv_bfloat16>(s, args...);
    return norm_ring_launch<__nv_bfloat16, __nv_bfloat16>(s, args...);
}

}  // namespace

extern "C" {

int coli_moe_sort_workspace_size(int32_t T, int32_t k, int32_t E, size_t* bytes) {
    if (!bytes) return fail(COLI_E_INVAL, "sort_workspace_size: NULL pointer");
    const int rc = picks_ok("sort_workspace_size", T, k);
    if (rc) return rc;
    if (E < 1 || E > 1024) return fail(COLI_E_INVAL, "sort_workspace_size: E=%d outside [1, 1024]", E);
    // counts of the most chunks that P picks or fewer are cut into: a chunk grows by whole groups of
    // picks, so that a few more picks may need fewer chunks, and a workspace for P serves fewer too
    const int64_t P = (int64_t)T * k, group = 32 * kSortWarps;
    *bytes = P <= kSortOneCta ? 0 : (size_t)std::min<int64_t>((P + group - 1) / group, kSortMaxChunks) * E * 4;
    return COLI_OK;
}

int coli_moe_sort(const int32_t* idx, const float* w, int32_t T, int32_t k, int32_t E,
                  int32_t* offsets, int32_t* pair_tok, int32_t* pair_slot, int32_t* inv, void* ws,
                  size_t ws_bytes, coli_stream_t stream) {
    size_t need;
    int rc = coli_moe_sort_workspace_size(T, k, E, &need);
    if (rc) return rc;
    if (!offsets || (T > 0 && (!idx || !inv))) return fail(COLI_E_INVAL, "sort: NULL pointer");
    if (need && (!ws || ws_bytes < need || !aligned(ws, 4)))
        return fail(COLI_E_WORKSPACE, "sort: workspace of %zu bytes, %zu needed", ws ? ws_bytes : 0, need);
    if ((rc = elements_ok("sort", {{idx, 4}, {w, 4}, {offsets, 4}, {pair_tok, 4}, {pair_slot, 4}, {inv, 4}}))) return rc;
    const int64_t P = (int64_t)T * k;
    const int one_smem = (kSortWarps * E + E + 1) * 4, place_smem = one_smem + E * 4;
    if (P <= kSortOneCta) {
        if ((rc = set_smem((const void*)sort_one_kernel, one_smem))) return rc;
        return launch_pdl(sort_one_kernel, dim3(1), kSortThreads, one_smem, S(stream), "sort", idx, w, (int)P,
                          (int)k, (int)E, offsets, pair_tok, pair_slot, inv);
    }
    const int64_t chunk = sort_chunk(P);
    const dim3 grid((unsigned)((P + chunk - 1) / chunk));
    int32_t* counts = static_cast<int32_t*>(ws);
    const int count_smem = kSortWarps * E * 4;
    if ((rc = set_smem((const void*)sort_count_kernel, count_smem))) return rc;
    if ((rc = set_smem((const void*)sort_place_kernel, place_smem))) return rc;
    if ((rc = launch_pdl(sort_count_kernel, grid, kSortThreads, count_smem, S(stream), "sort count", idx, w, P,
                         chunk, (int)E, counts)))
        return rc;
    return launch_pdl(sort_place_kernel, grid, kSortThreads, place_smem, S(stream), "sort place", idx, w, P, chunk,
                      (int)k, (int)E, (const int32_t*)counts, offsets, pair_tok, pair_slot, inv);
}

int coli_moe_dispatch(const void* x, coli_dtype xt, int32_t T, int32_t H, int32_t k,
                      const int32_t* inv, void* xs, coli_stream_t stream) {
    int rc = rows_ok("dispatch", T, H, k);
    if (rc) return rc;
    if (!type_ok(xt)) return fail(COLI_E_INVAL, "dispatch: bad dtype");
    if (T == 0) return COLI_OK;
    if (!x || !inv || !xs) return fail(COLI_E_INVAL, "dispatch: NULL pointer");
    if ((rc = elements_ok("dispatch", {{x, type_size(xt)}, {inv, 4}, {xs, type_size(xt)}}))) return rc;
    const int64_t bytes = (int64_t)H * type_size(xt);
    if (bytes % 16 == 0 && aligned(x, 16) && aligned(xs, 16))
        return launch_dispatch<uint4, 1>(x, T, (int)(bytes / 16), k, inv, xs, S(stream));
    if (bytes % 4 == 0 && aligned(x, 4) && aligned(xs, 4))
        return launch_dispatch<uint32_t, 4>(x, T, (int)(bytes / 4), k, inv, xs, S(stream));
    return launch_dispatch<uint16_t, 8>(x, T, (int)(bytes / 2), k, inv, xs, S(stream));
}

int coli_moe_dispatch_backward(const void* dxs, coli_dtype xt, int32_t T, int32_t H, int32_t k,
                               const int32_t* inv, void* dx, coli_stream_t stream) {
    return rows_sum("dispatch_backward", dxs, xt, T, H, k, inv, nullptr, nullptr, dx, xt, S(stream));
}

int coli_moe_combine(const void* o, coli_dtype ot, int32_t T, int32_t H, int32_t k,
                     const int32_t* inv, const float* w, const void* residual, void* y,
                     coli_dtype yt, coli_stream_t stream) {
    return rows_sum("combine", o, ot, T, H, k, inv, w, residual, y, yt, S(stream));
}

int coli_moe_combine_backward(const void* dy, coli_dtype yt, const void* o, coli_dtype ot, int32_t T,
                              int32_t H, int32_t k, const int32_t* inv, const float* w, void* d_o,
                              float* dw, coli_stream_t stream) {
    int rc = rows_ok("combine_backward", T, H, k);
    if (rc) return rc;
    if (!type_ok(ot) || !type_ok(yt)) return fail(COLI_E_INVAL, "combine_backward: bad dtype");
    if (T == 0) return COLI_OK;
    if (!dy || !inv || (!d_o && !dw) || (dw && !o)) return fail(COLI_E_INVAL, "combine_backward: NULL pointer");
    if ((rc = elements_ok("combine_backward", {{dy, type_size(yt)}, {o, type_size(ot)}, {inv, 4}, {w, 4},
                                               {d_o, type_size(ot)}, {dw, 4}})))
        return rc;
    if (yt == COLI_F32)
        return ot == COLI_F32 ? launch_rows_sum_backward<float, float>(dy, o, T, H, k, inv, w, d_o, dw, S(stream))
                              : launch_rows_sum_backward<float, __nv_bfloat16>(dy, o, T, H, k, inv, w, d_o, dw, S(stream));
    return ot == COLI_F32
               ? launch_rows_sum_backward<__nv_bfloat16, float>(dy, o, T, H, k, inv, w, d_o, dw, S(stream))
               : launch_rows_sum_backward<__nv_bfloat16, __nv_bfloat16>(dy, o, T, H, k, inv, w, d_o, dw, S(stream));
}

int coli_moe_block_norm(const coli_norm_desc* desc, const void* x, const void* o, const float* gate,
                        int32_t T, void* x_out, void* n_out, float* rstd_post, float* rstd_pre,
                        coli_stream_t stream) {
    int rc = norm_ok("block_norm", desc, T);
    if (rc) return rc;
    if (T == 0) return COLI_OK;
    if (!x || (o && !x_out) || (!o && !n_out)) return fail(COLI_E_INVAL, "block_norm: NULL pointer");
    if (o && (desc->gate_kind != COLI_GATE_NONE) != (gate != nullptr))
        return fail(COLI_E_INVAL, "block_norm: gate and gate_kind disagree");
    const int xs = type_size(desc->xt), bs = type_size(desc->bt);
    if ((rc = elements_ok("block_norm", {{x, xs}, {x_out, xs}, {o, bs}, {n_out, bs}, {desc->post_gain, 4},
                                         {desc->pre_gain, 4}, {gate, 4}, {rstd_post, 4}, {rstd_pre, 4}})))
        return rc;
    const int W = chunk_of<8>(desc->H, {{x, xs}, {x_out, xs}, {o, bs}, {n_out, bs}, {desc->post_gain, 4},
                                        {desc->pre_gain, 4}, {gate, 4}});
    const NormArgs a = norm_args(*desc, gate, T);
    return norm_dispatch<NormForward>(*desc, norm_shape(desc->H, T, W, false), a, x, o, x_out, n_out, rstd_post, rstd_pre,
                                      S(stream));
}

int coli_moe_block_norm_backward_workspace_size(const coli_norm_desc* desc, int32_t T, size_t* bytes) {
    int rc = norm_ok("block_norm_backward_workspace_size", desc, T);
    if (rc) return rc;
    if (!bytes) return fail(COLI_E_INVAL, "block_norm_backward_workspace_size: NULL pointer");
    const int grid = norm_backward_grid(T, std::max(norm_plain_ctas(*desc, T), norm_ring_ctas(*desc, T)));  // of either form
    *bytes = (size_t)(grid / norm_backward_cluster(grid)) * kNormSums * desc->H * 4;
    return COLI_OK;
}

int coli_moe_block_norm_backward(const coli_norm_desc* desc, const void* x_out, const void* o,
                                 const float* gate, int32_t T, const float* rstd_post,
                                 const float* rstd_pre, const void* dx_out, const void* dn, void* dx,
                                 void* d_o, float* dpost_gain, float* dgate, float* dpre_gain, void* ws,
                                 size_t ws_bytes, coli_stream_t stream) {
    size_t need;
    int rc = norm_ok("block_norm_backward", desc, T);
    if (rc) return rc;
    if ((rc = coli_moe_block_norm_backward_workspace_size(desc, T, &need))) return rc;
    // zero tokens: empty tensors have no address, so only what the sums over tokens go to is looked at
    if (T > 0) {
        if (!dx || (!dx_out && !dn) || (dn && (!x_out || !rstd_pre)) || (o != nullptr) != (d_o != nullptr) ||
            (o && desc->post_norm && !rstd_post))
            return fail(COLI_E_INVAL, "block_norm_backward: NULL pointer");
        if (o && (desc->gate_kind != COLI_GATE_NONE) != (gate != nullptr))
            return fail(COLI_E_INVAL, "block_norm_backward: gate and gate_kind disagree");
    }
    if ((dgate && ((T > 0 && !o) || desc->gate_kind == COLI_GATE_NONE)) ||
        (dpost_gain && ((T > 0 && !o) || !desc->post_norm)) || (dpre_gain && T > 0 && !dn))
        return fail(COLI_E_INVAL, "block_norm_backward: gradient of an input that this call does not have");
    const int xs = type_size(desc->xt), bs = type_size(desc->bt);
    if ((rc = elements_ok("block_norm_backward", {{x_out, xs}, {dx_out, xs}, {dx, xs}, {o, bs}, {dn, bs}, {d_o, bs},
                                                  {desc->post_gain, 4}, {desc->pre_gain, 4}, {gate, 4}, {rstd_post, 4},
                                                  {rstd_pre, 4}, {dpost_gain, 4}, {dgate, 4}, {dpre_gain, 4}})))
        return rc;
    // sums over tokens: partial rows in the workspace, then the second kernel
    const bool channel = dgate && desc->gate_kind == COLI_GATE_CHANNEL;
    NormSums keep;
    keep.n = 0;
    keep.at[0] = dpost_gain ? keep.n++ : -1;
    keep.at[1] = channel ? keep.n++ : -1;
    keep.at[2] = dpre_gain ? keep.n++ : -1;
    if (keep.n && need && (!ws || ws_bytes < need || !aligned(ws, 16)))
        return fail(COLI_E_WORKSPACE, "block_norm_backward: workspace of %zu bytes, %zu needed", ws ? ws_bytes : 0,
                    need);
    float* partial = static_cast<float*>(ws);
    int grid = 0;
    if (T > 0) {
        const int W = chunk_of<8>(desc->H, {{x_out, xs}, {dx_out, xs}, {dx, xs}, {o, bs}, {dn, bs}, {d_o, bs},
                                            {desc->post_gain, 4}, {desc->pre_gain, 4}, {gate, 4}, {dgate, 4}});
        const NormArgs a = norm_args(*desc, gate, T);
        const int ctas = norm_ring_ctas(*desc, T);
        const NormRing ring = norm_ring(*desc, ctas, W == 8, dn != nullptr, dx_out != nullptr, o != nullptr, dn != nullptr);
        grid = norm_backward_grid(T, ring.stages > 0 ? ctas : norm_plain_ctas(*desc, T));
        if (g_norm_withhold >= 0 && (ring.stages == 0 || desc->xt != COLI_F32 || desc->bt != COLI_BF16 || desc->H > 8 * 768))
            return fail(COLI_E_UNSUPPORTED, "block_norm_backward: the wait test takes the ring's rows of up to 6144 f32 with bf16 blocks");
        if (ring.stages > 0) {
            NormShape s;
            s.W = 8;
            s.N = desc->H / 8 <= 768 ? 1 : 2;  // more warps hide more of each other's waits
            s.threads = ((desc->H / 8 + s.N - 1) / s.N + 31) / 32 * 32;
            rc = norm_ring_dispatch(*desc, s, a, keep, ring, x_out, o, rstd_post, rstd_pre, dx_out, dn, dx, d_o, dgate,
                                    partial, grid, S(stream));
        } else {
            rc = norm_dispatch<NormBackwardPlain>(*desc, norm_shape(desc->H, T, W, true), a, keep, ring, x_out, o,
                                                  rstd_post, rstd_pre, dx_out, dn, dx, d_o, dgate, partial, grid,
                                                  S(stream));
        }
        if (rc) return rc;
    }
    if (!keep.n) return COLI_OK;
    // few partial rows: small CTAs, many of them at once; many (short rows): more runs
    const int rows = grid / norm_backward_cluster(grid);
    const auto reduce = rows <= 128 ? norm_reduce_kernel<8> : norm_reduce_kernel<32>;
    return launch_pdl(reduce, dim3((desc->H + 31) / 32, kNormSums), 32 * (rows <= 128 ? 8 : 32), 0, S(stream),
                      "block norm sums", (const float*)partial, rows, (int)desc->H, keep, dpost_gain,
                      channel ? dgate : nullptr, dpre_gain);
}

int coli_moe_block_norm_set_wait_test(int32_t withhold) {
    g_norm_withhold = withhold < 0 ? -1 : withhold;
    return COLI_OK;
}

}  // extern "C"
