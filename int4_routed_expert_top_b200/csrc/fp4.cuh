// fp4.cuh - 4-bit floating point in blocks with a shared scale: the quantiser of
// rows, and the grouped product of quantised rows with quantised weights on
// the block-scaled tensor cores.  Formats and layouts: include/coli_moe.h.
//
// Product.  D[r, n] = sum_k W[r, k] X[n, k]: weight rows are the MMA's M (128
// of one expert's), the rows of that expert its N (up to NT).  tcgen05.mma with
// block scales multiplies 64 columns of E2M1 at a time and applies the two
// blocks' scales itself (kind::mxf4, 32-column blocks, E8M0; kind::mxf4nvf4,
// 16-column blocks, E4M3), f32 accumulators in TMEM.  At few rows per expert
// the work is bound by the weights' bytes from HBM, at many by the tensor
// pipe and the shared memory that feeds it.
//
// One unit of work is a stage: 256 columns (128 bytes) of one tile.  A tile is
// (expert, 128 weight rows, NT of its rows), in the order (expert, weight rows,
// rows).  As many whole waves of tiles as there are go to the CTAs in turn, so
// that the SMs work on neighbouring tiles, whose weights and rows then come from
// L2 (runs of tiles per CTA read 3.6 GB from HBM where this order reads
// WAVE_READ, at 4096 tokens x 8 picks on 32 experts of 4096 x 6144).  The tiles
// that are left over, all of them at few rows, are cut by units into equal runs, one
// per CTA, so that every SM streams the same number of bytes.  A tile that a
// run's border cuts leaves f32 partial sums in the workspace: every
// CTA that does not begin the tile stores its piece and raises a flag, and the
// one that begins it, whose piece is the last of its run, adds them in the
// order of their columns.  No atomics, the same bits at every run; the others
// take these pieces first, so the wait is short, and it is never for a CTA with
// a lower index, so CTAs that are scheduled late cannot stop the earlier ones.
//
// CTA roles: warp 0 copies (codes by 2-D TMA with the 128-byte swizzle, the
// weights' scales by bulk copy), warps 2-3 bring the rows' scales (rows of an
// expert start anywhere, a scale tile only at multiples of 128, so those are
// gathered by plain loads into a tile in shared memory), warp 1 copies scales
// to TMEM and issues the products, warps 4-7 store.  Accumulators are
// double-buffered, so a tile's stores overlap the next one's products.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "tc.cuh"
#include "vec.cuh"

namespace coli {

// ---------------------------------------------------------------------------
// quantiser
// ---------------------------------------------------------------------------
struct Fp4QuantArgs {
    int64_t n_src, rows;
    int K, words;            // words: 4-block scale words per row
    int swiglu;
    const int32_t* src;
    const int32_t* count;
    const float* gscale;
    uint8_t* codes;
    uint32_t* scales;
};

// word index of the scales of (row r, blocks 4w .. 4w + 3)
__device__ __forceinline__ int64_t scale_word(int64_t r, int w, int words) {
    return ((r >> 7) * words + w) * 128 + (r & 31) * 4 + ((r >> 5) & 3);
}

// A lane holds 8 columns of a row, a warp 256 at a time: 16 bytes of bf16 (32
// of f32) per load, a block's maximum by one or two shuffles.  A CTA's 8 warps
// share out `rows_per` rows, 8 / rows_per warps each; one chunk per warp, since
// many small CTAs hide the loads better than a warp's loop over its row does.
// Bound by HBM (x once, codes, scales and values once).
template <typename T, bool NV>
__device__ __forceinline__ void fp4_quantize_chunk(const Fp4QuantArgs& a, const T* __restrict__ x,
                                                   T* __restrict__ values, int64_t r, int64_t from, int c,
                                                   float g) {
    const int lane = threadIdx.x & 31;
    const bool in = c < a.K;
    F<8> f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = 0.0f;
    if (in && from >= 0 && from < a.n_src) {
        if (a.swiglu) {
            const T* p = x + from * 2 * a.K + c;
            f = ldf<T, 8>(p);
            const F<8> u = ldf<T, 8>(p + a.K);
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = silu_f(f.v[i]) * u.v[i];
        } else {
            f = ldf<T, 8>(x + from * a.K + c);
        }
    }
    const float (&v)[8] = f.v;
    // the largest magnitude as bits: infinities and NaN come out on top
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const bool bad = m >= 0x7f800000u;
    uint32_t byte;
    float d, r_d;  // what a code of 1 stands for, and its reciprocal
    if (NV) {
        const float t = __fdiv_rn(__uint_as_float(m), __fmul_rn(6.0f, g));
        byte = __nv_cvt_float_to_fp8(fminf(t, 448.0f), __NV_SATFINITE, __NV_E4M3);
        d = __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3))), g);
        r_d = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        if (bad) byte = 0x7f;
    } else {
        const int b = max((int)(m >> 23) - 2, 0);
        byte = bad ? 255u : (uint32_t)b;
        d = __uint_as_float(b ? (uint32_t)b << 23 : 0x00400000u);
        r_d = __uint_as_float((uint32_t)(254 - b) << 23);
    }
    uint32_t code = 0;
    if (!bad && (!NV || d > 0.0f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code |= (uint32_t)__nv_cvt_float2_to_fp4x2(
                        make_float2(__fmul_rn(v[2 * i], r_d), __fmul_rn(v[2 * i + 1], r_d)), __NV_E2M1,
                        cudaRoundNearest) << (8 * i);
    }
    if (!in) byte = 0;
    // four blocks' bytes make a word: a block is 2 (NV) or 4 lanes
    constexpr int per = NV ? 2 : 4;
    const int first = lane & ~(4 * per - 1);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, byte, first + i * per) << (8 * i);
    if (!in) {
        if (lane == first && c / (32 * per) < a.words) a.scales[scale_word(r, c / (32 * per), a.words)] = word;
        return;
    }
    if (lane == first) a.scales[scale_word(r, c / (32 * per), a.words)] = word;
    *reinterpret_cast<uint32_t*>(a.codes + (r * a.K + c) / 2) = code;
    if (values) {
        F<8> q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(code >> (8 * i)), __NV_E2M1));
            q.v[2 * i] = __fmul_rn(__low2float(h), d);
            q.v[2 * i + 1] = __fmul_rn(__high2float(h), d);
            if (bad) q.v[2 * i] = q.v[2 * i + 1] = __uint_as_float(0x7fc00000u);
        }
        stf<T, 8>(values + r * a.K + c, q);
    }
}

template <typename T, bool NV>
__global__ void __launch_bounds__(256)
fp4_quantize_kernel(Fp4QuantArgs a, int rows_per, const T* __restrict__ x, T* __restrict__ values) {
    const int warps = 8 / rows_per, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * rows_per + warp / warps;
    const int c0 = ((int)blockIdx.y * warps + (warp & (warps - 1))) * 256;
    pdl_trigger();
    pdl_wait();
    if (r >= a.rows || c0 >= a.K || (a.count && r >= *a.count)) return;
    fp4_quantize_chunk<T, NV>(a, x, values, r, a.src ? a.src[r] : r, c0 + lane * 8,
                              NV && a.gscale ? *a.gscale : 1.0f);
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
constexpr int kFpThreads = 256;
constexpr int kFpMaxE = 1024;
constexpr int kFpMinUnits = 2;     // stages per CTA at least, before fewer CTAs take part
constexpr int kFpMaxGrid = 160;    // B200 has 148 SMs; the workspace is sized for this many
// the workspace: error flags, a flag per CTA and store warp, then partial sums
constexpr int kFpFlagBytes = 256;
constexpr int kFpHeadBytes = kFpFlagBytes + kFpMaxGrid * 4 * 8;
// a raised flag: a value that unset memory does not hold (0 after every call)
constexpr uint64_t kFpRaised = 0x9d3ac1f5e8276b41ull;

template <int NT, bool NV>
struct FpShape {
    static constexpr int box = NT < 64 ? NT : 64;            // rows per TMA box of X
    static constexpr int atoms = NV ? 4 : 2;                 // 512-byte scale tiles per 256 columns
    static constexpr int nb = (NT + 127) / 128;              // of the rows, per atom
    static constexpr int a_bytes = 128 * 128;
    static constexpr int b_bytes = NT * 128;
    static constexpr int sfa_bytes = atoms * 512;
    static constexpr int sfb_bytes = atoms * nb * 512;
    static constexpr int stage = (a_bytes + b_bytes + sfa_bytes + sfb_bytes + 1023) / 1024 * 1024;
    static constexpr int stages = 196608 / stage;
    static constexpr int smem = stages * stage + 1024;
    static constexpr int sf_cols = atoms * 4 * (1 + nb);     // TMEM columns of one stage's scales
    static constexpr int sf0 = 2 * NT;                       // after two accumulators
    static constexpr int cols_used = sf0 + 2 * sf_cols;
    static constexpr int cols = cols_used <= 128 ? 128 : cols_used <= 256 ? 256 : 512;
    static_assert(NT % box == 0 && NT % 16 == 0 && cols_used <= 512, "TMEM holds 512 columns");
};

struct FpArgs {
    const uint32_t* xs;      // scale words of the rows
    const uint8_t* ws;       // scale tiles of the weights
    int64_t P;
    int K, E, R, KS;         // KS: stages per tile
    int xwords, wwords;      // scale words per row
    const int32_t* offsets;
    const float* alpha;
    uint64_t* flags;
    float* partial;
    int32_t* err;
};

// Where every expert's tiles start, in shared memory.
struct FpPlan {
    int32_t begin[kFpMaxE + 1];
    int64_t tile0[kFpMaxE + 1];
    int64_t warp_sum[8];
};

// Each thread takes four experts; offsets are clamped so that no value of them
// leads out of the buffers.
template <int NT>
__device__ __forceinline__ void fp_plan(const FpArgs& a, FpPlan& p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int RT = (a.R + 127) / 128;
    if (!a.offsets) {
        if (threadIdx.x == 0) {
            p.begin[0] = 0;
            p.begin[1] = (int)a.P;
            p.tile0[0] = 0;
            p.tile0[1] = (a.P + NT - 1) / NT * RT;
        }
        __syncthreads();
        return;
    }
    int64_t n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * threadIdx.x + i;
        n[i] = 0;
        if (e < a.E) {
            const int64_t b = min(max((int64_t)a.offsets[e], (int64_t)0), a.P);
            const int64_t end = min(max((int64_t)a.offsets[e + 1], b), a.P);
            p.begin[e] = (int)b;
            if (e == a.E - 1) p.begin[a.E] = (int)end;
            n[i] = (end - b + NT - 1) / NT * RT;
        }
        sum += n[i];
    }
    int64_t v = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) p.warp_sum[warp] = v;
    __syncthreads();
    int64_t at = v - sum;
    for (int i = 0; i < warp; ++i) at += p.warp_sum[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * threadIdx.x + i;
        if (e < a.E) p.tile0[e] = at;
        at += n[i];
        if (e == a.E - 1) p.tile0[a.E] = at;
    }
    __syncthreads();
}

// The share of every CTA: tiles c, c + G, .. of the first waves * G, and units
// [lo(c), lo(c + 1)) of the tiles from tile0 on.
struct FpRun {
    int64_t G, waves, tile0, U;
    __device__ __forceinline__ FpRun(const FpArgs& a, const FpPlan& p, int grid) {
        const int64_t tiles = p.tile0[a.E];
        G = min((int64_t)grid, max((int64_t)1, tiles * a.KS / kFpMinUnits));
        waves = tiles / G;
        tile0 = waves * G;
        U = (tiles - tile0) * a.KS;
    }
    __device__ __forceinline__ int64_t lo(int64_t c) const { return c >= G ? U : U * c / G; }
};

struct FpTile {
    int e, rt, n;       // expert, weight-row tile, rows in the tile
    int64_t p0;         // first row
};

template <int NT>
__device__ __forceinline__ FpTile fp_tile(const FpPlan& p, int E, int64_t tile) {
    int lo = 0, hi = E;  // the last expert whose first tile is not after this one
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (p.tile0[m] <= tile) lo = m; else hi = m;
    }
    FpTile t;
    t.e = lo;
    const int rows = p.begin[lo + 1] - p.begin[lo];
    const int nj = (rows + NT - 1) / NT;
    const int i = (int)(tile - p.tile0[lo]);
    t.rt = i / nj;
    const int j = i - t.rt * nj;
    t.p0 = p.begin[lo] + (int64_t)j * NT;
    t.n = min(NT, rows - j * NT);
    return t;
}

// A CTA's pieces in order: (tile, stages [k0, k1) of it), the cut tiles first.
struct FpPieces {
    int64_t u, hi, tile0, left, at, step;
    int KS;
    int64_t tile;
    int k0, k1;
    __device__ __forceinline__ FpPieces(const FpArgs& a, const FpRun& r, int64_t c) {
        u = r.lo(c);
        hi = r.lo(c + 1);
        tile0 = r.tile0;
        left = c < r.G ? r.waves : 0;
        at = c;
        step = r.G;
        KS = a.KS;
        tile = 0;
        k0 = k1 = 0;
    }
    __device__ __forceinline__ int64_t stages() const { return hi - u + left * KS; }  // before the first next()
    __device__ __forceinline__ bool next() {
        if (u < hi) {
            tile = u / KS;
            k0 = (int)(u - tile * KS);
            k1 = (int)min((int64_t)KS, k0 + (hi - u));
            u += k1 - k0;
            tile += tile0;
            return true;
        }
        if (left == 0) return false;
        --left;
        tile = at;
        at += step;
        k0 = 0;
        k1 = KS;
        return true;
    }
};

// shared-memory descriptor of a 32-row, 16-byte-wide scale tile (no swizzle,
// 8-row groups 128 bytes apart)
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// 32 rows x 16 bytes of shared memory to 32 lanes x 4 columns of TMEM, repeated
// in the four lane quarters
__device__ __forceinline__ void tc_copy_scales(uint32_t dst, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(dst), "l"(desc) : "memory");
}

// instruction descriptor of a block-scaled product of E2M1 operands, both
// K-major, M = 128: types 1 (E2M1), N / 8, scale type (1 E8M0, 0 E4M3), M / 128;
// the bytes of a scale word that apply are added per product
template <bool NV>
__device__ __forceinline__ constexpr uint32_t idesc_fp4(int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((NV ? 0u : 1u) << 23) | (1u << 27);
}

template <bool NV>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if (NV)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n}"
            ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}"
            ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}

// Warp-wide wait for a flag of another CTA's store warp, a second at most
__device__ __forceinline__ bool fp_wait_flag(const uint64_t* flag, int32_t* err) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0) {
        uint64_t v = 0;
        for (int i = 0; i < (1 << 21) && v != kFpRaised; ++i)
            asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(flag) : "memory");
        ok = v == kFpRaised;
        if (!ok) atomicOr(err, kErrWaitTimeout);
    }
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

template <int NT, bool NV, typename YT>
__global__ void __launch_bounds__(kFpThreads, 1)
fp4_product_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   FpArgs a, YT* y) {
    using C = FpShape<NT, NV>;
    extern __shared__ uint8_t fp_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(fp_raw) + 1023) & ~uintptr_t(1023));
    __shared__ FpPlan plan;
    __shared__ __align__(8) uint64_t full[C::stages], empty[C::stages], accfull[2], accempty[2];
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) tmem_alloc(&tmem_slot, C::cols);
    if (threadIdx.x == 32) {
        for (int s = 0; s < C::stages; ++s) {
            mbar_init(&full[s], 3);   // the copies' announcement and two scale warps
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accfull[b], 1);
            mbar_init(&accempty[b], 4);
        }
        fence_mbar_init();
    }
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x == 0 && threadIdx.x == 64) *a.err = 0;
    fp_plan<NT>(a, plan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const FpRun run(a, plan, gridDim.x);
    FpPieces q(a, run, blockIdx.x);
    bool ok = true;  // cleared by a wait that gave up: then no further waits

    if (warp == 0) {
        // ---------------- copies (whole warp, elected lane issues) ----------------
        int cnt = 0;
        while (q.next()) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            const int64_t wrow = (int64_t)t.e * a.R + (int64_t)t.rt * 128;
            const int boxes = (t.n + C::box - 1) / C::box;
            const uint8_t* sfa = a.ws + (wrow >> 7) * a.wwords * 512;
            for (int k = q.k0; k < q.k1; ++k, ++cnt) {
                const int s = cnt % C::stages;
                if (cnt >= C::stages && ok && !mbar_wait_warp(&empty[s], ((cnt / C::stages) - 1) & 1, a.err)) ok = false;
                uint8_t* st = smem + s * C::stage;
                const int na = min(C::atoms, a.wwords - k * C::atoms);
                mbar_expect_tx_elect(&full[s], (uint32_t)(C::a_bytes + boxes * C::box * 128 + na * 512));
                tma_load_2d_elect(st, &wmap, k * 128, (int)wrow, &full[s]);
                for (int b = 0; b < boxes; ++b)
                    tma_load_2d_elect(st + C::a_bytes + b * C::box * 128, &xmap, k * 128,
                                      (int)t.p0 + b * C::box, &full[s]);
                bulk_g2s_elect(st + C::a_bytes + C::b_bytes, sfa + (int64_t)k * C::atoms * 512, na * 512, &full[s]);
            }
        }
        // the last copies have landed before the CTA may end
        for (int i = max(0, cnt - C::stages); i < cnt; ++i)
            mbar_wait_warp_sleep(&full[i % C::stages], (i / C::stages) & 1, a.err);
    } else if (warp == 1) {
        // ---------------- products ----------------
        const uint32_t one = elect_one();
        const uint32_t sbase = smem_u32(smem);
        int cnt = 0, piece = 0;
        for (; q.next(); ++piece) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            const uint32_t idesc = idesc_fp4<NV>((t.n + 15) / 16 * 16);
            const int buf = piece & 1;
            if (piece >= 2 && ok && !mbar_wait_warp(&accempty[buf], ((piece >> 1) - 1) & 1, a.err)) ok = false;
            tc_fence_after();
            const uint32_t d = tmem + NT * buf;
            const int nbk = (t.n + 127) / 128;
            for (int k = q.k0; k < q.k1; ++k, ++cnt) {
                const int s = cnt % C::stages;
                if (ok && !mbar_wait_warp(&full[s], (cnt / C::stages) & 1, a.err)) ok = false;
                tc_fence_after();
                if (one) {
                    const uint32_t st = sbase + s * C::stage;
                    const uint32_t sf = tmem + C::sf0 + (cnt & 1) * C::sf_cols;
                    const uint32_t sfa = st + C::a_bytes + C::b_bytes, sfb = sfa + C::sfa_bytes;
                    const int cols = min(256, a.K - 256 * k);
                    const int na = (cols + 256 / C::atoms - 1) / (256 / C::atoms);
#pragma unroll
                    for (int i = 0; i < C::atoms; ++i) {
                        if (i >= na) break;
                        tc_copy_scales(sf + 4 * i, smem_desc_scales(sfa + 512 * i));
#pragma unroll
                        for (int b = 0; b < C::nb; ++b)
                            if (b < nbk)
                                tc_copy_scales(sf + 4 * C::atoms + 4 * (C::nb * i + b),
                                               smem_desc_scales(sfb + 512 * (C::nb * i + b)));
                    }
                    const uint64_t ad = smem_desc_sw128(smem + s * C::stage);
                    const uint64_t bd = smem_desc_sw128(smem + s * C::stage + C::a_bytes);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (64 * j >= cols) break;
                        const int at = NV ? j : j >> 1;          // scale tile
                        const uint32_t id = NV ? 0u : 2u * (j & 1);  // first byte of its words
                        tc_mma_fp4<NV>(d, ad + 2 * j, bd + 2 * j, idesc | id << 29 | id << 4, sf + 4 * at,
                                       sf + 4 * C::atoms + 4 * C::nb * at, (k > q.k0 || j > 0) ? 1u : 0u);
                    }
                    tc_commit(&empty[s]);
                }
                __syncwarp();
            }
            if (one) tc_commit(&accfull[buf]);
            __syncwarp();
        }
    } else if (warp < 4) {
        // ---------------- scales of the rows: atoms of one parity ----------------
        // The loads of a stage are issued `ahead` stages before it is stored.
        constexpr int mine = C::atoms / 2;
        constexpr int words = NT / 32;        // per lane and atom
        constexpr int ahead = NT > 64 ? 4 : 8;
        const int par = warp - 2;
        uint32_t w[ahead][mine][words];
        FpTile t;
        const int64_t total = q.stages();
        const auto load = [&](uint32_t (&to)[mine][words]) {  // the next stage's words, if there is one
            if (q.k0 == q.k1) {
                if (!q.next()) return;
                t = fp_tile<NT>(plan, a.E, q.tile);
            }
#pragma unroll
            for (int i = 0; i < mine; ++i) {
                const int ch = q.k0 * C::atoms + 2 * i + par;
#pragma unroll
                for (int j = 0; j < words; ++j) {
                    const int64_t r = t.p0 + 32 * j + lane;
                    to[i][j] = 0;
                    if (ch < a.xwords && 32 * j < t.n && r < a.P) to[i][j] = __ldg(a.xs + scale_word(r, ch, a.xwords));
                }
            }
            ++q.k0;
        };
#pragma unroll
        for (int d = 0; d < ahead; ++d) load(w[d]);
        for (int64_t base = 0; base < total; base += ahead) {
#pragma unroll
            for (int d = 0; d < ahead; ++d) {
                const int cnt = (int)base + d;
                if (cnt >= total) break;
                const int s = cnt % C::stages;
                if (cnt >= C::stages && ok && !mbar_wait_warp(&empty[s], ((cnt / C::stages) - 1) & 1, a.err)) ok = false;
                uint8_t* sfb = smem + s * C::stage + C::a_bytes + C::b_bytes + C::sfa_bytes;
#pragma unroll
                for (int i = 0; i < mine; ++i)
#pragma unroll
                    for (int j = 0; j < words; ++j)
                        *reinterpret_cast<uint32_t*>(sfb + 512 * (C::nb * (2 * i + par) + j / 4) + 16 * lane + 4 * (j & 3)) =
                            w[d][i][j];
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                load(w[d]);
            }
        }
    } else {
        // ---------------- stores: weight rows 32 quarter + lane of the tile ----------------
        const int quarter = warp & 3;
        for (int piece = 0; q.next(); ++piece) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            const int buf = piece & 1;
            const int row = t.rt * 128 + 32 * quarter + lane;
            const bool begins = q.k0 == 0;
            const float al = begins && a.alpha ? a.alpha[t.e] : 1.0f;
            float* part = a.partial + 32 * quarter + lane;
            // the CTAs after this one with pieces of the tile: up to the first whose run
            // starts at its end or later
            int64_t last = blockIdx.x + 1;
            if (begins && q.k1 < a.KS)
                while (run.lo(last) < (q.tile + 1 - run.tile0) * a.KS) ++last;
            if (ok && !mbar_wait_warp(&accfull[buf], (piece >> 1) & 1, a.err)) ok = false;
            tc_fence_after();
            for (int64_t c = blockIdx.x + 1; c < last; ++c)
                if (ok && !fp_wait_flag(a.flags + 4 * c + quarter, a.err)) ok = false;
            const uint32_t d = tmem + ((uint32_t)(32 * quarter) << 16) + NT * buf;
            for (int c0 = 0; c0 < t.n; c0 += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(d + c0, v);
                tmem_wait_ld();
                if (!begins) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < t.n) part[(int64_t)blockIdx.x * (128 * NT) + (c0 + i) * 128] = __uint_as_float(v[i]);
                    continue;
                }
                for (int64_t c = blockIdx.x + 1; c < last; ++c)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < t.n)
                            v[i] = __float_as_uint(__uint_as_float(v[i]) + __ldcg(part + c * (128 * NT) + (c0 + i) * 128));
                if (row < a.R) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < t.n)
                            y[(t.p0 + c0 + i) * a.R + row] = from_f32<YT>(__uint_as_float(v[i]) * al);
                }
            }
            if (!begins) {
                __syncwarp();
                if (lane == 0) {
                    __threadfence();
                    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.flags + 4 * blockIdx.x + quarter), "l"(kFpRaised)
                                 : "memory");
                }
            } else {
                __syncwarp();
                for (int64_t c = blockIdx.x + 1; c < last; ++c)
                    if (lane == 0) a.flags[4 * c + quarter] = 0;  // read once: down again for the next call
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&accempty[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, C::cols);
}

}  // namespace coli
