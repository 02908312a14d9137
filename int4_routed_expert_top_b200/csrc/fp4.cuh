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
// 0.55 GB, at 4096 tokens x 8 picks on 32 experts of 4096 x 6144).  The tiles
// that are left over, all of them at few rows, are cut by units into equal runs, one
// per CTA, so that every SM streams the same number of bytes.  A tile that a
// run's border cuts leaves f32 partial sums in the workspace: every
// CTA that does not begin the tile stores its piece and raises a flag, and the
// one that begins it, whose piece is the last of its run, adds them in the
// order of their columns.  No atomics, the same bits at every run; the others
// take these pieces first, so the wait is short, and it is never for a CTA with
// a lower index, so CTAs that are scheduled late cannot stop the earlier ones.
//
// Every wait is tried by all lanes of its warp: one lane's answer passed on by a
// shuffle or a vote costs the issuing warps some 300 cycles a stage (the tile
// loop took 1.6 to 2.5 times as long).
//
// At few rows per expert a CTA works by itself on 128 weight rows and up to 32 of
// the expert's.  At many, two CTAs of a cluster share a tile of 256 weight rows and
// up to 224 rows (tcgen05 cta_group::2): each holds 128 of the weight rows and half
// of the others in its shared memory and the accumulators of its weight rows, and
// CTA 0 issues the products for both.  A stage is then 33 KB per SM instead of the
// 43 KB of a 128 x 192 tile for 1.17 times the work.
//
// Measured (B200, calls one after the other in a graph): 8 rows, one to an expert, of 4096 x
// 6144: 21.5 us, 5.0 TB/s of weights (launch, schedule and first loads are some 6 us of it);
// 512 rows on 64 experts of 6144 x 2048: 74 us, 6.1 TB/s, 0.94 of a copy's rate; 32768 rows on
// 32 experts of 4096 x 6144 with skewed counts: 346 to 355 us from run to run, 4.7 PFLOP/s, the
// tensor pipe 74% active (NVFP4: 376 us); one matrix of 18944 x 6144 and 14336 rows:
// 5.5 PFLOP/s: under sustained load the chip's power limit sets the clock (1.4 GHz).
//
// CTA roles: warp 0 copies (codes by 2-D TMA with the 128-byte swizzle, the
// weights' scales by bulk copy), warp 1 copies scales to TMEM and issues the
// products, warps 4-7 (of a pair also 8-11) store.  Rows of an expert start
// anywhere, a scale tile only at multiples of 128, so the rows' scales are gathered
// word by word: in a CTA by itself by four warps into a tile in shared memory, for pairs
// by a kernel of its own before the product, whose tiles then come by TMA.  Accumulators
// are double-buffered, so a tile's stores overlap the next one's products.
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
    uint32_t n_src;          // of the source, 2^31 at most
    int rows, K, words;      // words: 4-block scale words per row
    const int32_t* src;
    const int32_t* count;
    const float* gscale;
    uint8_t* codes;
    uint32_t* scales;
};

// word index of the scales of (row r, blocks 4w .. 4w + 3)
__device__ __forceinline__ int64_t scale_word(int64_t r, int w, int words) {
    return ((int64_t)(int)(r >> 7) * words + w) * 128 + ((int)r & 31) * 4 + ((int)(r >> 5) & 3);
}

// eight f32 to E2M1 (nearest, ties to even, saturating), the first in the lowest
// nibble
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
    uint32_t r;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// the largest magnitude of three, NaN if one is
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A lane holds 16 columns of a row (two or four loads of 16 or 32 bytes), a warp
// 512: a block is one lane (NVFP4) or two, so its maximum takes at most one
// shuffle.  Every warp of a CTA has one chunk of one of its rows: that hides the
// loads better than a warp's loop over its row does.  Rows of 256 columns or fewer
// share a warp (1 << lg lanes to a row: 8, 16 or 32; a scale word is 4 or 8).  Bound by HBM (x
// once, codes, scales and values once) where values are written: 32768 x 6144 f32
// 251 us, 6.8 TB/s; bf16 without them 84 us, 6.1 TB/s (107 us with rows and chunks
// found by divisions and 64-bit indexes).
constexpr int kQuantCols = 512;
constexpr int kQuantWarps = 16;  // of a CTA, at most

template <typename T, bool NV, bool GLU>
__global__ void __launch_bounds__(32 * kQuantWarps)
fp4_quantize_kernel(Fp4QuantArgs a, int lg, const T* __restrict__ x, T* __restrict__ values) {
    const int lane = threadIdx.x & 31;
    // threadIdx.y: a row (or 32 >> lg rows of 1 << lg lanes); the warps along x: its chunks
    const uint32_t r0 = (blockIdx.x * blockDim.y + threadIdx.y) << (5 - lg), r = r0 + (lane >> lg);
    const int c0 = (int)(blockIdx.y * blockDim.x + (threadIdx.x & ~31u)) * (kQuantCols / 32);
    const int c = c0 + (lane & ((1 << lg) - 1)) * 16;
    pdl_trigger();
    pdl_wait();
    const uint32_t rows = a.count ? (uint32_t)max(min(a.rows, *a.count), 0) : (uint32_t)a.rows;
    if (c0 >= a.K || r0 >= rows) return;               // the whole warp
    const bool live = r < rows, in = live && c < a.K;  // K is a multiple of 32: all 16 columns or none
    const uint32_t from = !live ? 0 : a.src ? (uint32_t)a.src[r] : r;
    const float g = NV && a.gscale ? *a.gscale : 1.0f;
    const bool read = in && from < a.n_src;            // a negative entry is 2^31 or more
    const T* p = x + (int64_t)((uint64_t)from * (uint32_t)(GLU ? 2 * a.K : a.K)) + c;
    Vec<T, 8> raw[GLU ? 4 : 2];
#pragma unroll
    for (int i = 0; i < (GLU ? 4 : 2); ++i) {
        if (read) raw[i] = ldv<T, 8>(p + (i & 1) * 8 + (i >> 1) * a.K);
        else
#pragma unroll
            for (int j = 0; j < (int)(sizeof(raw[i].u) / 4); ++j) raw[i].u[j] = 0;
    }
    float v[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        F<8> f = widen<T, 8>(raw[h]);
        if (GLU) {
            const F<8> u = widen<T, 8>(raw[GLU ? 2 + h : 0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) f.v[i] = silu_f(f.v[i]) * u.v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = f.v[i];
    }
    // the largest magnitude; infinities and NaN come out on top, as bits too
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max3_abs(top, v[i], v[i + 1]);
    uint32_t m = __float_as_uint(top);
    if (!NV) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
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
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(v[i], r_d);
    uint32_t code[2] = {e2m1x8(v), e2m1x8(v + 8)};
    if (bad || (NV && !(d > 0.0f))) code[0] = code[1] = 0;
    // four blocks' bytes make a word: a block is 1 (NV) or 2 lanes
    constexpr int per = NV ? 1 : 2;
    if (!in) byte = 0;
    uint32_t word = byte << (8 * (lane / per & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, per);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * per);
    const int at = c / (64 * per);
    if (live && (lane & (4 * per - 1)) == 0 && at < a.words) a.scales[scale_word(r, at, a.words)] = word;
    if (!in) return;
    const int64_t at_c = (int64_t)((uint64_t)r * (uint32_t)a.K) + c;
    *reinterpret_cast<uint2*>(a.codes + at_c / 2) = make_uint2(code[0], code[1]);
    if (values) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            F<8> q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 two = __half2(
                    __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(code[h] >> (8 * i)), __NV_E2M1));
                q.v[2 * i] = __fmul_rn(__low2float(two), d);
                q.v[2 * i + 1] = __fmul_rn(__high2float(two), d);
                if (bad) q.v[2 * i] = q.v[2 * i + 1] = __uint_as_float(0x7fc00000u);
            }
            stf<T, 8>(values + at_c + 8 * h, q);
        }
    }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
// warps 0 copies, 1 products, 4-7 stores; by itself 2-3 and 8-9 scales of the rows, in a pair
// 8-11 stores as well
constexpr int kFpScaleWarps = 4;
constexpr int kFpStoreWarps = 8;   // at most
constexpr int kFpMaxWarps = 12;
constexpr int kFpMaxE = 1024;
// Stages that a cut tile's pieces have at least: shorter ones save less than joining
// them takes (8 rows, 20 experts of 1024 x 2048: 6.7 us with 8, 8.8 with 4; 512 rows, 64
// experts of 6144 x 2048: 74 and 80 us; pairs, 400 rows of 1000 x 2048: 8.0 and 15.2).
constexpr int kFpMinUnits = 8;
constexpr int kFpMaxGrid = 160;    // B200 has 148 SMs; the workspace is sized for this many
// the workspace: error flags, a flag per CTA and store warp, then partial sums
constexpr int kFpFlagBytes = 256;
constexpr int kFpHeadBytes = kFpFlagBytes + kFpMaxGrid * kFpStoreWarps * 8;
// a raised flag: a value that unset memory does not hold (0 after every call); and one
// whose piece is not there, which is also what the workspace's first word becomes when
// a wait gives up, and stays
constexpr uint64_t kFpRaised = 0x9d3ac1f5e8276b41ull, kFpBroken = 0x62c53e0a17d894beull;
// tries of a wait for flags (some ten seconds); of every wait under the wait test
constexpr uint32_t kFpFlagTries = 1u << 25, kFpTestTries = 4096;

// NT: rows of a tile at most; PAIR: two CTAs to a tile, M = 256 weight rows
template <int NT, bool NV, bool PAIR>
struct FpShape {
    static constexpr int M = PAIR ? 256 : 128;
    static constexpr int ctas = PAIR ? 2 : 1;
    static constexpr int rows = NT / ctas;                   // of X in a CTA's shared memory
    static constexpr int box = PAIR ? rows / 2 : rows;       // rows per TMA box of X
    static constexpr int store_warps = PAIR ? kFpStoreWarps : 4;
    static constexpr int groups = store_warps / 4;           // warps to a quarter of the lanes
    static constexpr int threads = 32 * (PAIR ? 12 : 10);
    // the launch bound: 128 registers a thread of a pair, so that the next product's gather of
    // scales (14336 of them) fits beside its CTAs (400 rows of 10240 x 2048 in one run: 14.7 us, 15.4 with 131)
    static constexpr int bound = PAIR ? 512 : threads;
    static constexpr int step = 16 * ctas;                   // N is a multiple of it
    static constexpr int atoms = NV ? 4 : 2;                 // 512-byte scale tiles per 256 columns
    static constexpr int nb = (NT + 127) / 128;              // of the rows, per atom
    static constexpr int a_bytes = 128 * 128;
    static constexpr int b_bytes = rows * 128;
    static constexpr int sfa_bytes = atoms * 512;
    static constexpr int sfb_bytes = atoms * nb * 512;
    static constexpr int stage = (a_bytes + b_bytes + sfa_bytes + sfb_bytes + 1023) / 1024 * 1024;
    static constexpr int stages = 200 * 1024 / stage;
    static constexpr int smem = stages * stage + 1024;
    static constexpr int sf_cols = atoms * 4 * (1 + nb);     // TMEM columns of one stage's scales
    static constexpr int sf0 = 2 * NT;                       // after two accumulators
    static constexpr int sf_sets = sf0 + 2 * sf_cols <= 512 ? 2 : 1;
    static constexpr int cols_used = sf0 + sf_sets * sf_cols;
    static constexpr int cols = cols_used <= 128 ? 128 : cols_used <= 256 ? 256 : 512;
    static_assert(NT % step == 0 && NT % 32 == 0 && rows % box == 0 && box % 8 == 0, "whole swizzle atoms");
    static_assert(cols_used <= 512, "TMEM holds 512 columns");
};

struct FpArgs {
    const uint32_t* xs;      // scale words of the rows
    const uint8_t* ws;       // scale tiles of the weights
    uint4* xtiles;           // pairs: the scales of every row tile, see fp4_tile_scales_kernel
    int64_t max_xtiles;
    int64_t P;
    int K, E, R, KS;         // KS: stages per tile
    int xwords, wwords;      // scale words per row
    const int32_t* offsets;
    const float* alpha;
    uint64_t* flags;
    float* partial;
    uint64_t* err;
    int withhold;            // the wait test: 0 CTA 0's first stage, 1 the flags
};

// Where every expert's tiles start, in shared memory.
struct FpPlan {
    int32_t begin[kFpMaxE + 1];
    int64_t tile0[kFpMaxE + 1];
    int64_t warp_sum[kFpMaxWarps];
};

// Each thread takes four experts; offsets are clamped so that no value of them
// leads out of the buffers.
template <int NT, int M>
__device__ __forceinline__ void fp_plan(const FpArgs& a, FpPlan& p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int RT = (a.R - 1) / M + 1;                     // R may be 2^31 - 1
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

// The share of every CTA (or pair): tiles c, c + G, .. of the first waves * G, and
// units [lo(c), lo(c + 1)) of the tiles from tile0 on.  As many CTAs share those as
// get min_units each, or one tile each where that is more, so that no run between
// two others is empty: whoever begins a tile waits for every CTA up to the tile's
// end.
struct FpRun {
    int64_t G, waves, tile0, U, sharers;
    __device__ __forceinline__ FpRun(const FpArgs& a, const FpPlan& p, int grid, int min_units) {  // grid: CTAs, or pairs
        const int64_t tiles = p.tile0[a.E];
        G = min((int64_t)grid, max(tiles, tiles * a.KS / min_units));
        G = max(G, (int64_t)1);
        waves = tiles / G;
        tile0 = waves * G;
        U = (tiles - tile0) * a.KS;
        sharers = max(min(G, max(tiles - tile0, U / min_units)), (int64_t)1);
    }
    __device__ __forceinline__ int64_t lo(int64_t c) const { return c >= sharers ? U : U * c / sharers; }
};

// Tensor maps of a launch: codes of the weights and of the rows; for pairs their scale
// tiles as well (rows of 512 bytes).
template <bool PAIR> struct FpMaps {
    CUtensorMap w, x;
};
template <> struct FpMaps<true> {
    CUtensorMap w, x, ws, xs;
};

struct FpTile {
    int e, rt, n;       // expert, weight-row tile, rows in the tile
    int64_t p0;         // first row
};

// Not inlined: five roles call it once a tile, and the loops between those calls
// have to stay in the instruction cache together.
template <int NT>
__device__ __noinline__ FpTile fp_tile(const FpPlan& p, int E, int64_t tile) {
    int lo = 0, hi = E;  // the last expert whose first tile is not after this one
    while (hi - lo > 1) {
        const int m = (lo + hi) / 2;
        if (p.tile0[m] <= tile) lo = m; else hi = m;
    }
    FpTile t;
    t.e = lo;
    const int rows = p.begin[lo + 1] - p.begin[lo];
    const int nj = (rows - 1) / NT + 1;  // a tile's expert has rows, up to 2^31 - 1
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
// in the four lane quarters (in both CTAs of a pair, each from its own)
template <bool PAIR>
__device__ __forceinline__ void tc_copy_scales_elect(uint32_t dst, uint64_t desc, uint32_t go) {
    if (PAIR)
        asm volatile(
            "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n setp.ne.and.b32 e, %2, 0, e;\n"
            " @e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}" ::"r"(dst), "l"(desc), "r"(go) : "memory");
    else
        asm volatile(
            "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n setp.ne.and.b32 e, %2, 0, e;\n"
            " @e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}" ::"r"(dst), "l"(desc), "r"(go) : "memory");
}

// instruction descriptor of a block-scaled product of E2M1 operands, both
// K-major: types 1 (E2M1), N / 8, scale type (1 E8M0, 0 E4M3), M / 128;
// the bytes of a scale word that apply are added per product
template <bool NV, int M>
__device__ __forceinline__ constexpr uint32_t idesc_fp4(int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((NV ? 0u : 1u) << 23) | ((uint32_t)(M >> 7) << 27);
}

#define COLI_MMA_FP4(GROUP, KIND)                                                                              \
    asm volatile("{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"             \
                 " setp.ne.and.b32 e, %7, 0, e;\n"                                                            \
                 " @e tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], p;\n}"    \
                 ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(go))
template <bool NV, bool PAIR>
__device__ __forceinline__ void tc_mma_fp4_elect(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t sfa, uint32_t sfb, uint32_t accumulate, uint32_t go) {
    if constexpr (PAIR && NV) COLI_MMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (PAIR) COLI_MMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
    else if constexpr (NV) COLI_MMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else COLI_MMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
}
#undef COLI_MMA_FP4

// A whole stage in one piece of code that one elected lane runs: the scale tiles
// to TMEM (A's at sf, then B's, NB of them per scale tile of K), four products and
// the arrival at `empty`.  Issued one by one, each with its own election and
// address arithmetic, the eleven to seventeen instructions take 510 cycles, more
// than the 448 that a 256 x 224 stage keeps the tensor unit busy.
#define COLI_CP(G, P, DST, SRC)                                                                                  \
    " add.u32 t, %6, " #DST ";\n add.u64 x, %" SRC ";\n"                                                        \
    " @" P " tcgen05.cp.cta_group::" G ".32x128b.warpx4 [t], x;\n"
#define COLI_STAGE_MMA(G, KIND, J, M, ID, SFA, SFB)                                                               \
    " add.u64 x, %1, " #J ";\n add.u64 z, %2, " #J ";\n add.u32 i, %3, " #ID ";\n add.u32 t, %6, " #SFA ";\n"    \
    " add.u32 u, %6, " #SFB ";\n @e tcgen05.mma.cta_group::" G ".kind::" KIND " [%0], x, z, i, [t], [u], " M ";\n"
#define COLI_STAGE_BEGIN                                                                                          \
    "{\n .reg .pred e, f, m, n;\n .reg .b64 x, z;\n .reg .b32 t, u, i;\n elect.sync _|e, 0xffffffff;\n"          \
    " setp.ne.and.b32 e, %11, 0, e;\n"                                                                            \
    " setp.ne.b32 m, %7, 0;\n setp.ne.and.b32 f, %8, 0, e;\n setp.eq.b32 n, 0, 0;\n"
#define COLI_STAGE_OPERANDS                                                                                       \
    ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "l"(sfa), "l"(sfb), "r"(sf), "r"(more), "r"(second), "r"(empty),      \
        "h"((uint16_t)3), "r"(go)                                                                                 \
        : "memory"
#define COLI_COMMIT_1 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%9];\n}"
#define COLI_COMMIT_2                                                                                             \
    " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%9], %10;\n}"
// ID of a product that takes the upper two bytes of its scale words: 2 << 29 | 2 << 4
#define COLI_MX "mxf4.block_scale.scale_vec::2X"
#define COLI_NV "mxf4nvf4.block_scale.scale_vec::4X"
template <bool NV, bool PAIR>
__device__ __forceinline__ void fp4_stage(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint64_t sfa,
                                          uint64_t sfb, uint32_t sf, uint32_t more, uint32_t second, uint32_t empty,
                                          uint32_t go) {
    if constexpr (PAIR && NV)
        asm volatile(COLI_STAGE_BEGIN
                     COLI_CP("2", "e", 0, "4, 0") COLI_CP("2", "e", 16, "5, 0") COLI_CP("2", "f", 20, "5, 32")
                     COLI_CP("2", "e", 4, "4, 32") COLI_CP("2", "e", 24, "5, 64") COLI_CP("2", "f", 28, "5, 96")
                     COLI_CP("2", "e", 8, "4, 64") COLI_CP("2", "e", 32, "5, 128") COLI_CP("2", "f", 36, "5, 160")
                     COLI_CP("2", "e", 12, "4, 96") COLI_CP("2", "e", 40, "5, 192") COLI_CP("2", "f", 44, "5, 224")
                     COLI_STAGE_MMA("2", COLI_NV, 0, "m", 0, 0, 16) COLI_STAGE_MMA("2", COLI_NV, 2, "n", 0, 4, 24)
                     COLI_STAGE_MMA("2", COLI_NV, 4, "n", 0, 8, 32) COLI_STAGE_MMA("2", COLI_NV, 6, "n", 0, 12, 40)
                     COLI_COMMIT_2 COLI_STAGE_OPERANDS);
    else if constexpr (PAIR)
        asm volatile(COLI_STAGE_BEGIN
                     COLI_CP("2", "e", 0, "4, 0") COLI_CP("2", "e", 8, "5, 0") COLI_CP("2", "f", 12, "5, 32")
                     COLI_CP("2", "e", 4, "4, 32") COLI_CP("2", "e", 16, "5, 64") COLI_CP("2", "f", 20, "5, 96")
                     COLI_STAGE_MMA("2", COLI_MX, 0, "m", 0, 0, 8) COLI_STAGE_MMA("2", COLI_MX, 2, "n", 0x40000020, 0, 8)
                     COLI_STAGE_MMA("2", COLI_MX, 4, "n", 0, 4, 16) COLI_STAGE_MMA("2", COLI_MX, 6, "n", 0x40000020, 4, 16)
                     COLI_COMMIT_2 COLI_STAGE_OPERANDS);
    else if constexpr (NV)
        asm volatile(COLI_STAGE_BEGIN
                     COLI_CP("1", "e", 0, "4, 0") COLI_CP("1", "e", 16, "5, 0")
                     COLI_CP("1", "e", 4, "4, 32") COLI_CP("1", "e", 20, "5, 32")
                     COLI_CP("1", "e", 8, "4, 64") COLI_CP("1", "e", 24, "5, 64")
                     COLI_CP("1", "e", 12, "4, 96") COLI_CP("1", "e", 28, "5, 96")
                     COLI_STAGE_MMA("1", COLI_NV, 0, "m", 0, 0, 16) COLI_STAGE_MMA("1", COLI_NV, 2, "n", 0, 4, 20)
                     COLI_STAGE_MMA("1", COLI_NV, 4, "n", 0, 8, 24) COLI_STAGE_MMA("1", COLI_NV, 6, "n", 0, 12, 28)
                     COLI_COMMIT_1 COLI_STAGE_OPERANDS);
    else
        asm volatile(COLI_STAGE_BEGIN
                     COLI_CP("1", "e", 0, "4, 0") COLI_CP("1", "e", 8, "5, 0")
                     COLI_CP("1", "e", 4, "4, 32") COLI_CP("1", "e", 12, "5, 32")
                     COLI_STAGE_MMA("1", COLI_MX, 0, "m", 0, 0, 8) COLI_STAGE_MMA("1", COLI_MX, 2, "n", 0x40000020, 0, 8)
                     COLI_STAGE_MMA("1", COLI_MX, 4, "n", 0, 4, 12) COLI_STAGE_MMA("1", COLI_MX, 6, "n", 0x40000020, 4, 12)
                     COLI_COMMIT_1 COLI_STAGE_OPERANDS);
}
#undef COLI_CP
#undef COLI_STAGE_MMA
#undef COLI_STAGE_BEGIN
#undef COLI_STAGE_OPERANDS
#undef COLI_COMMIT_1
#undef COLI_COMMIT_2
#undef COLI_MX
#undef COLI_NV

// A role's place in the ring: slot, the phase of its barriers, and whether the
// slot has been used before.
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    bool again = false;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
            again = true;
        }
    }
    __device__ __forceinline__ Ring back(int stages) const {  // a whole ring earlier
        Ring r;
        r.s = s;
        r.phase = phase ^ 1;
        return r;
    }
};

// Warp-wide wait for the flags of `parts` CTAs' store warps, `step` flags apart, a
// lane each: some ten seconds at most, since those CTAs may have to wait for an SM
// that another stream's kernel holds.  False as well where a CTA has no piece to give.
__device__ __forceinline__ bool fp_wait_flags(const uint64_t* flags, int64_t step, int64_t parts, uint32_t tries) {
    bool ok = true;
    for (int64_t c = threadIdx.x & 31; c < parts; c += 32) {
        uint64_t v = 0;
        for (uint32_t i = 0; i < tries && v != kFpRaised && v != kFpBroken; ++i)
            asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(flags + c * step) : "memory");
        if (v != kFpRaised) ok = false;
    }
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();  // what one lane has acquired, all lanes read
    return ok;
}

// A barrier's wait; of a pair's barriers, which either CTA's copies and products arrive at,
// acquiring what the cluster has released there.
template <bool PAIR>
__device__ __forceinline__ bool fp_wait(uint64_t* bar, uint32_t parity, uint32_t tries) {
    return PAIR ? mbar_wait_cluster(bar, parity, nullptr, tries) : mbar_wait(bar, parity, nullptr, tries);
}

// boxes of the TMA copies of `count` rows, none for fewer than one
template <class C> __device__ __forceinline__ int fp_boxes(int count) { return max(0, (count + C::box - 1) / C::box); }

// Scales of the rows for pairs: for every tile of NT rows of an expert and every stage the
// scale tiles that the products read ([atoms][nb] of 512 bytes, see FpShape), since an
// expert's rows start anywhere and a scale tile only at multiples of 128.  A pair's
// products read both CTAs' shared memory on the word of one barrier: what is there has to
// have come by copies that arrive at that barrier themselves.  (Gathered by cp.async in
// each CTA, CTA 1's writes need a release to the cluster before every arrival at CTA 0,
// which takes some 1650 cycles: 842 us for 32768 rows on 32 experts of 4096 x 6144 with one
// warp that releases, 396 with four, 357 without the release, which nothing then orders;
// 346 this way; 400 rows of 10240 x 2048: 13.0 and 15.3, this kernel's chain of loads before
// the product's own.)
// A warp takes two words of a tile's rows at a time: 16 loads of a lane in flight.
constexpr int kFpTileScaleThreads = 256;
template <int NT, int M, int NB>
__global__ void __launch_bounds__(kFpTileScaleThreads)
fp4_tile_scales_kernel(FpArgs a, int words) {   // words: of a tile's row, a multiple of 2
    __shared__ FpPlan plan;
    static_assert(4 * kFpTileScaleThreads >= kFpMaxE, "fp_plan takes four experts a thread");
    pdl_trigger();
    pdl_wait();
    fp_plan<NT, M>(a, plan);
    const int lane = threadIdx.x & 31, RT = (a.R - 1) / M + 1;
    const int64_t xtiles = min(plan.tile0[a.E] / RT, a.max_xtiles);
    const int64_t step = (int64_t)gridDim.x * (kFpTileScaleThreads / 32), pairs = words / 2;
    for (int64_t i = (int64_t)blockIdx.x * (kFpTileScaleThreads / 32) + (threadIdx.x >> 5); i < xtiles * pairs; i += step) {
        const int64_t xt = i / pairs;
        const int w0 = 2 * (int)(i - xt * pairs);
        int lo = 0, hi = a.E;  // the last expert whose first tile is not after this one
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (plan.tile0[m] <= xt * RT) lo = m; else hi = m;
        }
        const int64_t p0 = plan.begin[lo] + (xt - plan.tile0[lo] / RT) * NT, end = plan.begin[lo + 1];
        uint32_t v[2][NB][4];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int h = 0; h < NB; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t r = p0 + 128 * h + 32 * j + lane;
                    v[w][h][j] = r < end && w0 + w < a.xwords ? a.xs[scale_word(r, w0 + w, a.xwords)] : 0;
                }
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int h = 0; h < NB; ++h)
                a.xtiles[((xt * words + w0 + w) * NB + h) * 32 + lane] = make_uint4(v[w][h][0], v[w][h][1], v[w][h][2], v[w][h][3]);
    }
}

// NaN where a store warp has no sums: groups of 16 columns of y from c0 on, `step` apart
// (not inlined: the loop that stores has to keep its registers, few enough that the next
// kernel's CTAs fit beside this one's)
template <typename YT>
__device__ __noinline__ void fp_store_nan(YT* yp, int R, int c0, int n, int step) {
    for (; c0 < n; c0 += step, yp += (int64_t)step * R)
        for (int i = 0; i < min(16, n - c0); ++i) yp[i * (int64_t)R] = from_f32<YT>(__uint_as_float(0x7fc00000u));
}

// A wait that gives up (ok) makes its lane issue nothing more.  What is then never issued
// makes the waits on it give up in turn, the store warps write NaN for the tiles that they
// begin and raise kFpBroken for those they do not, and the workspace's first word becomes
// kFpBroken: a call that finds it there has nothing but NaN to give, for the flags may hold
// what that call left.  Every copy is in flight for microseconds and was issued before the
// wait that gave up began, so none is when the CTAs leave; products in flight are waited for.
// TW: the wait test (coli_moe_fp4_set_wait_test), an instantiation of its own so that the
// others keep their limits at compile time.
template <int NT, bool NV, bool PAIR, typename YT, bool TW>
__global__ void __launch_bounds__(FpShape<NT, NV, PAIR>::bound, 1)
fp4_product_kernel(const __grid_constant__ FpMaps<PAIR> maps, FpArgs a, YT* y) {
    using C = FpShape<NT, NV, PAIR>;
    extern __shared__ uint8_t fp_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(fp_raw) + 1023) & ~uintptr_t(1023));
    __shared__ FpPlan plan;
    __shared__ __align__(8) uint64_t full[C::stages], empty[C::stages], accfull[2], accempty[2], done;
    __shared__ uint32_t tmem_slot;
    constexpr uint32_t tries = TW ? kFpTestTries : kWaitTries;
    const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    // of the pair's work, this CTA's part
    const int rank = PAIR ? (int)cluster_rank() : 0, unit = (int)blockIdx.x / C::ctas;

    if (warp == 0) {
        if (PAIR) tmem_alloc_pair(&tmem_slot, C::cols);
        else tmem_alloc(&tmem_slot, C::cols);
    }
    if (threadIdx.x == 32) {
        for (int s = 0; s < C::stages; ++s) {
            // the copies' announcement (of a pair's: CTA 0's, for both), the lanes of the scale warps
            mbar_init(&full[s], PAIR ? 1 : 1 + 32 * kFpScaleWarps);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accfull[b], 1);
            mbar_init(&accempty[b], C::store_warps * C::ctas);
        }
        mbar_init(&done, 1);
        fence_mbar_init();
    }
    pdl_trigger();
    pdl_wait();
    const uint64_t before = *reinterpret_cast<const volatile uint64_t*>(a.err);
    fp_plan<NT, C::M>(a, plan);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the other CTA's barriers are set up
    tc_fence_after();
    const uint32_t tmem = uniform(tmem_slot);
    const FpRun run(a, plan, gridDim.x / C::ctas, kFpMinUnits);
    FpPieces q(a, run, unit);
    bool ok = before != kFpBroken;  // cleared by a wait that gave up

    if (warp == 0) {
        // ---------------- copies (whole warp, an elected lane issues) ----------------
        Ring ring;
        const uint32_t bars = PAIR ? uniform(mapa_u32(smem_u32(full), 0)) : 0;  // CTA 0's
        while (uniform((int)q.next())) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            // this CTA's share of the rows: half of N, itself a multiple of 16
            const int half = (t.n + C::step - 1) / C::step * 16;
            const int first = PAIR ? rank * half : 0;
            const int p0 = uniform((int)min(t.p0 + first, a.P - 1));  // past the last row: nothing to copy
            const int boxes = uniform(PAIR ? fp_boxes<C>(min(half, t.n - first)) : 1);
            const int wrow = uniform(t.e * a.R + t.rt * C::M + rank * 128);
            const int k0 = uniform(q.k0), k1 = uniform(q.k1);
            // past the expert's last weight row (the second half of a tile may be) the products are
            // not stored: any scales do
            const int block = uniform(t.rt * C::M + rank * 128 < a.R ? wrow >> 7 : (wrow >> 7) - 1);
            if constexpr (PAIR) {
                // What both CTAs copy is counted at CTA 0's barrier, which announces it.
                const int both = uniform(fp_boxes<C>(min(half, t.n)) + fp_boxes<C>(min(half, t.n - half)));
                const uint32_t bytes = 2 * (C::a_bytes + C::sfa_bytes + C::sfb_bytes) + both * C::box * 128;
                const int64_t xtile = plan.tile0[t.e] / ((a.R - 1) / C::M + 1) + (t.p0 - plan.begin[t.e]) / NT;
                const int wsrow = uniform((int)((int64_t)block * a.wwords));
                const int xsrow = uniform((int)(xtile * a.KS * (C::atoms * C::nb)));
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                    if (ok && ring.again && !fp_wait<PAIR>(&empty[ring.s], ring.phase ^ 1, tries)) ok = false;
                    const uint32_t go = ok && !(TW && a.withhold == 0 && blockIdx.x == 0 && !ring.again && ring.s == 0);
                    uint8_t* st = smem + ring.s * C::stage;
                    const uint32_t bar = bars + 8 * ring.s;
                    if (rank == 0) mbar_expect_tx_elect(&full[ring.s], bytes, go);
                    tma_load_2d_pair_elect(st, &maps.w, k * 128, wrow, bar, go);
#pragma unroll
                    for (int b = 0; b < C::rows / C::box; ++b)
                        if (b < boxes)
                            tma_load_2d_pair_elect(st + C::a_bytes + b * C::box * 128, &maps.x, k * 128, p0 + b * C::box,
                                                   bar, go);
                    uint8_t* sf = st + C::a_bytes + C::b_bytes;
                    tma_load_2d_pair_elect(sf, &maps.ws, 0, wsrow + k * C::atoms, bar, go);
                    tma_load_2d_pair_elect(sf + C::sfa_bytes, &maps.xs, 0, xsrow + k * (C::atoms * C::nb), bar, go);
                    ring.next(C::stages);
                }
            } else {
                const uint8_t* sfa = a.ws + ((int64_t)block * a.wwords + k0 * C::atoms) * 512;
                const uint32_t bytes = (uint32_t)(C::a_bytes + C::b_bytes);
#pragma unroll 1
                for (int k = k0; k < k1; ++k) {
                    if (ok && ring.again && !fp_wait<PAIR>(&empty[ring.s], ring.phase ^ 1, tries)) ok = false;
                    const uint32_t go = ok && !(TW && a.withhold == 0 && blockIdx.x == 0 && !ring.again && ring.s == 0);
                    uint8_t* st = smem + ring.s * C::stage;
                    uint64_t* bar = &full[ring.s];
                    const uint32_t na = (uint32_t)min(C::atoms, a.wwords - k * C::atoms) * 512;
                    mbar_expect_tx_elect(bar, bytes + na, go);
                    tma_load_2d_elect(st, &maps.w, k * 128, wrow, bar, go);
                    tma_load_2d_elect(st + C::a_bytes, &maps.x, k * 128, p0, bar, go);
                    bulk_g2s_elect(st + C::a_bytes + C::b_bytes, sfa, na, bar, go);
                    sfa += C::atoms * 512;
                    ring.next(C::stages);
                }
            }
        }
        // the last copies (of a pair, both CTAs') have landed before a CTA may end
        Ring last = ring.back(C::stages);
        if (rank == 0 && ok)
            for (int i = 0; i < C::stages; ++i, last.next(C::stages))
                if ((ring.again || last.s < ring.s) && !fp_wait<PAIR>(&full[last.s], last.phase, TW ? tries : kSleepTries))
                    ok = false;
    } else if (warp == 1 && rank == 1) {
        // CTA 0 issues the products of a pair
    } else if (warp == 1) {
        // ---------------- products (whole warp, an elected lane issues) ----------------
        Ring ring;
        const uint32_t sbase = uniform(smem_u32(smem));
        uint32_t sf = uniform(tmem + C::sf0);  // the stage's scales in TMEM: the sets in turn
        int piece = 0;
        bool ready = false;                   // the ring's next stage has been seen to be full
        for (; uniform((int)q.next()); ++piece) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            const uint32_t idesc = uniform(idesc_fp4<NV, C::M>((t.n + C::step - 1) / C::step * C::step));
            const int second = C::nb > 1 ? uniform(t.n > 128 ? 1 : 0) : 0;
            const int k0 = uniform(q.k0), k1 = uniform(q.k1);
            const int buf = piece & 1;
            if (piece >= 2 && ok && !mbar_wait_cluster(&accempty[buf], ((piece >> 1) - 1) & 1, nullptr, tries)) ok = false;
            tc_fence_after();
            const uint32_t d = tmem + NT * buf;
            uint32_t more = 0;                // 0: the tile's first product clears the accumulator
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
                if (!ready && ok && !fp_wait<PAIR>(&full[ring.s], ring.phase, tries)) ok = false;
                const uint32_t go = ok;
                tc_fence_after();
                // the scale warps' copies are writes of the generic proxy, and the tensor unit reads
                // them: fenced here, where they are known to have landed
                if (!PAIR) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                const uint32_t st = sbase + ring.s * C::stage;
                const uint64_t sfa = smem_desc_scales(st + C::a_bytes + C::b_bytes);
                const uint64_t sfb = sfa + (C::sfa_bytes >> 4);
                const uint64_t ad = smem_desc_sw128_at(st), bd = ad + (C::a_bytes >> 4);
                const int cols = a.K - 256 * k;
                uint64_t* empty_s = &empty[ring.s];
                ring.next(C::stages);
                // asked before this stage is issued, so that the answer is there after it
                ready = PAIR ? mbar_test_cluster(&full[ring.s], ring.phase) : mbar_test(&full[ring.s], ring.phase);
                if (cols >= 256) {
                    fp4_stage<NV, PAIR>(d, ad, bd, idesc, sfa, sfb, sf, more, second, smem_u32(empty_s), go);
                } else {  // the row's last columns
#pragma unroll
                    for (int i = 0; i < C::atoms; ++i) {
                        if (i * (256 / C::atoms) >= cols) break;
                        tc_copy_scales_elect<PAIR>(sf + 4 * i, sfa + 32 * i, go);
                        tc_copy_scales_elect<PAIR>(sf + 4 * C::atoms + 4 * C::nb * i, sfb + 32 * C::nb * i, go);
                        if (second)
                            tc_copy_scales_elect<PAIR>(sf + 4 * C::atoms + 4 * C::nb * i + 4, sfb + 32 * C::nb * i + 32, go);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (64 * j >= cols) break;
                        const int at = NV ? j : j >> 1;              // scale tile
                        const uint32_t id = NV ? 0u : 2u * (j & 1);  // first byte of its words
                        tc_mma_fp4_elect<NV, PAIR>(d, ad + 2 * j, bd + 2 * j, idesc | id << 29 | id << 4, sf + 4 * at,
                                                   sf + 4 * C::atoms + 4 * C::nb * at, j > 0 ? 1u : more, go);
                    }
                    if (PAIR) tc_commit_pair_elect(empty_s, go);
                    else tc_commit_elect(empty_s, go);
                }
                more = 1;
                if (C::sf_sets == 2) sf = 2 * (tmem + C::sf0) + C::sf_cols - sf;
            }
            if (PAIR) tc_commit_pair_elect(&accfull[buf], ok);
            else tc_commit_elect(&accfull[buf], ok);
        }
        if (PAIR) tc_commit_of_pair_elect(&done, !ok);
        else tc_commit_elect(&done, !ok);
        if (!ok) mbar_wait(&done, 0, nullptr, tries);
    } else if (PAIR && warp < 4) {
        // nothing: a warp reads the accumulator's quarter of its index, so the stores begin at warp 4
    } else if (!PAIR && (warp < 4 || warp >= 8)) {
        // ---------------- scales of the rows ----------------
        // A stage has atoms * NT / 32 runs of 32 rows' words; warp f takes runs f, f + 4, ..: a
        // lane copies its row's word to where the scale tile has it.  The copies are asynchronous
        // and arrive at the barrier by themselves, so a stage's are in flight as long as its TMA
        // copies are; through registers, loaded some stages ahead, the unrolled code took more
        // time in the instruction cache than its loads saved.
        constexpr int words = NT / 32;
        constexpr int items = C::atoms * words;
        constexpr int mine = (items + kFpScaleWarps - 1) / kFpScaleWarps;
        const int f = warp < 4 ? warp - 2 : warp - 6;
        const uint32_t sbase = uniform(smem_u32(smem));
        uint32_t to[mine];           // byte of the stage
#pragma unroll
        for (int i = 0; i < mine; ++i) {
            const int it = min(f + kFpScaleWarps * i, items - 1), atom = it / words, j = it - atom * words;
            to[i] = sbase + C::a_bytes + C::b_bytes + C::sfa_bytes + 512 * (C::nb * atom + j / 4) + 16 * lane + 4 * (j & 3);
        }
        Ring ring;
        bool free = false;           // the ring's next slot has been seen to be free
        while (uniform((int)q.next())) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            const int k0 = uniform(q.k0), k1 = uniform(q.k1);
            const uint32_t* from[mine];
#pragma unroll
            for (int i = 0; i < mine; ++i) {
                const int it = min(f + kFpScaleWarps * i, items - 1), atom = it / words, j = it - atom * words;
                // rows past the tile's are not stored: any row's scales do for them
                from[i] = a.xs + scale_word(min(t.p0 + 32 * j + lane, a.P - 1), k0 * C::atoms + atom, a.xwords);
            }
#pragma unroll 1
            for (int k = k0; k < k1; ++k) {
                if (ok && ring.again && !free && !mbar_wait(&empty[ring.s], ring.phase ^ 1, nullptr, tries)) ok = false;
                if (!ok) continue;
                const uint32_t at = ring.s * C::stage;
                uint64_t* full_s = &full[ring.s];
                ring.next(C::stages);
                free = ring.again && mbar_test(&empty[ring.s], ring.phase ^ 1);
                const int left = a.xwords - k * C::atoms;  // scale tiles that the row still has
#pragma unroll
                for (int i = 0; i < mine; ++i) {
                    const int atom = min(f + kFpScaleWarps * i, items - 1) / words;
                    if (atom < left) cp_async4(at + to[i], from[i]);
                    from[i] += C::atoms * 128;
                }
                cp_async_arrive(full_s);
            }
        }
        cp_async_wait_all();         // the last copies have landed before the CTA may end
    } else {
        // ---------------- stores: weight rows 32 quarter + lane of the tile ----------------
        // A warp reaches its own quarter of the accumulator's lanes alone.  Tiles of many rows have
        // two warps to a quarter, each with every second group of 16 columns: with one, a tile's
        // stores take 4.2 us, as long as ten stages (with two, 3.3 us).
        const int quarter = warp & 3, half = warp < 8 ? 0 : 1, flag = 2 * quarter + half;
        for (int piece = 0; uniform((int)q.next()); ++piece) {
            const FpTile t = fp_tile<NT>(plan, a.E, q.tile);
            const int buf = piece & 1, n = uniform(t.n);
            const int row = t.rt * C::M + 128 * rank + 32 * quarter + lane;
            const bool begins = uniform((int)(q.k0 == 0));
            const float al = begins && a.alpha ? a.alpha[t.e] : 1.0f;
            // the CTAs (or pairs) after this one with pieces of the tile: up to the first whose
            // run starts at its end or later; of a pair, the CTA with the same weight rows
            int64_t parts = 0;
            if (begins && q.k1 < a.KS)
                while (run.lo(unit + 1 + parts) < (q.tile + 1 - run.tile0) * a.KS) ++parts;
            parts = uniform(parts);
            const int64_t other = (int64_t)blockIdx.x + C::ctas;  // the first of them
            uint64_t* flags = a.flags + kFpStoreWarps * other + flag;
            const float* theirs = a.partial + other * (128 * NT) + 16 * half * 128 + 32 * quarter + lane;
            if (ok && !fp_wait<PAIR>(&accfull[buf], (piece >> 1) & 1, tries)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            if (parts && ok && !fp_wait_flags(flags, kFpStoreWarps * C::ctas, parts, TW ? tries : kFpFlagTries)) ok = false;
            const uint32_t d = tmem + ((uint32_t)(32 * quarter) << 16) + NT * buf;
            YT* yp = y + (t.p0 + 16 * half) * a.R + row;  // this lane's row of y's columns
            float* pp = a.partial + (int64_t)blockIdx.x * (128 * NT) + 16 * half * 128 + 32 * quarter + lane;
            if (!ok && begins && row < a.R) fp_store_nan(yp, a.R, 16 * half, n, 16 * C::groups);
#pragma unroll 1
            for (int c0 = ok ? 16 * half : n; c0 < n; c0 += 16 * C::groups) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(d + c0, v);
                tmem_wait_ld();
                const int m = n - c0;             // columns of this group, if fewer than 16
                if (!begins) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < m) pp[i * 128] = __uint_as_float(v[i]);
                }
                // pieces in the order of their columns, the loads of some at a time in flight
                constexpr int at_once = PAIR ? 2 : 4;
#pragma unroll 1
                for (int64_t c = 0; c < parts; c += at_once) {
                    float p[at_once][16];
#pragma unroll
                    for (int u = 0; u < at_once; ++u)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + u < parts && i < m) p[u][i] = __ldcg(theirs + (c + u) * (C::ctas * 128 * NT) + i * 128);
#pragma unroll
                    for (int u = 0; u < at_once; ++u)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + u < parts && i < m) v[i] = __float_as_uint(__uint_as_float(v[i]) + p[u][i]);
                }
                if (begins && row < a.R) {
                    if (m >= 16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) yp[i * (int64_t)a.R] = from_f32<YT>(__uint_as_float(v[i]) * al);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < m) yp[i * (int64_t)a.R] = from_f32<YT>(__uint_as_float(v[i]) * al);
                    }
                }
                yp += 16 * C::groups * (int64_t)a.R;
                pp += 16 * C::groups * 128;
                theirs += 16 * C::groups * 128;
            }
            __syncwarp();
            if (!begins && lane == 0 && !(TW && a.withhold == 1)) {
                __threadfence();
                asm volatile("st.release.gpu.global.u64 [%0], %1;"
                             ::"l"(a.flags + kFpStoreWarps * (int64_t)blockIdx.x + flag), "l"(ok ? kFpRaised : kFpBroken)
                             : "memory");
            }
            for (int64_t c = lane; c < parts; c += 32)  // read once: down again for the next call
                flags[c * (kFpStoreWarps * C::ctas)] = 0;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_cluster(&accempty[buf], 0);
                else mbar_arrive(&accempty[buf]);
            }
        }
    }
    if (!ok) *reinterpret_cast<volatile uint64_t*>(a.err) = kFpBroken;
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // neither CTA leaves while the other may reach into it
    tc_fence_after();
    if (warp == 0) {
        if (PAIR) tmem_dealloc_pair(tmem, C::cols);
        else tmem_dealloc(tmem, C::cols);
    }
}

}  // namespace coli
