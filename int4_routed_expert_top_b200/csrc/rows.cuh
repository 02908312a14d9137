// rows.cuh - picks sorted by expert, tokens copied into that order and rows
// summed back to their tokens, with the gradients of both.
//
// Sort: a stable counting sort of the linear pick index i = t * k + j by its
// expert, so rows come in the order (expert, token, slot) with no atomics and
// the same result at every run.  A warp reads 32 consecutive picks, finds the
// lanes of equal expert with match.any, and keeps its own counts per expert in
// shared memory; a pick's row is the count of its expert in everything before
// it.  Up to kSortOneCta picks one CTA does it all (one launch, the case of
// decode: 2.7 us at 8 picks; 4096 picks would take it 11.3 us, the two launches
// take 7.4 us for 8192); above, at most kSortMaxChunks CTAs count their chunk of
// the picks first and a second launch places them (65536 picks: 14.9 us; with
// 128 chunks, whose counts every CTA adds up, 21.8 us).
//
// The copies and sums are bound by HBM (each row of xs / o once): a lane owns 16
// bytes of columns and walks the token's picks.  8192 tokens x 8 picks (a fifth
// dropped) of 6144 bf16: copies 118 us (6.3 TB/s), sort 15 us.  4096 x 8 (a tenth
// dropped): sums 95 us (5.9 TB/s), their gradient 131 us (6.3), sums without
// weights 73 us (5.6).  Rows whose length or address allows no 16-byte access take
// about 1.5 times as long.
#pragma once

#include "vec.cuh"

namespace coli {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortOneCta = 1024;     // picks
constexpr int kSortMaxChunks = 64;

// expert of pick i, E for one that is not computed
__device__ __forceinline__ int pick_expert(const int32_t* idx, const float* w, int64_t i, int E) {
    const int e = idx[i];
    const bool live = e >= 0 && e < E && (w == nullptr || w[i] != 0.0f);
    return live ? e : E;
}

// Counts of the picks [begin, end) by expert and warp, cnt [warps][E]: warp w
// takes the w-th of equal runs of whole 32-pick groups.
__device__ __forceinline__ void sort_count(const int32_t* idx, const float* w, int64_t begin,
                                           int64_t end, int64_t run, int E, int* cnt) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    int* mine = cnt + warp * E;
    const int64_t b = begin + warp * run, e1 = min(end, b + run);
    for (int64_t i0 = b; i0 < e1; i0 += 32) {
        const int e = i0 + lane < e1 ? pick_expert(idx, w, i0 + lane, E) : E;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e < E && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

// Exclusive prefix over the CTA of one value per expert (tot[e], E <= 1024),
// in place; tot[E] = the sum.  Two experts per thread.
__device__ __forceinline__ void sort_scan(int* tot, int E, int* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = 2 * threadIdx.x;
    const int a = e0 < E ? tot[e0] : 0, b = e0 + 1 < E ? tot[e0 + 1] : 0;
    int v = a + b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < warp; ++i) before += part[i];
    const int excl = before + v - a - b;
    if (e0 < E) tot[e0] = excl;
    if (e0 + 1 < E) tot[e0 + 1] = excl + a;
    if (threadIdx.x == kSortThreads - 1) tot[E] = before + v;
    __syncthreads();
}

// cnt [warps][E] -> first row of each (warp, expert); base[e] = the expert's
// first row of this CTA
__device__ __forceinline__ void sort_bases(int* cnt, const int* base, int E) {
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int at = base[e];
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = at;
            at += c;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void sort_place(const int32_t* idx, const float* w, int64_t begin,
                                           int64_t end, int64_t run, int k, int E, int* cnt,
                                           int32_t* pair_tok, int32_t* pair_slot, int32_t* inv) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* mine = cnt + warp * E;
    const int64_t b = begin + warp * run, e1 = min(end, b + run);
    for (int64_t i0 = b; i0 < e1; i0 += 32) {
        const int64_t i = i0 + lane;
        const bool in = i < e1;
        const int e = in ? pick_expert(idx, w, i, E) : E;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int p = -1;
        if (e < E) p = mine[e] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (e < E && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
        if (in) inv[i] = p;
        if (p >= 0) {
            const int t = (int)((uint32_t)i / (uint32_t)k);  // T * k <= 2^30
            if (pair_tok) pair_tok[p] = t;
            if (pair_slot) pair_slot[p] = (int)i - t * k;
        }
    }
}

// One CTA: all picks.  Dynamic shared memory: ints [warps][E], tot [E + 1].
__global__ void __launch_bounds__(kSortThreads)
sort_one_kernel(const int32_t* idx, const float* w, int P, int k, int E, int32_t* offsets,
                int32_t* pair_tok, int32_t* pair_slot, int32_t* inv) {
    extern __shared__ int so_smem[];
    __shared__ int part[kSortWarps];
    int* cnt = so_smem;
    int* tot = so_smem + kSortWarps * E;
    pdl_trigger();
    pdl_wait();
    const int run = ((P + 31) / 32 + kSortWarps - 1) / kSortWarps * 32;
    sort_count(idx, w, 0, P, run, E, cnt);
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int s = 0;
        for (int i = 0; i < kSortWarps; ++i) s += cnt[i * E + e];
        tot[e] = s;
    }
    __syncthreads();
    sort_scan(tot, E, part);
    for (int e = threadIdx.x; e <= E; e += kSortThreads) offsets[e] = tot[e];
    sort_bases(cnt, tot, E);
    sort_place(idx, w, 0, P, run, k, E, cnt, pair_tok, pair_slot, inv);
}

// counts[chunk][E] of each CTA's chunk of `chunk` picks
__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const int32_t* idx, const float* w, int64_t P, int64_t chunk, int E,
                  int32_t* counts) {
    extern __shared__ int so_smem[];
    pdl_trigger();
    pdl_wait();
    const int64_t b = blockIdx.x * chunk;
    sort_count(idx, w, b, min(P, b + chunk), chunk / kSortWarps, E, so_smem);
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int s = 0;
        for (int i = 0; i < kSortWarps; ++i) s += so_smem[i * E + e];
        counts[(int64_t)blockIdx.x * E + e] = s;
    }
}

// every CTA sums the chunks' counts before its own and places its picks
__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const int32_t* idx, const float* w, int64_t P, int64_t chunk, int k, int E,
                  const int32_t* counts, int32_t* offsets, int32_t* pair_tok, int32_t* pair_slot,
                  int32_t* inv) {
    extern __shared__ int so_smem[];
    __shared__ int part[kSortWarps];
    int* cnt = so_smem;
    int* tot = cnt + kSortWarps * E;
    int* before = tot + E + 1;
    const int64_t b = blockIdx.x * chunk;
    pdl_trigger();
    pdl_wait();
    sort_count(idx, w, b, min(P, b + chunk), chunk / kSortWarps, E, cnt);
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int all = 0, mine = 0;
#pragma unroll 16
        for (int c = 0; c < (int)gridDim.x; ++c) {
            const int v = counts[(int64_t)c * E + e];
            if (c < (int)blockIdx.x) mine += v;
            all += v;
        }
        tot[e] = all;
        before[e] = mine;
    }
    __syncthreads();
    sort_scan(tot, E, part);
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += kSortThreads) offsets[e] = tot[e];
    for (int e = threadIdx.x; e < E; e += kSortThreads) before[e] += tot[e];
    __syncthreads();
    sort_bases(cnt, before, E);
    sort_place(idx, w, b, min(P, b + chunk), chunk / kSortWarps, k, E, cnt, pair_tok, pair_slot, inv);
}

// A warp's picks of one token: lane j holds pick j's row and weight; live has a
// bit for each pick that is computed (0 <= row < P).
struct Picks {
    int row;
    float w;
    unsigned live;
    __device__ __forceinline__ Picks(const int32_t* inv, const float* weights, int64_t t, int k, int64_t P) {
        const int lane = threadIdx.x & 31;
        row = lane < k ? inv[t * k + lane] : -1;
        const bool in = row >= 0 && row < P;
        w = in && weights ? weights[t * k + lane] : 1.0f;
        live = __ballot_sync(0xffffffffu, in);
    }
};

// xs[inv[t, j]] = x[t]: block = (token, run of 256 N elements of type T, which
// stands for 16 bytes of a row or, where rows or pointers allow no more, for one or two
// of its elements, N of them a thread)
template <typename T, int N>
__global__ void __launch_bounds__(256)
dispatch_kernel(const T* __restrict__ x, int64_t P, int nvec, int per_row, int k,
                const int32_t* __restrict__ inv, T* __restrict__ xs) {
    const int64_t t = blockIdx.x / per_row;
    const int c = (int)(blockIdx.x - t * per_row) * 256 * N + threadIdx.x;
    pdl_trigger();
    pdl_wait();
    T v[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (c + 256 * i < nvec) v[i] = x[t * nvec + c + 256 * i];
    const Picks picks(inv, nullptr, t, k, P);
    for (unsigned live = picks.live; live; live &= live - 1) {
        const int64_t p = __shfl_sync(0xffffffffu, picks.row, __ffs(live) - 1);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + 256 * i < nvec) xs[p * nvec + c + 256 * i] = v[i];
    }
}

// y[t] = residual[t] + sum_j w[t, j] o[inv[t, j]]: a warp owns 32 N columns of
// one token, then the next of its share.  Picks are taken in slot order, eight
// at a time so that their loads are in flight together; the next item's picks
// are read while this one's rows are on their way, and the residual is asked
// for before them, so that a warp waits for HBM about once an item.
template <typename OT, typename YT, int N, int W>
__global__ void __launch_bounds__(256, W == N ? 3 : 2)
rows_sum_kernel(const OT* __restrict__ o, int64_t P, int T, int H, int k,
                const int32_t* __restrict__ inv, const float* __restrict__ w,
                const YT* residual, YT* y) {
    const int per = (H + 32 * N - 1) / (32 * N);        // items of a token
    const int64_t items = (int64_t)T * per, step = (int64_t)gridDim.x * 8;
    int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (item >= items) return;
    Picks picks(inv, w, item / per, k, P);
    for (;;) {
        const int64_t t = item / per;
        const int c = (int)(item - t * per) * 32 * N + (threadIdx.x & 31) * W;
        F<N> acc;
        Cols<YT, N, W> res;
#pragma unroll
        for (int i = 0; i < N; ++i) acc.v[i] = 0.0f;
        if (residual) res = ldc<YT, N, W>(residual + t * H, c, 32 * W, H);
        item += step;
        Picks after = picks;
        bool first = true;
        for (unsigned live = picks.live; live || first;) {
            Cols<OT, N, W> v[8];
            const unsigned group = live;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (live) {
                    const int64_t p = __shfl_sync(0xffffffffu, picks.row, __ffs(live) - 1);
                    live &= live - 1;
                    v[j] = ldc<OT, N, W>(o + p * H, c, 32 * W, H);
                }
            if (first && item < items) after = Picks(inv, w, item / per, k, P);
            first = false;
            unsigned m = group;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (m) {
                    const float wj = __shfl_sync(0xffffffffu, picks.w, __ffs(m) - 1);
                    m &= m - 1;
                    const F<N> f = widen<OT, N, W>(v[j]);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc.v[i] = fmaf(wj, f.v[i], acc.v[i]);
                }
        }
        if (residual) {
            const F<N> r = widen<YT, N, W>(res);
#pragma unroll
            for (int i = 0; i < N; ++i) acc.v[i] += r.v[i];
        }
        stc<YT, N, W>(y + t * H, c, 32 * W, H, narrow_cols<YT, N, W>(acc));
        if (item >= items) return;
        picks = after;
    }
}

// Gradients of the weighted sum: one warp per pick walks its row, writes w * dy
// into it and keeps the dot product of dy and o, with no barrier; the warps of a
// token's picks meet its dy in L1.
template <typename YT, typename OT, int N, int W>
__global__ void __launch_bounds__(256, W == N ? 3 : 2)
rows_sum_backward_kernel(const YT* __restrict__ dy, const OT* __restrict__ o, int64_t P, int H,
                         int k, const int32_t* __restrict__ inv, const float* __restrict__ w,
                         OT* __restrict__ d_o, float* __restrict__ dw) {
    constexpr int U = 4;  // vectors of a lane in flight
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_trigger();
    pdl_wait();
    if (i >= P) return;
    const int64_t p = inv[i];
    if (p < 0 || p >= P) {
        if (dw && lane == 0) dw[i] = 0.0f;
        return;
    }
    const float wj = w ? w[i] : 1.0f;
    const YT* g_row = dy + i / k * H;
    const OT* o_row = o + p * H;
    OT* d_row = d_o + p * H;
    F<N> dot;  // a sum per element of the vector: N short chains
#pragma unroll
    for (int e = 0; e < N; ++e) dot.v[e] = 0.0f;
    for (int c0 = lane * W; c0 < H; c0 += 32 * N * U) {
        Cols<YT, N, W> g[U];
        Cols<OT, N, W> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * N;
            if (dw) v[u] = ldc<OT, N, W>(o_row, c, 32 * W, H);
            g[u] = ldc<YT, N, W>(g_row, c, 32 * W, H);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * N;
            F<N> gf = widen<YT, N, W>(g[u]);
            if (dw) {
                const F<N> f = widen<OT, N, W>(v[u]);
#pragma unroll
                for (int e = 0; e < N; ++e) dot.v[e] = fmaf(f.v[e], gf.v[e], dot.v[e]);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) gf.v[e] *= wj;
            if (d_o) stc<OT, N, W>(d_row, c, 32 * W, H, narrow_cols<OT, N, W>(gf));
        }
    }
    if (dw) {
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) sum += dot.v[e];
        sum = warp_sum(sum);
        if (lane == 0) dw[i] = sum;
    }
}

}  // namespace coli
