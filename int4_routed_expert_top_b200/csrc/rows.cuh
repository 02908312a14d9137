// rows.cuh - picks sorted by expert, tokens copied into that order and rows
// summed back to their tokens, with the gradients of both.
//
// Sort: a stable counting sort of the linear pick index i = t * k + j by its
// expert, so rows come in the order (expert, token, slot) with no atomics and
// the same result at every run.  A warp reads 32 consecutive picks, finds the
// lanes of equal expert with match.any, and keeps its own counts per expert in
// shared memory; a pick's row is the count of its expert in everything before
// it.  Up to kSortOneCta picks one CTA does it all (one launch, the case of
// decode); above, at most kSortMaxChunks CTAs count their chunk of the picks
// first and a second launch places them.
//
// The copies and sums are bound by HBM (each row of xs / o once): a thread owns
// 16 bytes of columns and walks the token's picks.
#pragma once

#include "vec.cuh"

namespace coli {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortOneCta = 4096;     // picks
constexpr int kSortMaxChunks = 128;

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
            const int t = (int)(i / k);
            if (pair_tok) pair_tok[p] = t;
            if (pair_slot) pair_slot[p] = (int)(i - (int64_t)t * k);
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

// xs[inv[t, j]] = x[t]: block = (token, run of 256 vectors)
template <typename V>
__global__ void __launch_bounds__(256)
dispatch_kernel(const V* __restrict__ x, int64_t P, int nvec, int per_row, int k,
                const int32_t* __restrict__ inv, V* __restrict__ xs) {
    const int64_t t = blockIdx.x / per_row;
    const int c = (int)(blockIdx.x - t * per_row) * 256 + threadIdx.x;
    pdl_trigger();
    pdl_wait();
    V v;
    if (c < nvec) v = x[t * nvec + c];
    const Picks picks(inv, nullptr, t, k, P);
    for (unsigned live = picks.live; live; live &= live - 1) {
        const int64_t p = __shfl_sync(0xffffffffu, picks.row, __ffs(live) - 1);
        if (c < nvec) xs[p * nvec + c] = v;
    }
}

// y[t] = residual[t] + sum_j w[t, j] o[inv[t, j]]: a thread owns N columns of
// one token.  Picks are taken in slot order, eight at a time so that their
// loads are in flight together; every warp reads the token's picks once, a lane
// each, instead of every thread all of them.  64 registers keep 1024 threads
// of an SM (128 KB of loads) busy: 4096 tokens x 8 picks of 6144 bf16 take
// KERNEL_TIME.
template <typename OT, typename YT, int N>
__global__ void __launch_bounds__(256, 3)
rows_sum_kernel(const OT* __restrict__ o, int64_t P, int H, int per_row, int k,
                const int32_t* __restrict__ inv, const float* __restrict__ w,
                const YT* residual, YT* y) {
    const int64_t t = blockIdx.x / per_row;
    const int c = ((int)(blockIdx.x - t * per_row) * 256 + threadIdx.x) * N;
    pdl_trigger();
    pdl_wait();
    const Picks picks(inv, w, t, k, P);
    const bool in = c < H;
    F<N> acc;
#pragma unroll
    for (int i = 0; i < N; ++i) acc.v[i] = 0.0f;
    unsigned live = picks.live;
    while (live) {
        Vec<OT, N> v[8];
        float wj[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            wj[j] = 0.0f;
            if (live) {
                const int at = __ffs(live) - 1;
                live &= live - 1;
                const int64_t p = __shfl_sync(0xffffffffu, picks.row, at);
                wj[j] = __shfl_sync(0xffffffffu, picks.w, at);
                if (in) v[j] = ldv<OT, N>(o + p * H + c);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) v[j].v[i] = from_f32<OT>(0.0f);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) acc.v[i] = fmaf(wj[j], to_f32(v[j].v[i]), acc.v[i]);
    }
    if (!in) return;
    if (residual) {
        const F<N> r = ldf<YT, N>(residual + t * H + c);
#pragma unroll
        for (int i = 0; i < N; ++i) acc.v[i] += r.v[i];
    }
    stf<YT, N>(y + t * H + c, acc);
}

// Gradients of the weighted sum: one CTA per token, eight picks at a time; a
// thread walks its columns of dy, writes w * dy into the picks' rows and keeps
// their dot products with o, which the CTA then sums in a fixed order.
template <typename YT, typename OT, int N>
__global__ void __launch_bounds__(256, 2)
rows_sum_backward_kernel(const YT* __restrict__ dy, const OT* __restrict__ o, int64_t P, int H,
                         int k, const int32_t* __restrict__ inv, const float* __restrict__ w,
                         OT* __restrict__ d_o, float* __restrict__ dw) {
    __shared__ float part[8][8];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const Picks picks(inv, w, t, k, P);
    if (dw && threadIdx.x < 32 && lane < k && !(picks.live >> lane & 1)) dw[t * k + lane] = 0.0f;
    for (unsigned live = picks.live, next; live; live = next) {
        float dot[8];
        int n = 0;
        next = live;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dot[j] = 0.0f;
            if (next) { next &= next - 1; ++n; }
        }
        for (int c0 = 0; c0 < H; c0 += 256 * N) {
            const int c = c0 + (int)threadIdx.x * N;
            const bool in = c < H;
            F<N> g;
            if (in) g = ldf<YT, N>(dy + t * H + c);
            Vec<OT, N> v[8];
            if (dw) {
                unsigned m = live;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j >= n) break;
                    const int64_t p = __shfl_sync(0xffffffffu, picks.row, __ffs(m) - 1);
                    m &= m - 1;
                    if (in) v[j] = ldv<OT, N>(o + p * H + c);
                }
            }
            unsigned m = live;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= n) break;
                const int at = __ffs(m) - 1;
                m &= m - 1;
                const int64_t p = __shfl_sync(0xffffffffu, picks.row, at);
                const float wj = __shfl_sync(0xffffffffu, picks.w, at);
                if (!in) continue;
                F<N> out;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (dw) dot[j] = fmaf(to_f32(v[j].v[i]), g.v[i], dot[j]);
                    out.v[i] = wj * g.v[i];
                }
                if (d_o) stf<OT, N>(d_o + p * H + c, out);
            }
        }
        if (!dw) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = warp_sum(dot[j]);
            if (lane == 0) part[j][warp] = s;
        }
        __syncthreads();
        if (threadIdx.x < n) {
            unsigned m = live;
            for (int j = 0; j < (int)threadIdx.x; ++j) m &= m - 1;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += part[threadIdx.x][i];
            dw[t * k + __ffs(m) - 1] = s;
        }
        __syncthreads();
    }
}

}  // namespace coli
