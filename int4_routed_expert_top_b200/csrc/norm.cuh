// norm.cuh - the step from one block to the next on a residual stream, and its
// gradient:
//   u = o r_o post_gain, r_o = 1 / sqrt(mean(o^2) + eps)   (or u = o)
//   x' = x + alpha gate u
//   n = x' r_x pre_gain, r_x = 1 / sqrt(mean(x'^2) + eps)
// Bound by HBM: x and o read once, x' and n written once.  One CTA owns a row
// and keeps it in registers, in the types it was read in, between the two sums
// over the row, so nothing is read twice; 64 registers a thread let an SM hold
// several rows (over 100 KB of loads) while others wait at their sums.  Rows are
// cut into vectors of eight elements (single elements where H or a pointer
// allows no more), N of them per thread; few tokens take N = 1, which spreads a
// row over more threads and asks for the gains before the first sum.
//
// Backward, with xh = x' r_x, oh = o r_o, v = pre_gain dn, <.> the mean over H:
//   d  = dx' + r_x (v - xh <v xh>)          dx = d, dpre_gain = sum_t dn xh
//   e  = alpha gate d                       dgate = alpha u d (summed over what it is shared by)
//   do = r_o (q - oh <q oh>), q = post_gain e    dpost_gain = sum_t e oh
// The sums over tokens stay in shared memory (a thread owns its columns for all
// rows of its CTA); the CTAs of a cluster add theirs through distributed shared
// memory, write one partial row, and a second kernel adds those: always in the
// same order, so the result does not change between runs.
#pragma once

#include "vec.cuh"

namespace coli {

constexpr int kNormMaxH = 16384;
constexpr int kNormSums = 3;  // dpost_gain, dgate (channel gates), dpre_gain

struct NormArgs {
    int H, T;
    int post_norm, gate_kind;   // coli_gate
    float alpha, eps;
    const float* post_gain;
    const float* pre_gain;
    const float* gate;
};

template <int V>
__device__ __forceinline__ F<V> ones() {
    F<V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r.v[j] = 1.0f;
    return r;
}
template <int V>
__device__ __forceinline__ F<V> gain_at(const float* g, int c) {
    return g ? ldf<float, V>(g + c) : ones<V>();
}

// gate of token t, columns c .. c + V - 1
template <int V>
__device__ __forceinline__ F<V> gate_at(const NormArgs& a, int64_t t, int c) {
    if (a.gate_kind == 1) return ldf<float, V>(a.gate + c);
    if (a.gate_kind == 3) return ldf<float, V>(a.gate + t * a.H + c);
    F<V> r = ones<V>();
    if (a.gate_kind == 2) {
        const float g = a.gate[t];
#pragma unroll
        for (int j = 0; j < V; ++j) r.v[j] = g;
    }
    return r;
}

// Sums of K values over the CTA, the same in every thread; part holds K * 32
// floats and may be written again after the CTA's next barrier.
template <int K>
__device__ __forceinline__ void cta_sum(float (&s)[K], float* part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        s[i] = warp_sum(s[i]);
        if (lane == 0) part[i * 32 + warp] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] = warp_sum(lane < warps ? part[i * 32 + lane] : 0.0f);
}

constexpr int norm_max_threads(int N) { return N == 1 ? 1024 : 512; }

template <typename XT, typename BT, int V, int N>
__global__ void __launch_bounds__(norm_max_threads(N), N == 2 || N == 3 ? 2 : 1)
block_norm_kernel(NormArgs a, const XT* x, const BT* o, XT* x_out, BT* n_out, float* rstd_post,
                  float* rstd_pre) {
    __shared__ float part[2][32];
    const int64_t t = blockIdx.x;
    const int64_t row = t * a.H;
    const int step = (int)blockDim.x * V, c0 = (int)threadIdx.x * V;
    pdl_trigger();
    pdl_wait();
    Vec<XT, V> xv[N];
    Vec<BT, V> ov[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = c0 + i * step;
        if (c >= a.H) continue;
        if (o) ov[i] = ldv<BT, V>(o + row + c);
        xv[i] = ldv<XT, V>(x + row + c);
    }
    F<V> early_post, early_gate, early_pre;  // N == 1: asked for before the sums
    if (N == 1 && c0 < a.H) {
        if (o) {
            early_gate = gate_at<V>(a, t, c0);
            if (a.post_norm) early_post = gain_at<V>(a.post_gain, c0);
        }
        if (n_out) early_pre = gain_at<V>(a.pre_gain, c0);
    }
    float s[1] = {0.0f};
    if (o) {
        float r = 1.0f;
        if (a.post_norm) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (c0 + i * step >= a.H) continue;
                const F<V> f = widen<BT, V>(ov[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] = fmaf(f.v[j], f.v[j], s[0]);
            }
            cta_sum(s, part[0]);
            r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
            if (rstd_post && threadIdx.x == 0) rstd_post[t] = r;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = c0 + i * step;
            if (c >= a.H) continue;
            const F<V> g = N == 1 ? early_gate : gate_at<V>(a, t, c);
            F<V> f = widen<BT, V>(ov[i]);
            if (a.post_norm) {
                const F<V> pg = N == 1 ? early_post : gain_at<V>(a.post_gain, c);
#pragma unroll
                for (int j = 0; j < V; ++j) f.v[j] = f.v[j] * r * pg.v[j];
            }
            const F<V> xf = widen<XT, V>(xv[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) f.v[j] = fmaf(a.alpha * g.v[j], f.v[j], xf.v[j]);
            xv[i] = narrow<XT, V>(f);  // the stored value, which the norm below reads
            stv<XT, V>(x_out + row + c, xv[i]);
        }
    }
    if (!n_out) return;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (c0 + i * step >= a.H) continue;
        const F<V> f = widen<XT, V>(xv[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] = fmaf(f.v[j], f.v[j], s[0]);
    }
    cta_sum(s, part[1]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
    if (rstd_pre && threadIdx.x == 0) rstd_pre[t] = r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = c0 + i * step;
        if (c >= a.H) continue;
        const F<V> pg = N == 1 ? early_pre : gain_at<V>(a.pre_gain, c);
        F<V> f = widen<XT, V>(xv[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) f.v[j] = f.v[j] * r * pg.v[j];
        stf<BT, V>(n_out + row + c, f);
    }
}

// Sums of this CTA in shared memory, kept so that a warp's 16-byte accesses meet
// no bank twice: for vectors of eight, the first four elements of all vectors,
// then the last four.
template <int V>
__device__ __forceinline__ int sum_at(int c, int H) {  // column c of one sum
    return V == 8 ? (((c >> 2) & 1) * (H >> 3) + (c >> 3)) * 4 + (c & 3) : c;
}
template <int V>
__device__ __forceinline__ void sum_add(float* sums, int c, int H, const F<V>& f) {
    if constexpr (V == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4* p = reinterpret_cast<float4*>(sums + sum_at<V>(c + 4 * h, H));
            float4 v = *p;
            v.x += f.v[4 * h]; v.y += f.v[4 * h + 1]; v.z += f.v[4 * h + 2]; v.w += f.v[4 * h + 3];
            *p = v;
        }
    } else {
        sums[c] += f.v[0];
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
    uint32_t addr = (uint32_t)__cvta_generic_to_shared(p);
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Where each sum lives among the kept ones, -1 for one that is not asked for.
struct NormSums {
    int at[kNormSums];
    int n;
};

// partial [clusters][sums.n][H]
template <typename XT, typename BT, int V, int N>
__global__ void __launch_bounds__(512)
block_norm_backward_kernel(NormArgs a, NormSums keep, const XT* x_out, const BT* o, const float* rstd_post,
                           const float* rstd_pre, const XT* dx_out, const BT* dn, XT* dx, BT* d_o,
                           float* dgate, float* partial) {
    extern __shared__ __align__(16) float nb_sums[];
    __shared__ float part[2][64];
    const int step = (int)blockDim.x * V, c0 = (int)threadIdx.x * V;
    for (int i = threadIdx.x; i < keep.n * a.H; i += blockDim.x) nb_sums[i] = 0.0f;
    __syncthreads();
    float* s_post = keep.at[0] >= 0 ? nb_sums + keep.at[0] * a.H : nullptr;
    float* s_gate = keep.at[1] >= 0 ? nb_sums + keep.at[1] * a.H : nullptr;
    float* s_pre = keep.at[2] >= 0 ? nb_sums + keep.at[2] * a.H : nullptr;
    pdl_trigger();
    pdl_wait();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.H;
        F<V> d[N];
        Vec<XT, V> xv[N];
        Vec<BT, V> ov[N], gv[N];
        float s1[1] = {0.0f};
        const float rx = dn ? rstd_pre[t] : 0.0f;
        const float ro = o && a.post_norm ? rstd_post[t] : 1.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = c0 + i * step;
            if (c >= a.H) continue;
            if (dn) {
                xv[i] = ldv<XT, V>(x_out + row + c);
                gv[i] = ldv<BT, V>(dn + row + c);
            }
            if (dx_out) {
                d[i] = ldf<XT, V>(dx_out + row + c);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) d[i].v[j] = 0.0f;
            }
            if (o) ov[i] = ldv<BT, V>(o + row + c);
        }
        if (dn) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * step;
                if (c >= a.H) continue;
                const F<V> pg = gain_at<V>(a.pre_gain, c);
                const F<V> xf = widen<XT, V>(xv[i]), gf = widen<BT, V>(gv[i]);
                F<V> p;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = xf.v[j] * rx;
                    p.v[j] = gf.v[j] * xh;
                    const float v = gf.v[j] * pg.v[j];
                    s1[0] = fmaf(v, xh, s1[0]);
                    d[i].v[j] = fmaf(rx, v, d[i].v[j]);
                }
                if (s_pre) sum_add<V>(s_pre, c, a.H, p);
            }
            cta_sum(s1, part[0]);
            const float m = rx * (s1[0] / (float)a.H);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (c0 + i * step >= a.H) continue;
                const F<V> xf = widen<XT, V>(xv[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) d[i].v[j] = fmaf(-m, xf.v[j] * rx, d[i].v[j]);
            }
        }
        float s2[2] = {0.0f, 0.0f};  // q oh, alpha u d (token gates)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = c0 + i * step;
            if (c >= a.H) continue;
            stf<XT, V>(dx + row + c, d[i]);
            if (!o) continue;
            const F<V> g = gate_at<V>(a, t, c);
            const F<V> pg = a.post_norm ? gain_at<V>(a.post_gain, c) : ones<V>();
            const F<V> of = widen<BT, V>(ov[i]);
            F<V> dg, dp;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float oh = of.v[j] * ro;
                const float ad = a.alpha * d[i].v[j];
                dg.v[j] = ad * (oh * pg.v[j]);
                s2[1] += dg.v[j];
                const float e = ad * g.v[j];
                dp.v[j] = e * oh;
                d[i].v[j] = e * pg.v[j];  // q
                s2[0] = fmaf(d[i].v[j], oh, s2[0]);
            }
            if (s_gate) sum_add<V>(s_gate, c, a.H, dg);
            if (s_post) sum_add<V>(s_post, c, a.H, dp);
            if (dgate && a.gate_kind == 3) stf<float, V>(dgate + row + c, dg);
        }
        if (o) {
            const bool token = dgate && a.gate_kind == 2;
            float m = 0.0f;
            if (a.post_norm || token) {
                cta_sum(s2, part[1]);
                if (token && threadIdx.x == 0) dgate[t] = s2[1];
                if (a.post_norm) m = s2[0] / (float)a.H;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * step;
                if (c >= a.H) continue;
                F<V> r = widen<BT, V>(ov[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) r.v[j] = ro * fmaf(-m, r.v[j] * ro, d[i].v[j]);
                stf<BT, V>(d_o + row + c, r);
            }
        }
        __syncthreads();  // part is free for the next row
    }
    if (keep.n == 0) return;
    cluster_sync();
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    float* mine = partial + (int64_t)(blockIdx.x / cs) * keep.n * a.H;
    for (int i = rank * (int)blockDim.x + (int)threadIdx.x; i < keep.n * a.H; i += cs * (int)blockDim.x) {
        const int k = i / a.H, c = i - k * a.H;
        const float* p = nb_sums + k * a.H + sum_at<V>(c, a.H);
        float s = 0.0f;
        for (int q = 0; q < cs; ++q) s += ld_cluster(p, q);
        mine[i] = s;
    }
    cluster_sync();  // no CTA leaves while another reads its sums
}

// out[c] = sum over the partial rows, 32 columns by 8 runs of rows per CTA;
// blockIdx.y picks the sum
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float* __restrict__ partial, int rows, int H, NormSums keep, float* dpost, float* dgate,
                   float* dpre) {
    __shared__ float part[8][32];
    float* out = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dgate : dpre;
    const int k = keep.at[blockIdx.y];
    pdl_trigger();
    pdl_wait();
    if (k < 0) return;
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < H)
#pragma unroll 4
        for (int r = run; r < rows; r += 8) s += partial[((int64_t)r * keep.n + k) * H + c];
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        out[c] = s;
    }
}

}  // namespace coli
