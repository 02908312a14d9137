// norm.cuh - the step from one block to the next on a residual stream, and its
// gradient:
//   u = o r_o post_gain, r_o = 1 / sqrt(mean(o^2) + eps)   (or u = o)
//   x' = x + alpha gate u
//   n = x' r_x pre_gain, r_x = 1 / sqrt(mean(x'^2) + eps)
// Bound by HBM: x and o read once, x' and n written once.  One CTA owns a row
// and keeps it in registers between the two sums over the row, so nothing is
// read twice.  Rows are cut into vectors of four elements (single elements
// where H or a pointer allows no more), N of them per thread.
//
// Backward, with xh = x' r_x, oh = o r_o, v = pre_gain dn, <.> the mean over H:
//   d  = dx' + r_x (v - xh <v xh>)          dx = d, dpre_gain = sum_t dn xh
//   e  = alpha gate d                       dgate = alpha u d (summed over what it is shared by)
//   do = r_o (q - oh <q oh>), q = post_gain e    dpost_gain = sum_t e oh
// The sums over tokens stay in registers (a thread owns its columns for all
// rows of its CTA); each CTA then writes one partial row and a second kernel
// adds those in a fixed order, so the result does not change between runs.
#pragma once

#include "vec.cuh"

namespace coli {

constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxH = 16384;
constexpr float kNoGate = 1.0f;

struct NormArgs {
    int H, T;
    int post_norm, gate_kind;   // coli_gate
    float alpha, eps;
    const float* post_gain;
    const float* pre_gain;
    const float* gate;
};

template <int V> struct F { float v[V]; };

template <typename T, int V>
__device__ __forceinline__ F<V> load_f32(const T* p, int64_t i) {
    const Vec<T, V> a = *reinterpret_cast<const Vec<T, V>*>(p + i);
    F<V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r.v[j] = to_f32(a.v[j]);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_f32(T* p, int64_t i, const F<V>& a) {
    Vec<T, V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r.v[j] = from_f32<T>(a.v[j]);
    *reinterpret_cast<Vec<T, V>*>(p + i) = r;
}
template <int V>
__device__ __forceinline__ F<V> gain_at(const float* g, int c) {
    if (g) return load_f32<float, V>(g, c);
    F<V> r;
#pragma unroll
    for (int j = 0; j < V; ++j) r.v[j] = 1.0f;
    return r;
}

// Sums of K values over the CTA, the same in every thread; part holds K * 32
// floats and is free again after the call (two buffers alternate).
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

// gate of token t, columns c .. c + V - 1
template <int V>
__device__ __forceinline__ F<V> gate_at(const NormArgs& a, int64_t t, int c) {
    F<V> r;
    if (a.gate_kind == 1) return load_f32<float, V>(a.gate, c);
    if (a.gate_kind == 3) return load_f32<float, V>(a.gate, t * a.H + c);
    const float g = a.gate_kind == 2 ? a.gate[t] : kNoGate;
#pragma unroll
    for (int j = 0; j < V; ++j) r.v[j] = g;
    return r;
}

template <typename XT, typename BT, int V, int N>
__global__ void __launch_bounds__(kNormMaxThreads)
block_norm_kernel(NormArgs a, const XT* x, const BT* o, XT* x_out, BT* n_out, float* rstd_post,
                  float* rstd_pre) {
    __shared__ float part[2][32];
    const int64_t t = blockIdx.x;
    const int64_t row = t * a.H;
    pdl_trigger();
    pdl_wait();
    F<V> xv[N], ov[N];
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c >= a.H) continue;
        xv[i] = load_f32<XT, V>(x, row + c);
        if (!o) continue;
        ov[i] = load_f32<BT, V>(o, row + c);
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] = fmaf(ov[i].v[j], ov[i].v[j], s[0]);
    }
    if (o) {
        float r = 1.0f;
        if (a.post_norm) {
            cta_sum(s, part[0]);
            r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
            if (rstd_post && threadIdx.x == 0) rstd_post[t] = r;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c >= a.H) continue;
            const F<V> g = gate_at<V>(a, t, c);
            F<V> pg;
            if (a.post_norm) pg = gain_at<V>(a.post_gain, c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = a.post_norm ? ov[i].v[j] * r * pg.v[j] : ov[i].v[j];
                // the stored value, which the norm below reads
                xv[i].v[j] = to_f32(from_f32<XT>(fmaf(a.alpha * g.v[j], u, xv[i].v[j])));
            }
            store_f32<XT, V>(x_out, row + c, xv[i]);
        }
    }
    if (!n_out) return;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c >= a.H) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] = fmaf(xv[i].v[j], xv[i].v[j], s[0]);
    }
    cta_sum(s, part[1]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
    if (rstd_pre && threadIdx.x == 0) rstd_pre[t] = r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c >= a.H) continue;
        const F<V> pg = gain_at<V>(a.pre_gain, c);
        F<V> n;
#pragma unroll
        for (int j = 0; j < V; ++j) n.v[j] = xv[i].v[j] * r * pg.v[j];
        store_f32<BT, V>(n_out, row + c, n);
    }
}

// partial [gridDim.x][3][H]: this CTA's sums for dpost_gain, dgate (channel
// gates) and dpre_gain
template <typename XT, typename BT, int V, int N>
__global__ void __launch_bounds__(kNormMaxThreads)
block_norm_backward_kernel(NormArgs a, const XT* x_out, const BT* o, const float* rstd_post,
                           const float* rstd_pre, const XT* dx_out, const BT* dn, XT* dx, BT* d_o,
                           float* dgate, float* partial) {
    __shared__ float part[2][64];
    pdl_trigger();
    pdl_wait();
    F<V> s_post[N], s_gate[N], s_pre[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s_post[i].v[j] = s_gate[i].v[j] = s_pre[i].v[j] = 0.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.H;
        F<V> d[N], xh[N], ov[N];
        float s1[1] = {0.0f};
        const float rx = dn ? rstd_pre[t] : 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c >= a.H) continue;
            if (o) ov[i] = load_f32<BT, V>(o, row + c);
            if (dx_out) {
                d[i] = load_f32<XT, V>(dx_out, row + c);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) d[i].v[j] = 0.0f;
            }
            if (dn) {
                xh[i] = load_f32<XT, V>(x_out, row + c);
                const F<V> g = load_f32<BT, V>(dn, row + c);
                const F<V> pg = gain_at<V>(a.pre_gain, c);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xh[i].v[j] *= rx;
                    s_pre[i].v[j] = fmaf(g.v[j], xh[i].v[j], s_pre[i].v[j]);
                    const float v = g.v[j] * pg.v[j];
                    s1[0] = fmaf(v, xh[i].v[j], s1[0]);
                    d[i].v[j] = fmaf(rx, v, d[i].v[j]);
                }
            }
        }
        if (dn) {
            cta_sum(s1, part[0]);
            const float m = rx * (s1[0] / (float)a.H);
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
                    if (c < a.H) d[i].v[j] = fmaf(-m, xh[i].v[j], d[i].v[j]);
                }
        }
        const float ro = o && a.post_norm ? rstd_post[t] : 1.0f;
        float s2[2] = {0.0f, 0.0f};  // q oh, alpha u d (token gates)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
            if (c >= a.H) continue;
            store_f32<XT, V>(dx, row + c, d[i]);
            if (!o) continue;
            const F<V> g = gate_at<V>(a, t, c);
            F<V> pg, dg;
            if (a.post_norm) pg = gain_at<V>(a.post_gain, c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                ov[i].v[j] *= ro;
                const float p = a.post_norm ? pg.v[j] : 1.0f;
                const float ad = a.alpha * d[i].v[j];
                dg.v[j] = ad * (ov[i].v[j] * p);
                s_gate[i].v[j] += dg.v[j];
                s2[1] += dg.v[j];
                const float e = ad * g.v[j];
                s_post[i].v[j] = fmaf(e, ov[i].v[j], s_post[i].v[j]);
                d[i].v[j] = e * p;  // q
                s2[0] = fmaf(d[i].v[j], ov[i].v[j], s2[0]);
            }
            if (dgate && a.gate_kind == 3) store_f32<float, V>(dgate, row + c, dg);
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
                const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
                if (c >= a.H) continue;
                F<V> r;
#pragma unroll
                for (int j = 0; j < V; ++j) r.v[j] = ro * fmaf(-m, ov[i].v[j], d[i].v[j]);
                store_f32<BT, V>(d_o, row + c, r);
            }
        }
        __syncthreads();  // part is free for the next row
    }
    if (!partial) return;
    float* mine = partial + (int64_t)blockIdx.x * 3 * a.H;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c >= a.H) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mine[c + j] = s_post[i].v[j];
            mine[a.H + c + j] = s_gate[i].v[j];
            mine[2 * a.H + c + j] = s_pre[i].v[j];
        }
    }
}

// out[c] = sum over the CTAs' partial rows, 32 columns by 8 runs of rows per
// CTA; blockIdx.y picks the sum (0 dpost_gain, 1 dgate, 2 dpre_gain)
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float* __restrict__ partial, int rows, int H, float* dpost, float* dgate,
                   float* dpre) {
    __shared__ float part[8][32];
    float* out = blockIdx.y == 0 ? dpost : blockIdx.y == 1 ? dgate : dpre;
    pdl_trigger();
    pdl_wait();
    if (!out) return;
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < H)
        for (int r = run; r < rows; r += 8) s += partial[((int64_t)r * 3 + blockIdx.y) * H + c];
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][lane];
        out[c] = s;
    }
}

}  // namespace coli
