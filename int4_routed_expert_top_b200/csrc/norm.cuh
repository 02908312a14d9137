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
// The sums over tokens stay with the thread that owns the columns, for all rows
// of its CTA; the CTAs of a cluster then add theirs through distributed shared
// memory, write one partial row, and a second kernel adds those: always in the
// same order, so the result does not change between runs.
// A row's four inputs and two barriers leave an SM waiting for HBM most of the
// time if it only loads a row when it gets to it (4096 x 6144, f32 stream, bf16
// blocks: 185 us, 0.37 of the HBM rate).  With many tokens the rows therefore
// come through a ring in shared memory: one thread issues the bulk copies of the
// rows ahead, one CTA per SM (RING_TIME).  The sums are then in registers.  Rows
// that leave no room for two stages, or few tokens, take the loads as they come.
#pragma once

#include "pipeline.cuh"
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
__device__ __forceinline__ void sum_add(float* sums, int c, int H, const F<V>& f, const F<V>& g) {
    if constexpr (V == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float4* p = reinterpret_cast<float4*>(sums + sum_at<V>(c + 4 * h, H));
            float4 v = *p;
            v.x = fmaf(f.v[4 * h], g.v[4 * h], v.x);
            v.y = fmaf(f.v[4 * h + 1], g.v[4 * h + 1], v.y);
            v.z = fmaf(f.v[4 * h + 2], g.v[4 * h + 2], v.z);
            v.w = fmaf(f.v[4 * h + 3], g.v[4 * h + 3], v.w);
            *p = v;
        }
    } else {
        sums[c] = fmaf(f.v[0], g.v[0], sums[c]);
    }
}

// Where each sum lives among the kept ones, -1 for one that is not asked for.
struct NormSums {
    int at[kNormSums];
    int n;
};

// Shared memory of the ring form: the vectors of H that every row needs
// (pre_gain, post_gain, a channel gate: in sum_at's order), then the stages, each
// with the rows x_out, dx_out, o, dn one after the other.  What a call does not
// have is not there.
struct NormRing {
    int stages;
    int stage;          // bytes, a multiple of 16
    int off[4];         // of a row in its stage, -1: absent
    int gain[3];        // of a vector, -1: absent
    int first;          // of the first stage
};
constexpr int kNormMaxStages = 4;

// N elements of a row in shared memory (V = 8) as they lie there
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> lds_row(const uint8_t* row, int c) {
    Vec<T, V> r;
    static_assert(r.bytes >= 16, "vectors of eight");
#pragma unroll
    for (int i = 0; i < r.bytes / 16; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + c * (int)sizeof(T) + 16 * i);
        r.u[4 * i] = v.x; r.u[4 * i + 1] = v.y; r.u[4 * i + 2] = v.z; r.u[4 * i + 3] = v.w;
    }
    return r;
}

// V elements from column c of a vector kept in sum_at's order, 1 where there is none
template <int V>
__device__ __forceinline__ F<V> lds_gain(const uint8_t* smem, int off, int c, int H) {
    F<V> r = ones<V>();
    if (off >= 0) {
        const float* p = reinterpret_cast<const float*>(smem + off);
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const float4 v = *reinterpret_cast<const float4*>(p + sum_at<V>(c + 4 * h, H));
            r.v[4 * h] = v.x; r.v[4 * h + 1] = v.y; r.v[4 * h + 2] = v.z; r.v[4 * h + 3] = v.w;
        }
    }
    return r;
}

// partial [clusters][sums.n][H]
template <typename XT, typename BT, int V, int N, bool RING>
__global__ void __launch_bounds__(RING && N == 1 ? 768 : 512)
block_norm_backward_kernel(NormArgs a, NormSums keep, NormRing ring, const XT* x_out, const BT* o,
                           const float* rstd_post, const float* rstd_pre, const XT* dx_out, const BT* dn, XT* dx,
                           BT* d_o, float* dgate, float* partial) {
    extern __shared__ __align__(128) uint8_t nb_smem[];   // the ring, or the sums; at the end the sums
    __shared__ float part[2][64];
    __shared__ __align__(8) uint64_t full[kNormMaxStages];
    float* sums = reinterpret_cast<float*>(nb_smem);
    const int step = (int)blockDim.x * V, c0 = (int)threadIdx.x * V;
    float* s_of[kNormSums];
#pragma unroll
    for (int i = 0; i < kNormSums; ++i) s_of[i] = keep.at[i] >= 0 ? sums + keep.at[i] * a.H : nullptr;
    F<V> acc[RING ? kNormSums : 1][RING ? N : 1];
    if (RING) {
#pragma unroll
        for (int k = 0; k < kNormSums; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) acc[RING ? k : 0][RING ? i : 0].v[j] = 0.0f;
        if (threadIdx.x == 0) {
            for (int i = 0; i < ring.stages; ++i) mbar_init(&full[i], 1);
            fence_mbar_init();
        }
    } else {
        for (int i = threadIdx.x; i < keep.n * a.H; i += blockDim.x) sums[i] = 0.0f;
    }
    __syncthreads();
    // sum k += f * h
    const auto add = [&](int k, int i, int c, const F<V>& f, const F<V>& h) {
        if (!s_of[k]) return;
        if (RING) {
            F<V>& s = acc[RING ? k : 0][RING ? i : 0];
#pragma unroll
            for (int j = 0; j < V; ++j) s.v[j] = fmaf(f.v[j], h.v[j], s.v[j]);
        } else {
            sum_add<V>(s_of[k], c, a.H, f, h);
        }
    };
    const float inv_h = 1.0f / (float)a.H;
    // row t into stage `at` (one thread)
    const auto fetch = [&](int64_t t, int at) {
        if (t >= a.T) return;
        uint8_t* st = nb_smem + ring.first + at * ring.stage;
        const uint32_t xb = a.H * (uint32_t)sizeof(XT), bb = a.H * (uint32_t)sizeof(BT);
        mbar_expect_tx(&full[at], (ring.off[0] >= 0 ? xb : 0) + (ring.off[1] >= 0 ? xb : 0) +
                                      (ring.off[2] >= 0 ? bb : 0) + (ring.off[3] >= 0 ? bb : 0));
        if (ring.off[0] >= 0) bulk_g2s(st + ring.off[0], x_out + t * a.H, xb, &full[at]);
        if (ring.off[1] >= 0) bulk_g2s(st + ring.off[1], dx_out + t * a.H, xb, &full[at]);
        if (ring.off[2] >= 0) bulk_g2s(st + ring.off[2], o + t * a.H, bb, &full[at]);
        if (ring.off[3] >= 0) bulk_g2s(st + ring.off[3], dn + t * a.H, bb, &full[at]);
    };
    pdl_trigger();
    pdl_wait();
    float rx = 0.0f, ro = 1.0f;  // of the next row
    const auto rstd = [&](int64_t t) {
        if (t >= a.T) return;
        if (dn) rx = rstd_pre[t];
        if (o && a.post_norm) ro = rstd_post[t];
    };
    if (RING) {
        if (threadIdx.x == 0)
            for (int i = 0; i < ring.stages; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
        const float* from[3] = {a.pre_gain, a.post_gain, a.gate};
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (ring.gain[k] >= 0)
                for (int c = threadIdx.x; c < a.H; c += blockDim.x)
                    reinterpret_cast<float*>(nb_smem + ring.gain[k])[sum_at<V>(c, a.H)] = from[k][c];
        __syncthreads();
    }
    rstd(blockIdx.x);
    int at = 0;
    uint32_t phase = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t row = t * a.H;
        F<V> d[N];
        Vec<XT, V> xv[N];
        Vec<BT, V> ov[N], gv[N];
        float s1[1] = {0.0f};
        const float rx_t = rx, ro_t = ro;
        rstd(t + gridDim.x);
        const uint8_t* st = nb_smem + ring.first + at * ring.stage;
        // a copy that never lands (a wait of seconds) makes the row NaN
        bool landed = true;
        if (RING) landed = mbar_wait(&full[at], phase, nullptr);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = c0 + i * step;
            if (c >= a.H) continue;
            if constexpr (RING) {
                if (dn) {
                    xv[i] = lds_row<XT, V>(st + ring.off[0], c);
                    gv[i] = lds_row<BT, V>(st + ring.off[3], c);
                }
                if (dx_out) d[i] = widen<XT, V>(lds_row<XT, V>(st + ring.off[1], c));
                if (o) ov[i] = lds_row<BT, V>(st + ring.off[2], c);
            } else {
                if (dn) {
                    xv[i] = ldv<XT, V>(x_out + row + c);
                    gv[i] = ldv<BT, V>(dn + row + c);
                }
                if (dx_out) d[i] = ldf<XT, V>(dx_out + row + c);
                if (o) ov[i] = ldv<BT, V>(o + row + c);
            }
            if (!dx_out) {
#pragma unroll
                for (int j = 0; j < V; ++j) d[i].v[j] = 0.0f;
            }
            if (!landed) d[i].v[0] = __uint_as_float(0x7fc00000u);
        }
        if (dn) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * step;
                if (c >= a.H) continue;
                F<V> pg;
                if constexpr (RING) pg = lds_gain<V>(nb_smem, ring.gain[0], c, a.H);
                else pg = gain_at<V>(a.pre_gain, c);
                const F<V> xf = widen<XT, V>(xv[i]), gf = widen<BT, V>(gv[i]);
                F<V> xh;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xh.v[j] = xf.v[j] * rx_t;
                    const float v = gf.v[j] * pg.v[j];
                    s1[0] = fmaf(v, xh.v[j], s1[0]);
                    d[i].v[j] = fmaf(rx_t, v, d[i].v[j]);
                }
                add(2, i, c, gf, xh);
            }
            cta_sum(s1, part[0]);
        } else if (RING) {
            __syncthreads();
        }
        // every thread has its part of the row: the stage takes the row that comes next in it
        if (RING) {
            if (threadIdx.x == 0) fetch(t + (int64_t)ring.stages * gridDim.x, at);
            if (++at == ring.stages) {
                at = 0;
                phase ^= 1;
            }
        }
        if (dn) {
            const float m = -rx_t * rx_t * (s1[0] * inv_h);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (c0 + i * step >= a.H) continue;
                const F<V> xf = widen<XT, V>(xv[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) d[i].v[j] = fmaf(m, xf.v[j], d[i].v[j]);
            }
        }
        float s2[2] = {0.0f, 0.0f};  // q oh, u d
        const bool token = dgate && a.gate_kind == 2;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = c0 + i * step;
            if (c >= a.H) continue;
            stf<XT, V>(dx + row + c, d[i]);
            if (!o) continue;
            F<V> g, pg;
            if (RING && ring.gain[2] >= 0) g = lds_gain<V>(nb_smem, ring.gain[2], c, a.H);
            else g = gate_at<V>(a, t, c);
            if constexpr (RING) pg = lds_gain<V>(nb_smem, ring.gain[1], c, a.H);
            else pg = a.post_norm ? gain_at<V>(a.post_gain, c) : ones<V>();
            F<V> oh = widen<BT, V>(ov[i]), u, e;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                oh.v[j] *= ro_t;
                u.v[j] = oh.v[j] * pg.v[j];
                e.v[j] = d[i].v[j] * (a.alpha * g.v[j]);
            }
            if (token) {
#pragma unroll
                for (int j = 0; j < V; ++j) s2[1] = fmaf(u.v[j], d[i].v[j], s2[1]);
            }
            add(1, i, c, u, d[i]);  // times alpha at the end
            add(0, i, c, e, oh);
            if (dgate && a.gate_kind == 3) {
                F<V> dg;
#pragma unroll
                for (int j = 0; j < V; ++j) dg.v[j] = a.alpha * (u.v[j] * d[i].v[j]);
                stf<float, V>(dgate + row + c, dg);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s2[0] = fmaf(e.v[j], u.v[j], s2[0]);
                d[i].v[j] = e.v[j] * pg.v[j];  // q
            }
        }
        if (o) {
            float m = 0.0f;
            if (a.post_norm || token) {
                cta_sum(s2, part[1]);
                if (token && threadIdx.x == 0) dgate[t] = a.alpha * s2[1];
                if (a.post_norm) m = -ro_t * (s2[0] * inv_h);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * step;
                if (c >= a.H) continue;
                F<V> r = widen<BT, V>(ov[i]);
#pragma unroll
                for (int j = 0; j < V; ++j) r.v[j] = ro_t * fmaf(m, r.v[j], d[i].v[j]);
                stf<BT, V>(d_o + row + c, r);
            }
        }
        __syncthreads();  // part is free for the next row
    }
    if (keep.n == 0) return;
    if (RING) {  // every row has been read: the ring's memory takes the sums
#pragma unroll
        for (int k = 0; k < kNormSums; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = c0 + i * step;
                if (!s_of[k] || c >= a.H) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) s_of[k][sum_at<V>(c + j, a.H)] = acc[RING ? k : 0][RING ? i : 0].v[j];
            }
    }
    cluster_sync();
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    float* mine = partial + (int64_t)(blockIdx.x / cs) * keep.n * a.H;
    for (int i = rank * (int)blockDim.x + (int)threadIdx.x; i < keep.n * a.H; i += cs * (int)blockDim.x) {
        const int k = i / a.H, c = i - k * a.H;
        const float* p = sums + k * a.H + sum_at<V>(c, a.H);
        float s = 0.0f;
        for (int q = 0; q < cs; ++q) s += ld_cluster(p, q);
        mine[i] = k == keep.at[1] ? a.alpha * s : s;  // dgate
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
