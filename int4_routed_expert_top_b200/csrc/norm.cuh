// norm.cuh - the step from one block to the next on a residual stream, and its
// gradient:
//   u = o r_o post_gain, r_o = 1 / sqrt(mean(o^2) + eps)   (or u = o)
//   x' = x + alpha gate u
//   n = x' r_x pre_gain, r_x = 1 / sqrt(mean(x'^2) + eps)
// Bound by HBM: x and o read once, x' and n written once.  One CTA owns a row
// and keeps it in registers, in the types it was read in, between the two sums
// over the row, so nothing is read twice; 64 registers a thread let an SM hold
// several rows (over 100 KB of loads) while others wait at their sums.  Rows are
// cut into vectors of eight elements (chunks of W = 2 or 1 neighbours where H or a
// pointer allows no more, see Cols), N of them per thread; few tokens take N = 1, which spreads a
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
// A row's four inputs and its barriers leave an SM waiting for HBM most of the
// time if it only loads a row when it gets to it (4096 x 6144, f32 stream, bf16
// blocks: 193 us).  With many tokens the rows therefore come through a ring in
// shared memory: one thread issues the bulk copies of the rows ahead (89 us, 5.1
// TB/s, with one barrier a row; with the two that follow the formulas 110 us).  The
// sums are then in registers.  Rows that leave no
// room for two stages, unaligned rows and few tokens take the loads as they come.
// Forward: 8192 x 6144 bf16 66 us (6.1 TB/s; 78 us with columns past the row filled in
// after every load), one token 2.9 us.
#pragma once

#include "pipeline.cuh"
#include "vec.cuh"

namespace coli {

constexpr int kNormMaxH = 16384;
constexpr int kNormSums = 3;  // dpost_gain, dgate (channel gates), dpre_gain
constexpr int kNormKept = 2;  // sums over tokens that a CTA keeps: z, of which the first two are made, and dpre_gain

struct NormArgs {
    int H, T;
    int post_norm, gate_kind;   // coli_gate
    float alpha, eps;
    const float* post_gain;
    const float* pre_gain;
    const float* gate;
};

template <int N>
__device__ __forceinline__ F<N> ones() {
    F<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = 1.0f;
    return r;
}
// this thread's part of vector i of a row: first column, and what lies between its chunks
template <int W> struct Part {
    int c, stride;
    __device__ __forceinline__ Part(int c0, int step, int i) : c(c0 + i * step), stride(step / 8 * W) {}
};
template <typename T, int W>
__device__ __forceinline__ Cols<T, 8, W> ld_part(const T* row, const Part<W>& p, int H) {
    return ldc<T, 8, W>(row, p.c, p.stride, H);
}
template <typename T, int W>
__device__ __forceinline__ void st_part(T* row, const Part<W>& p, int H, const F<8>& f) {
    stc<T, 8, W>(row, p.c, p.stride, H, narrow_cols<T, 8, W>(f));
}
template <int W>
__device__ __forceinline__ F<8> gain_at(const float* g, const Part<W>& p, int H) {
    return g ? widen<float, 8, W>(ld_part<float, W>(g, p, H)) : ones<8>();
}

// gate of token t at this part
template <int W>
__device__ __forceinline__ F<8> gate_at(const NormArgs& a, int64_t t, const Part<W>& p) {
    if (a.gate_kind == 1) return gain_at<W>(a.gate, p, a.H);
    if (a.gate_kind == 3) return gain_at<W>(a.gate + t * a.H, p, a.H);
    F<8> r = ones<8>();
    if (a.gate_kind == 2) {
        const float g = a.gate[t];
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j] = g;
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

template <typename XT, typename BT, int W, int N>
__global__ void __launch_bounds__(norm_max_threads(N), W == 8 && (N == 2 || N == 3) ? 2 : 1)
block_norm_kernel(NormArgs a, const XT* x, const BT* o, XT* x_out, BT* n_out, float* rstd_post,
                  float* rstd_pre) {
    __shared__ float part[2][32];
    const int64_t t = blockIdx.x;
    const int64_t row = t * a.H;
    const int step = (int)blockDim.x * 8, c0 = (int)threadIdx.x * W;
    pdl_trigger();
    pdl_wait();
    // u gate alpha = o (r_o c) w, w = post_gain times a gate of the channels, c = alpha times a token's
    const float* post_gain = a.post_norm ? a.post_gain : nullptr;
    const auto weight = [&](const Part<W>& p) {
        F<8> w = gain_at<W>(post_gain, p, a.H);
        if (a.gate_kind == 1 || a.gate_kind == 3) {
            const F<8> g = gate_at<W>(a, t, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) w.v[j] *= g.v[j];
        }
        return w;
    };
    Cols<XT, 8, W> xv[N];
    Cols<BT, 8, W> ov[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const Part<W> p(c0, step, i);
        if (p.c >= a.H) continue;
        if (o) ov[i] = ld_part<BT, W>(o + row, p, a.H);
        xv[i] = ld_part<XT, W>(x + row, p, a.H);
    }
    F<8> early_w, early_pre;  // N == 1: asked for before the sums
    if (N == 1 && c0 < a.H) {
        const Part<W> p(c0, step, 0);
        if (o) early_w = weight(p);
        if (n_out) early_pre = gain_at<W>(a.pre_gain, p, a.H);
    }
    float s[1] = {0.0f};
    if (o) {
        float rc = a.alpha * (a.gate_kind == 2 ? a.gate[t] : 1.0f);
        if (a.post_norm) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (c0 + i * step >= a.H) continue;
                const F<8> f = widen<BT, 8, W>(ov[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = fmaf(f.v[j], f.v[j], s[0]);
            }
            cta_sum(s, part[0]);
            const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
            if (rstd_post && threadIdx.x == 0) rstd_post[t] = r;
            rc *= r;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Part<W> p(c0, step, i);
            if (p.c >= a.H) continue;
            const F<8> w = N == 1 ? early_w : weight(p);
            const F<8> of = widen<BT, 8, W>(ov[i]), xf = widen<XT, 8, W>(xv[i]);
            F<8> f;
#pragma unroll
            for (int j = 0; j < 8; ++j) f.v[j] = fmaf(of.v[j] * rc, w.v[j], xf.v[j]);
            xv[i] = narrow_cols<XT, 8, W>(f);  // the stored value, which the norm below reads
            stc<XT, 8, W>(x_out + row, p.c, p.stride, a.H, xv[i]);
        }
    }
    if (!n_out) return;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const Part<W> p(c0, step, i);
        if (p.c >= a.H) continue;
        const F<8> f = widen<XT, 8, W>(xv[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p.c + j / W * p.stride < a.H) s[0] = fmaf(f.v[j], f.v[j], s[0]);
    }
    cta_sum(s, part[1]);
    const float r = 1.0f / sqrtf(s[0] / (float)a.H + a.eps);
    if (rstd_pre && threadIdx.x == 0) rstd_pre[t] = r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const Part<W> p(c0, step, i);
        if (p.c >= a.H) continue;
        const F<8> pg = N == 1 ? early_pre : gain_at<W>(a.pre_gain, p, a.H);
        F<8> f = widen<XT, 8, W>(xv[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) f.v[j] = f.v[j] * r * pg.v[j];
        st_part<BT, W>(n_out + row, p, a.H, f);
    }
}

// Sums of this CTA in shared memory, kept so that a warp's accesses meet no bank
// twice: for vectors of eight neighbours, the first four elements of all vectors, then
// the last four; else in the order of their columns.
template <int W>
__device__ __forceinline__ int sum_at(int c, int H) {  // column c of one sum
    return W == 8 ? (((c >> 2) & 1) * (H >> 3) + (c >> 3)) * 4 + (c & 3) : c;
}
template <int W>
__device__ __forceinline__ void sum_add(float* sums, const Part<W>& p, int H, const F<8>& f, const F<8>& g) {
    if constexpr (W == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (p.c >= H) break;
            float4* at = reinterpret_cast<float4*>(sums + sum_at<W>(p.c + 4 * h, H));
            float4 v = *at;
            v.x = fmaf(f.v[4 * h], g.v[4 * h], v.x);
            v.y = fmaf(f.v[4 * h + 1], g.v[4 * h + 1], v.y);
            v.z = fmaf(f.v[4 * h + 2], g.v[4 * h + 2], v.z);
            v.w = fmaf(f.v[4 * h + 3], g.v[4 * h + 3], v.w);
            *at = v;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = p.c + j / W * p.stride + j % W;
            if (c < H) sums[c] = fmaf(f.v[j], g.v[j], sums[c]);
        }
    }
}

// Where each sum lives among the partial rows, -1 for one that is not asked for.
struct NormSums {
    int at[kNormSums];
    int n;
};

// Shared memory of the ring form: the vectors of H that every row needs
// (pre_gain; w of the gradient, see below: in sum_at's order), then the stages, each
// with the rows x_out, dx_out, o, dn one after the other.  What a call does not
// have is not there.
struct NormRing {
    int stages;
    int stage;          // bytes, a multiple of 16
    int off[4];         // of a row in its stage, -1: absent
    int gain[2];        // of a vector, -1: absent
    int first;          // of the first stage
};
constexpr int kNormMaxStages = 4;

// eight elements of a row in shared memory as they lie there
template <typename T>
__device__ __forceinline__ Vec<T, 8> lds_row(const uint8_t* row, int c) {
    Vec<T, 8> r;
#pragma unroll
    for (int i = 0; i < r.bytes / 16; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + c * (int)sizeof(T) + 16 * i);
        r.u[4 * i] = v.x; r.u[4 * i + 1] = v.y; r.u[4 * i + 2] = v.z; r.u[4 * i + 3] = v.w;
    }
    return r;
}

// eight elements from column c of a vector kept in sum_at's order
__device__ __forceinline__ F<8> lds_gain(const uint8_t* smem, int off, int c, int H) {
    F<8> r;
    const float* p = reinterpret_cast<const float*>(smem + off);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 v = *reinterpret_cast<const float4*>(p + sum_at<8>(c + 4 * h, H));
        r.v[4 * h] = v.x; r.v[4 * h + 1] = v.y; r.v[4 * h + 2] = v.z; r.v[4 * h + 3] = v.w;
    }
    return r;
}

// One barrier a row.  With w = alpha gate post_gain (a token's gate g_t apart: w =
// post_gain, c = alpha g_t; else c = 1), d' = dx' + r_x v and d = d' - r_x <v xh> xh,
//   sum q oh = c (sum w oh d' - r_x <v xh> sum w oh xh)
// so the three sums over the row are taken together, before d is known.  Of the sums
// over tokens one, z = sum_t c d oh (c includes alpha gate where the gate is full),
// makes two gradients where the gate is the same for every token: dpost_gain = alpha
// gate z, dgate = alpha post_gain z.
// partial [clusters][keep.n][H]
// A copy that does not land within the limit of its wait (seconds; nothing but a fault keeps
// it) makes that row and the rest of its CTA's NaN in every gradient, the sums over
// tokens with them, without further waits or copies.  TW: the wait test
// (coli_moe_block_norm_set_wait_test): CTA 0 never copies its row `withhold`, and the limit is
// short.
constexpr uint32_t kNormTestTries = 4096;
template <typename XT, typename BT, int W, int N, bool RING, bool TW>
__global__ void __launch_bounds__(N == 1 ? 768 : 512)
block_norm_backward_kernel(NormArgs a, NormSums keep, NormRing ring, const XT* x_out, const BT* o,
                           const float* rstd_post, const float* rstd_pre, const XT* dx_out, const BT* dn, XT* dx,
                           BT* d_o, float* dgate, float* partial, int withhold) {
    extern __shared__ __align__(128) uint8_t nb_smem[];   // the ring, or the sums; at the end the sums
    __shared__ float part[2][96];                         // of even and odd rows
    __shared__ __align__(8) uint64_t full[kNormMaxStages];
    __shared__ float rstds[kNormMaxStages][2];
    __shared__ int gone;                                  // a wait of this CTA has given up
    float* sums = reinterpret_cast<float*>(nb_smem);
    static_assert(!RING || W == 8, "rows of the ring are read in vectors of eight");
    const int step = (int)blockDim.x * 8, c0 = (int)threadIdx.x * W;
    const bool token = a.gate_kind == 2, full_gate = a.gate_kind == 3;
    const bool keep_z = keep.at[0] >= 0 || keep.at[1] >= 0, keep_pre = keep.at[2] >= 0;
    float* z_sums = sums;
    float* pre_sums = sums + (keep_z ? a.H : 0);
    const int kept = (keep_z ? 1 : 0) + (keep_pre ? 1 : 0);
    F<8> z_acc[RING ? N : 1], pre_acc[RING ? N : 1];
    if (RING) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) z_acc[RING ? i : 0].v[j] = pre_acc[RING ? i : 0].v[j] = 0.0f;
        if (threadIdx.x == 0) {
            for (int i = 0; i < ring.stages; ++i) mbar_init(&full[i], 2);  // the rows, the two rstd
            fence_mbar_init();
            gone = 0;
        }
    } else {
        for (int i = threadIdx.x; i < kept * a.H; i += blockDim.x) sums[i] = 0.0f;
    }
    __syncthreads();
    const float inv_h = 1.0f / (float)a.H;
    const float fill = token ? 1.0f : a.alpha;            // w without gains
    const float* post_gain = a.post_norm ? a.post_gain : nullptr;
    // row t into stage `at` (one thread)
    const auto fetch = [&](int64_t t, int at) {
        if (t >= a.T || (TW && t == (int64_t)withhold * gridDim.x)) return;
        uint8_t* st = nb_smem + ring.first + at * ring.stage;
        const uint32_t xb = a.H * (uint32_t)sizeof(XT), bb = a.H * (uint32_t)sizeof(BT);
        mbar_expect_tx(&full[at], (ring.off[0] >= 0 ? xb : 0) + (ring.off[1] >= 0 ? xb : 0) +
                                      (ring.off[2] >= 0 ? bb : 0) + (ring.off[3] >= 0 ? bb : 0));
        if (ring.off[0] >= 0) bulk_g2s(st + ring.off[0], x_out + t * a.H, xb, &full[at]);
        if (ring.off[1] >= 0) bulk_g2s(st + ring.off[1], dx_out + t * a.H, xb, &full[at]);
        if (ring.off[2] >= 0) bulk_g2s(st + ring.off[2], o + t * a.H, bb, &full[at]);
        if (ring.off[3] >= 0) bulk_g2s(st + ring.off[3], dn + t * a.H, bb, &full[at]);
        if (dn) cp_async4(smem_u32(&rstds[at][0]), rstd_pre + t);
        if (o && a.post_norm) cp_async4(smem_u32(&rstds[at][1]), rstd_post + t);
        cp_async_arrive(&full[at]);
    };
    pdl_trigger();
    pdl_wait();
    if (RING) {
        if (threadIdx.x == 0)
            for (int i = 0; i < ring.stages; ++i) fetch(blockIdx.x + (int64_t)i * gridDim.x, i);
        for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
            const int to = sum_at<W>(c, a.H);
            if (ring.gain[0] >= 0) reinterpret_cast<float*>(nb_smem + ring.gain[0])[to] = a.pre_gain ? a.pre_gain[c] : 1.0f;
            if (ring.gain[1] >= 0)
                reinterpret_cast<float*>(nb_smem + ring.gain[1])[to] =
                    fill * (a.gate_kind == 1 ? a.gate[c] : 1.0f) * (post_gain ? post_gain[c] : 1.0f);
        }
        __syncthreads();
    }
    // w at this part of token t's row
    const auto weight = [&](int64_t t, const Part<W>& p) {
        if (RING && !full_gate) return lds_gain(nb_smem, ring.gain[1], p.c, a.H);
        F<8> w = gain_at<W>(post_gain, p, a.H);
        if (a.gate_kind == 1 || full_gate) {
            const F<8> g = gate_at<W>(a, t, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) w.v[j] *= fill * g.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w.v[j] *= fill;
        }
        return w;
    };
    int at = 0, odd = 0;
    uint32_t phase = 0;
    bool broken = false;                                  // as gone was at the last row's barrier
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, odd ^= 1) {
        const int64_t row = t * a.H;
        F<8> d[N];
        Cols<XT, 8, W> xv[N];
        Cols<BT, 8, W> ov[N];
        float s[3] = {0.0f, 0.0f, 0.0f};  // v xh, w oh d', w oh xh
        float rx = 0.0f, ro = 1.0f;
        const uint8_t* st = nb_smem + ring.first + at * ring.stage;
        if (RING && !broken && !mbar_wait(&full[at], phase, nullptr, TW ? kNormTestTries : kWaitTries))
            *(volatile int*)&gone = 1;
        if (dn) rx = RING ? rstds[at][0] : rstd_pre[t];
        if (o && a.post_norm) ro = RING ? rstds[at][1] : rstd_post[t];
        const float c = token && o ? a.alpha * a.gate[t] : 1.0f;
        Cols<BT, 8, W> gv[N];
        constexpr bool keep_w = !RING && N <= 2;           // as registers allow
        F<8> kept_w[keep_w ? N : 1];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Part<W> p(c0, step, i);
            if (p.c >= a.H) continue;
            if constexpr (RING) {
                if (dn) {
                    xv[i].q[0] = lds_row<XT>(st + ring.off[0], p.c);
                    gv[i].q[0] = lds_row<BT>(st + ring.off[3], p.c);
                }
                if (dx_out) d[i] = widen<XT, 8>(lds_row<XT>(st + ring.off[1], p.c));
                if (o) ov[i].q[0] = lds_row<BT>(st + ring.off[2], p.c);
            } else {
                if (dn) {
                    xv[i] = ld_part<XT, W>(x_out + row, p, a.H);
                    gv[i] = ld_part<BT, W>(dn + row, p, a.H);
                }
                if (dx_out) d[i] = widen<XT, 8, W>(ld_part<XT, W>(dx_out + row, p, a.H));
                if (o) ov[i] = ld_part<BT, W>(o + row, p, a.H);
            }
            if (!dx_out) {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i].v[j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Part<W> p(c0, step, i);
            if (p.c >= a.H) continue;
            F<8> xh;
            if (dn) {
                F<8> pg;
                if constexpr (RING) pg = lds_gain(nb_smem, ring.gain[0], p.c, a.H);
                else pg = gain_at<W>(a.pre_gain, p, a.H);
                const F<8> xf = widen<XT, 8, W>(xv[i]), gf = widen<BT, 8, W>(gv[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh.v[j] = xf.v[j] * rx;
                    const float v = gf.v[j] * pg.v[j];
                    s[0] = fmaf(v, xh.v[j], s[0]);
                    d[i].v[j] = fmaf(rx, v, d[i].v[j]);
                }
                if (keep_pre) {
                    if constexpr (RING) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) pre_acc[i].v[j] = fmaf(gf.v[j], xh.v[j], pre_acc[i].v[j]);
                    } else {
                        sum_add<W>(pre_sums, p, a.H, gf, xh);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) xh.v[j] = 0.0f;
            }
            if (o) {
                const F<8> w = weight(t, p);
                if (keep_w) kept_w[keep_w ? i : 0] = w;
                const F<8> of = widen<BT, 8, W>(ov[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float woh = of.v[j] * ro * w.v[j];
                    s[1] = fmaf(woh, d[i].v[j], s[1]);
                    s[2] = fmaf(woh, xh.v[j], s[2]);
                }
            }
        }
        if (dn || (o && (a.post_norm || token))) cta_sum(s, part[odd]);
        else if (RING) __syncthreads();
        // every thread has its part of the row: the stage takes the row that comes next in it
        if (RING) {
            broken = *(volatile int*)&gone != 0;
            if (broken) {
                s[1] = __uint_as_float(0x7fc00000u);
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[i].v[j] = pre_acc[RING ? i : 0].v[j] = s[1];
            }
            if (threadIdx.x == 0 && !broken) fetch(t + (int64_t)ring.stages * gridDim.x, at);
            if (++at == ring.stages) {
                at = 0;
                phase ^= 1;
            }
        }
        const float mean = s[0] * inv_h;                  // <v xh>
        const float s_q = fmaf(-rx * mean, s[2], s[1]);   // sum q oh, without c
        if (o && token && dgate && threadIdx.x == 0) dgate[t] = a.alpha * s_q;
        const float to_d = -rx * rx * mean;
        const float c_ro = c * ro, to_o = -ro * ro * (c * s_q * inv_h);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Part<W> p(c0, step, i);
            if (p.c >= a.H) continue;
            if (dn) {
                const F<8> xf = widen<XT, 8, W>(xv[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i].v[j] = fmaf(to_d, xf.v[j], d[i].v[j]);
            }
            st_part<XT, W>(dx + row, p, a.H, d[i]);
            if (!o) continue;
            const F<8> w = keep_w ? kept_w[keep_w ? i : 0] : weight(t, p);
            const F<8> of = widen<BT, 8, W>(ov[i]);
            F<8> oh, r;  // c oh; the gradient of o
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                oh.v[j] = of.v[j] * c_ro;
                r.v[j] = fmaf(c_ro, w.v[j] * d[i].v[j], a.post_norm ? to_o * of.v[j] : 0.0f);
            }
            st_part<BT, W>(d_o + row, p, a.H, r);
            if (full_gate) {
                const F<8> g = gate_at<W>(a, t, p), pg = gain_at<W>(post_gain, p, a.H);
                if (dgate) {
                    F<8> dg;
#pragma unroll
                    for (int j = 0; j < 8; ++j) dg.v[j] = a.alpha * (oh.v[j] * pg.v[j] * d[i].v[j]);
                    st_part<float, W>(dgate + row, p, a.H, dg);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) oh.v[j] *= a.alpha * g.v[j];
            }
            if (keep_z) {
                if constexpr (RING) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) z_acc[i].v[j] = fmaf(d[i].v[j], oh.v[j], z_acc[i].v[j]);
                } else {
                    sum_add<W>(z_sums, p, a.H, d[i], oh);
                }
            }
        }
    }
    if (keep.n == 0) return;
    __syncthreads();
    if (RING) {  // every row has been read: the ring's memory takes the sums
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Part<W> p(c0, step, i);
            if (p.c >= a.H) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (keep_z) z_sums[sum_at<W>(p.c + j, a.H)] = z_acc[RING ? i : 0].v[j];
                if (keep_pre) pre_sums[sum_at<W>(p.c + j, a.H)] = pre_acc[RING ? i : 0].v[j];
            }
        }
    }
    cluster_sync();
    const int cs = (int)cluster_size(), rank = (int)cluster_rank();
    float* mine = partial + (int64_t)(blockIdx.x / cs) * keep.n * a.H;
    for (int i = rank * (int)blockDim.x + (int)threadIdx.x; i < keep.n * a.H; i += cs * (int)blockDim.x) {
        const int k = i / a.H, col = i - k * a.H;
        const float* p = (k == keep.at[2] ? pre_sums : z_sums) + sum_at<W>(col, a.H);
        float s = 0.0f;
        for (int q = 0; q < cs; ++q) s += ld_cluster(p, q);
        if (k == keep.at[0] && !token && !full_gate) s *= a.alpha * (a.gate_kind == 1 ? a.gate[col] : 1.0f);
        if (k == keep.at[1]) s *= a.alpha * (post_gain ? post_gain[col] : 1.0f);
        mine[i] = s;
    }
    cluster_sync();  // no CTA leaves while another reads its sums
}

// out[c] = sum over the partial rows, 32 columns by RUNS runs of rows per CTA;
// blockIdx.y picks the sum
template <int RUNS>
__global__ void __launch_bounds__(32 * RUNS)
norm_reduce_kernel(const float* __restrict__ partial, int rows, int H, NormSums keep, float* dpost, float* dgate,
                   float* dpre) {
    __shared__ float part[RUNS][32];
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
        for (int r = run; r < rows; r += RUNS) s += partial[((int64_t)r * keep.n + k) * H + c];
    part[run][lane] = s;
    __syncthreads();
    if (run == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < RUNS; ++i) s += part[i][lane];
        out[c] = s;
    }
}

}  // namespace coli
