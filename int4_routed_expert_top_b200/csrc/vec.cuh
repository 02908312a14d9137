// vec.cuh - vector loads and conversions, and the two ends of a programmatic
// dependent launch, for the operators around the experts.
#pragma once

#include "common.cuh"

namespace coli {

// the next kernel of the stream may be scheduled now; wait: everything before
// this kernel is complete and visible
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// N consecutive elements of type T as they lie in memory, aligned to their size:
// one load or store (32 bytes are one access on sm_100, so that a lane writes
// whole sectors).  Kept as 32-bit words, so that values which wait in registers
// wait in the type they were read in.
template <typename T, int N> struct Vec {
    static constexpr int bytes = (int)sizeof(T) * N;
    static_assert(bytes == 2 || bytes == 4 || bytes == 8 || bytes == 16 || bytes == 32, "one access");
    uint32_t u[bytes < 4 ? 1 : bytes / 4];
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ldv(const T* p) {
    Vec<T, N> r;
    if constexpr (r.bytes == 32) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.u[0]), "=r"(r.u[1]), "=r"(r.u[2]), "=r"(r.u[3]), "=r"(r.u[4]), "=r"(r.u[5]),
                       "=r"(r.u[6]), "=r"(r.u[7])
                     : "l"(p) : "memory");
    } else if constexpr (r.bytes == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        r.u[0] = v.x; r.u[1] = v.y; r.u[2] = v.z; r.u[3] = v.w;
    } else if constexpr (r.bytes == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        r.u[0] = v.x; r.u[1] = v.y;
    } else if constexpr (r.bytes == 4) {
        r.u[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
        r.u[0] = *reinterpret_cast<const uint16_t*>(p);
    }
    return r;
}
template <typename T, int N>
__device__ __forceinline__ void stv(T* p, const Vec<T, N>& r) {
    if constexpr (r.bytes == 32)
        asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                     ::"r"(r.u[0]), "r"(r.u[1]), "r"(r.u[2]), "r"(r.u[3]), "r"(r.u[4]), "r"(r.u[5]), "r"(r.u[6]),
                       "r"(r.u[7]), "l"(p)
                     : "memory");
    else if constexpr (r.bytes == 16)
        *reinterpret_cast<uint4*>(p) = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
    else if constexpr (r.bytes == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(r.u[0], r.u[1]);
    else if constexpr (r.bytes == 4)
        *reinterpret_cast<uint32_t*>(p) = r.u[0];
    else
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)r.u[0];
}

// the same as f32 values, and back (rounded to nearest even)
template <int N> struct F { float v[N]; };
template <typename T, int N> __device__ __forceinline__ F<N> widen(const Vec<T, N>& a) {
    F<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (sizeof(T) == 4)
            r.v[i] = __uint_as_float(a.u[i]);
        else  // bf16 is the upper half of an f32
            r.v[i] = __uint_as_float(i & 1 ? a.u[i / 2] & 0xffff0000u : a.u[i / 2] << 16);
    }
    return r;
}
template <typename T, int N> __device__ __forceinline__ Vec<T, N> narrow(const F<N>& a) {
    Vec<T, N> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) r.u[i] = __float_as_uint(a.v[i]);
    } else if constexpr (N == 1) {
        r.u[0] = __bfloat16_as_ushort(__float2bfloat16_rn(a.v[0]));
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a.v[2 * i], a.v[2 * i + 1]);
            r.u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return r;
}
template <typename T, int N> __device__ __forceinline__ void stf(T* p, const F<N>& a) { stv<T, N>(p, narrow<T, N>(a)); }

// N elements of a row as N / W chunks of W neighbours, `stride` elements apart: W = N
// where rows and pointers allow one wide access; else a thread's chunks lie a
// warp's (or CTA's) worth of chunks apart, so that each access of a warp is still
// one run of memory, and as many bytes are in flight.  Chunks at column H or
// later are left out (a multiple of W).
template <typename T, int N, int W> struct Cols { Vec<T, W> q[N / W]; };

template <typename T, int N, int W>
__device__ __forceinline__ Cols<T, N, W> ldc(const T* row, int c, int stride, int H) {
    Cols<T, N, W> r;
#pragma unroll
    for (int i = 0; i < N / W; ++i)
        if (c + i * stride < H) r.q[i] = ldv<T, W>(row + c + i * stride);
        else
#pragma unroll
            for (int j = 0; j < (int)(sizeof(r.q[i].u) / 4); ++j) r.q[i].u[j] = 0;
    return r;
}
template <typename T, int N, int W>
__device__ __forceinline__ void stc(T* row, int c, int stride, int H, const Cols<T, N, W>& a) {
#pragma unroll
    for (int i = 0; i < N / W; ++i)
        if (c + i * stride < H) stv<T, W>(row + c + i * stride, a.q[i]);
}
template <typename T, int N, int W> __device__ __forceinline__ F<N> widen(const Cols<T, N, W>& a) {
    F<N> r;
#pragma unroll
    for (int i = 0; i < N / W; ++i) {
        const F<W> f = widen<T, W>(a.q[i]);
#pragma unroll
        for (int j = 0; j < W; ++j) r.v[i * W + j] = f.v[j];
    }
    return r;
}
template <typename T, int N, int W> __device__ __forceinline__ Cols<T, N, W> narrow_cols(const F<N>& a) {
    Cols<T, N, W> r;
#pragma unroll
    for (int i = 0; i < N / W; ++i) {
        F<W> f;
#pragma unroll
        for (int j = 0; j < W; ++j) f.v[j] = a.v[i * W + j];
        r.q[i] = narrow<T, W>(f);
    }
    return r;
}

}  // namespace coli
