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

// N consecutive elements of type T, aligned to their size: one load or store
// (32 bytes are one access on sm_100, so that a lane writes whole sectors)
template <typename T, int N> struct alignas(sizeof(T) * N) Vec { T v[N]; };

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ldv(const T* p) {
    Vec<T, N> r;
    if constexpr (sizeof(T) * N == 32) {
        uint32_t* u = reinterpret_cast<uint32_t*>(&r);
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "l"(p) : "memory");
    } else {
        static_assert(sizeof(T) * N <= 16, "a load is 1 to 16 or 32 bytes");
        r = *reinterpret_cast<const Vec<T, N>*>(p);
    }
    return r;
}
template <typename T, int N>
__device__ __forceinline__ void stv(T* p, const Vec<T, N>& r) {
    if constexpr (sizeof(T) * N == 32) {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
        asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};"
                     ::"r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "l"(p)
                     : "memory");
    } else {
        static_assert(sizeof(T) * N <= 16, "a store is 1 to 16 or 32 bytes");
        *reinterpret_cast<Vec<T, N>*>(p) = r;
    }
}

// the same as f32 values
template <int N> struct F { float v[N]; };
template <typename T, int N> __device__ __forceinline__ F<N> widen(const Vec<T, N>& a) {
    F<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = to_f32(a.v[i]);
    return r;
}
template <typename T, int N> __device__ __forceinline__ F<N> ldf(const T* p) { return widen<T, N>(ldv<T, N>(p)); }
template <typename T, int N> __device__ __forceinline__ void stf(T* p, const F<N>& a) {
    Vec<T, N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(a.v[i]);
    stv<T, N>(p, r);
}

}  // namespace coli
