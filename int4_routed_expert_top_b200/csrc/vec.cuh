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

// N elements of type T: 16 bytes, or fewer where a row's length or a pointer
// allows no more
template <typename T, int N> struct alignas(sizeof(T) * N) Vec { T v[N]; };

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

}  // namespace coli
