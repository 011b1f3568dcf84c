// sad_rows.cuh -- row matrices of the feature-field kernels: elements of
// float32, bfloat16 or binary16, read and written VEC at a time as float32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace sad {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// the one rounding of a result, to nearest even
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// VEC consecutive elements as one aligned load or store of VEC * sizeof(T)
// bytes (at most 16)
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
    __device__ __forceinline__ float get(int i) const { return to_f32<T>(v[i]); }
    __device__ __forceinline__ void set(int i, float f) { v[i] = from_f32<T>(f); }
};

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}
template <typename T, int VEC> __device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &v) {
    *reinterpret_cast<Pack<T, VEC> *>(p) = v;
}

// sum over the L (a power of two, at most 32) neighbouring lanes of a group,
// the same bits in every lane
template <int L> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace sad
