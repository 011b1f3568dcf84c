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
// bytes (at most 16).  Pairs of 16-bit elements stay 32-bit words: taken out
// one by one and rounded one by one they cost about twice the instructions
// (25 per element of a layer norm).
template <typename T, int VEC, bool PAIRS = sizeof(T) == 2 && VEC % 2 == 0> struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
    __device__ __forceinline__ float get(int i) const { return to_f32<T>(v[i]); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = from_f32<T>(f[i]);
    }
};
__device__ __forceinline__ float half_of(uint32_t w, int i, __nv_bfloat16) {
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float half_of(uint32_t w, int i, __half) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return i & 1 ? __high2float(h) : __low2float(h);
}
__device__ __forceinline__ uint32_t pair_of(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pair_of(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T, int VEC> struct alignas(sizeof(T) * VEC) Pack<T, VEC, true> {
    uint32_t w[VEC / 2];
    __device__ __forceinline__ float get(int i) const { return half_of(w[i / 2], i, T()); }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) w[i] = pair_of(f[2 * i], f[2 * i + 1], T());
    }
};

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, VEC> *>(p);
}
template <typename T, int VEC> __device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &v) {
    *reinterpret_cast<Pack<T, VEC> *>(p) = v;
}

// two float32 operations in one instruction
struct Two {
    unsigned long long v;
};
__device__ __forceinline__ Two two(float a, float b) {
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void both(Two t, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(t.v)); }
__device__ __forceinline__ Two fma_two(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two add_two(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two mul_two(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// elements i and i + 1 of a piece
template <typename P> __device__ __forceinline__ Two pair_at(const P &p, int i) { return two(p.get(i), p.get(i + 1)); }

// sum over the L (a power of two, at most 32) neighbouring lanes of a group,
// the same bits in every lane
template <int L> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// the largest piece that base, row distance and D allow: 16 bytes, 4 bytes
// (16-bit types) or one element
inline int piece_bytes(const void *p, long long ld, int D, int bytes) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * bytes) | (uintptr_t)((long long)D * bytes);
    return (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : bytes;
}

}  // namespace sad
