// packed.h -- vectors of f32, bf16 or f16 elements as 32-bit words: one wide access each way, two 16-bit
// elements a register.  (A struct of __nv_bfloat16 or __half is copied element by element, in 2-byte
// accesses, whatever its alignment: the same kernels ran at a third of the rate with them.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"

namespace trop {

#ifdef __CUDACC__

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// two f32 rounded to 16 bits each, the first in the low half
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if (BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

// VEC elements as they came, unpacked at each use.
template <typename T, int VEC, bool WORDS = (VEC * sizeof(T)) % 4 == 0>
struct Raw {
    static constexpr int N = VEC * sizeof(T) / 4;
    uint32_t w[N];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void read(const T* p)
    {
        if (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const uint4 q = reinterpret_cast<const uint4*>(p)[i];
                w[(4 * i) % N] = q.x, w[(4 * i + 1) % N] = q.y, w[(4 * i + 2) % N] = q.z, w[(4 * i + 3) % N] = q.w;
            }
        } else if (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const uint2 q = reinterpret_cast<const uint2*>(p)[i];
                w[(2 * i) % N] = q.x, w[(2 * i + 1) % N] = q.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
    }
    __device__ __forceinline__ void write(T* p) const
    {
        if (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[(4 * i) % N], w[(4 * i + 1) % N], w[(4 * i + 2) % N], w[(4 * i + 3) % N]);
        } else if (N % 2 == 0) {
#pragma unroll
            for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(w[(2 * i) % N], w[(2 * i + 1) % N]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        }
    }
    // (after this the compiler unpacks anew instead of keeping the unpacked values of an earlier pass)
    __device__ __forceinline__ void again()
    {
#pragma unroll
        for (int i = 0; i < N; ++i) asm volatile("" : "+r"(w[i]));
    }
    __device__ __forceinline__ float get(int i) const
    {
        if (sizeof(T) == 4) return __uint_as_float(w[i % N]);
        const uint32_t h = w[(i / 2) % N];
        if (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(i & 1 ? h & 0xffff0000u : h << 16);
        const __half2 q = *reinterpret_cast<const __half2*>(&h);
        return i & 1 ? __high2float(q) : __low2float(q);
    }
    __device__ __forceinline__ void set(const float (&v)[VEC])
    {
        if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i % VEC]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = pack2<std::is_same<T, __nv_bfloat16>::value>(v[(2 * i) % VEC], v[(2 * i + 1) % VEC]);
        }
    }
};
// a single 16-bit element
template <typename T, int VEC>
struct Raw<T, VEC, false> {
    T e[VEC];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(0.f);
    }
    __device__ __forceinline__ void read(const T* p)
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = p[i];
    }
    __device__ __forceinline__ void write(T* p) const
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = e[i];
    }
    __device__ __forceinline__ void again() {}
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
    __device__ __forceinline__ void set(const float (&v)[VEC])
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(v[i]);
    }
};
#endif

}  // namespace trop
