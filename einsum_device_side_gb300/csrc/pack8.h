// pack8.h -- activations in 8 bits: 32 consecutive elements of a row (a group; the row's last one may be part-filled)
// share a power of two.
//
//   e = max(6, exponent byte of the group's largest magnitude as f32),  unit = 2^(e - 133),
//   code = x / unit rounded to nearest even, at most 127 in magnitude,  value = code unit.
//
// The largest magnitude lies in [64, 128) units, so a code is off by at most half a unit, 1 / 128 of that magnitude,
// and magnitudes above 127.5 units by less than one.  A power of two makes every step exact: the product x / unit,
// and the value, whose seven bits bf16 holds as they are.  Groups below 2^-121 take the least unit, 2^-127, so that its
// inverse is an f32; e = 255 says that the group held an infinity or a NaN: its values are NaN.
#pragma once

#include <stdint.h>

#include "packed.h"

namespace trop {

constexpr int GROUP8 = 32;
constexpr uint32_t LEAST8 = 6, BAD8 = 255;

#ifdef __CUDACC__

// from the largest magnitude's f32 bits
__device__ __forceinline__ uint32_t scale8(uint32_t top) { return max(top >> 23, LEAST8); }
__device__ __forceinline__ float inverse_unit8(uint32_t e) { return __uint_as_float((260u - e) << 23); }
__device__ __forceinline__ float unit8(uint32_t e)
{
    return __uint_as_float(e == BAD8 ? 0x7fc00000u : e == LEAST8 ? 0x00400000u : (e - LEAST8) << 23);
}

// The largest magnitude of VEC elements, as f32 bits (of a NaN's or an infinity's, at least 255 << 23).  16-bit elements
// are compared as the integers that their magnitudes are in order of, two at a time.
template <typename T, int VEC>
__device__ __forceinline__ uint32_t top8(const Raw<T, VEC>& q)
{
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max(m, q.w[i] & 0x7fffffffu);
        return m;
    } else if constexpr (VEC % 2 == 0) {
        uint32_t m = q.w[0] & 0x7fff7fffu;
#pragma unroll
        for (int i = 1; i < VEC / 2; ++i) m = __vmaxu2(m, q.w[i] & 0x7fff7fffu);
        const uint32_t h = max(m & 0xffffu, m >> 16);
        if (std::is_same<T, __nv_bfloat16>::value) return h << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
    } else {
        return __float_as_uint(fabsf(q.get(0)));
    }
}
// over the lanes that share a group (32 / VEC neighbours)
template <int VEC>
__device__ __forceinline__ uint32_t group_top8(uint32_t m)
{
#pragma unroll
    for (int o = GROUP8 / VEC / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// VEC elements' codes as bytes in order: x / unit + 1.5 2^23 holds the rounded quotient in its low bits.
constexpr float ROUND8 = 12582912.f;
__device__ __forceinline__ uint32_t code8(float x, float inverse)
{
    return __float_as_uint(fminf(fmaxf(__fmaf_rn(x, inverse, ROUND8), ROUND8 - 127.f), ROUND8 + 127.f));
}
__device__ __forceinline__ uint32_t bytes8(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
template <typename T, int VEC>
__device__ __forceinline__ void codes8(const Raw<T, VEC>& q, uint32_t e, uint32_t (&w)[(VEC + 3) / 4])
{
    const float inverse = inverse_unit8(e);
    if constexpr (VEC == 1) {
        w[0] = code8(q.get(0), inverse) & 0xffu;
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            w[i] = bytes8(code8(q.get(4 * i), inverse), code8(q.get(4 * i + 1), inverse), code8(q.get(4 * i + 2), inverse),
                          code8(q.get(4 * i + 3), inverse));
    }
    if (e == BAD8)
#pragma unroll
        for (int i = 0; i < (VEC + 3) / 4; ++i) w[i] = 0;
}

// Code i of a word as an f32: its byte, with the sign bit turned, under 2^23 is 2^23 + 128 + code.
__device__ __forceinline__ float raised8(uint32_t turned, int i) { return __uint_as_float(__byte_perm(turned, 0x4b000000u, 0x7540 + i)); }
__device__ __forceinline__ float coded8(uint32_t turned, int i) { return raised8(turned, i) - 8388736.f; }
// VEC codes' values
template <int VEC>
__device__ __forceinline__ void values8(const uint32_t (&w)[(VEC + 3) / 4], float unit, float (&v)[VEC])
{
    if constexpr (VEC == 1) {
        v[0] = coded8(w[0] ^ 0x80808080u, 0) * unit;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {  // in packed pairs
            const uint32_t t = w[i / 4] ^ 0x80808080u;
            const float2 p = __fmul2_rn(__fadd2_rn(make_float2(raised8(t, i % 4), raised8(t, i % 4 + 1)), make_float2(-8388736.f, -8388736.f)),
                                        make_float2(unit, unit));
            v[i] = p.x, v[i + 1] = p.y;
        }
    }
}

// VEC codes in one access
template <int VEC>
struct Codes {
    uint32_t w[(VEC + 3) / 4];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (VEC + 3) / 4; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void read(const int8_t* p)
    {
        if constexpr (VEC == 1) w[0] = (uint8_t)*p;
        else if constexpr (VEC == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (VEC == 8) {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x, w[1] = q.y;
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 16; ++i) {
                const uint4 q = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
            }
        }
    }
    __device__ __forceinline__ void write(int8_t* p) const
    {
        if constexpr (VEC == 1) *p = (int8_t)w[0];
        else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else {
#pragma unroll
            for (int i = 0; i < VEC / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
};
// VEC codes from any byte on: the aligned words around them, where those lie in the matrix (whatever row of it), shifted
// together; at the matrix's own ends one by one.  Bytes outside the row are whatever they are: nobody stores them.
template <int VEC>
__device__ __forceinline__ void codes_any(const int8_t* p, int skip, int left, const int8_t* begin, const int8_t* end, Codes<VEC>& q,
                                          const Span& sp)
{
    (void)sp;
    constexpr int N = VEC / 4;
    const uint32_t off = (uint32_t)((uintptr_t)p & 3);
    const int8_t* const at = p - off;
    if (at >= begin && at + VEC + 4 <= end) {
        uint32_t w[N + 1];
#pragma unroll
        for (int i = 0; i <= N; ++i) w[i] = TROP_IN(at + 4 * i, 4, sp) ? reinterpret_cast<const uint32_t*>(at)[i] : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) q.w[i] = __funnelshift_r(w[i], w[i + 1], off * 8);
    } else {
        q.zero();
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i >= skip && i < left && TROP_IN(p + i, 1, sp)) q.w[i / 4] |= (uint32_t)(uint8_t)p[i] << 8 * (i % 4);
    }
}
#endif

}  // namespace trop
