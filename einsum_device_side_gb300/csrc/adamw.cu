// adamw.cu -- one AdamW step over many tensors at once, states in 32 or in 8 bits.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^k) * m / (sqrt(v) / sqrt(1 - b2^k) + eps)
//
// in f32, each operation rounded once and none contracted, so a step is reproducible bit for bit by
// any IEEE f32 arithmetic in the same order (the 8-bit codes below depend on that).
//
// 8-bit states: blocks of 256 consecutive elements share one f32 scale.  m is kept as a signed code
// c in -127 .. 127 that stands for c |c| top / 127^2, top being the block's largest |m|; of v its
// root r = sqrt(v) is kept, as a code 0 .. 255 that stands for c^2 top / 255^2.  The square law
// gives small entries a finer step (relative step 2 / c, down to top / 127^2 and top / 255^2) than
// an even code; r, not v, is what the update divides by, and no r > 0 is coded as 0: a kept r is at
// most 2.25 times too small (code 1 from 1.5^2 levels down; 1 + 1 / c above), which bounds what rounding
// adds to a later update.  The update itself uses the unrounded new m and v.
//
// The step moves 28 (f32) or 16 (8-bit, f32 parameters) bytes per element and is bound by memory.
// One launch covers hundreds of tensors: the grid has one block per 4096 elements of any tensor.  A
// single call's tensor table travels in the kernel's parameters, where a block finds its tensor by
// bisection; that of a plan of many tensors lies in device memory with each block's tensor written
// down, because a launch with 30 KB of parameters takes the host about 8 us instead of 2.
//
// Measured, 2^27 f32 elements in 96 tensors: 32-bit states 532 us, 7.1 TB/s; 8-bit states 633 us with the
// states' values read back (the step 435 us, the values 198 us; 2^25 elements: the step 119 us, 73 % of the issue slots:
// the codes' arithmetic, 98 instructions an element, bounds it before memory does).  Twelve small tensors: 4.7 us, the
// launch.  4096 elements a block: 16 of each array a thread, all loads on their way before the first is used.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <vector>

#define TROP_TU 8  // this file's id in a bounds-violation record
#include "internal.h"
#include "packed.h"
#include "train.h"

namespace trop {
namespace {

constexpr int CHUNK = 4096;   // elements of one block of threads
constexpr int BLOCK = 256;    // elements of one scale

// Codes move four to a word.  A byte becomes a float by putting it below the exponent of 2^23 (of which
// 2^23 is then taken off, exactly), and a float a byte by adding 1.5 * 2^23, which rounds it to the
// nearest whole number (ties to even) in the low bits: ordinary f32 adds at full rate, where
// conversions run at a quarter of it or less.
template <bool SIGNED>
__device__ __forceinline__ float byte_to_f32(uint32_t word, int i)
{
    if (SIGNED) word ^= 0x80808080u;  // -128 .. 127 -> 0 .. 255
    const float f = __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7650 | i));
    return f - (SIGNED ? 8388736.f : 8388608.f);
}
constexpr float TO_WHOLE = 12582912.f;  // 1.5 * 2^23

// Four elements at p (of a block's chunk; the first `left` exist): one access each way where the
// whole chunk exists and is aligned (FULL).
template <typename T, bool FULL>
__device__ __forceinline__ void load4(const T* p, int left, const Span& sp, float (&v)[4])
{
    (void)sp;
    if (FULL) {
        Raw<T, 4> q;
        if (TROP_IN(p, 4 * sizeof(T), sp)) q.read(p);
        else q.zero();
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = q.get(k);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k < left && TROP_IN(p + k, sizeof(T), sp) ? to_f32(p[k]) : 0.f;
    }
}
template <typename T, bool FULL>
__device__ __forceinline__ void store4(T* p, int left, const Span& sp, const float (&v)[4])
{
    (void)sp;
    if (FULL) {
        Raw<T, 4> q;
        q.set(v);
        if (TROP_IN(p, 4 * sizeof(T), sp)) q.write(p);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left && TROP_IN(p + k, sizeof(T), sp)) p[k] = from_f32<T>(v[k]);
    }
}
// Four codes as their word, and back.
template <bool FULL>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int left, const Span& sp)
{
    (void)sp;
    if (FULL) return TROP_IN(p, 4, sp) ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (k < left && TROP_IN(p + k, 1, sp)) w |= (uint32_t)p[k] << (8 * k);
    return w;
}
template <bool FULL>
__device__ __forceinline__ void store_codes(uint8_t* p, int left, const Span& sp, uint32_t w)
{
    (void)sp;
    if (FULL) {
        if (TROP_IN(p, 4, sp)) *reinterpret_cast<uint32_t*>(p) = w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < left && TROP_IN(p + k, 1, sp)) p[k] = (uint8_t)(w >> (8 * k));
    }
}

// rint(sqrt(u) * levels) for u in [0, 1], sqrt and product each rounded once, plus 1.5 * 2^23.  The
// approximate root (2^-23 relative) decides where the product is further from half way between two
// whole numbers than both ways' errors together, 2.5 * 2^-23 * 255 < NEAR; `off` takes the distance to the
// whole number, and where one of a lane's codes comes nearer to a half, code_exact forms them again.
constexpr float NEAR = 1.220703125e-4f;  // 2^-13
__device__ __forceinline__ float code_of(float u, float levels, float& off)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(u));  // (a flushed u has code 0 either way)
    const float t = r * levels, c = t + TO_WHOLE;
    off = fmaxf(off, fabsf(t - (c - TO_WHOLE)));
    return c;
}
__device__ __forceinline__ float code_exact(float u, float levels) { return __fmul_rn(__fsqrt_rn(u), levels) + TO_WHOLE; }
__device__ __forceinline__ uint32_t low_bytes(const uint32_t (&w)[4])
{
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// A tensor of a launch and the number of its first chunk.
template <typename E>
struct Entry {
    E e;
    uint32_t start;
    uint32_t vec;  // every buffer aligned for accesses of four elements
};
// The tensors of one launch in its parameters: chunk c belongs to entry i with start[i] <= c < start[i + 1].
template <typename E_, int CAP>
struct Table {
    using E = E_;
    int n;
    unsigned* rep;  // the bounds-checked build's record
    uint32_t start[CAP + 1];
    Entry<E> e[CAP];
    __device__ __forceinline__ const Entry<E>& of(uint32_t chunk) const
    {
        int lo = 0, hi = n;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= chunk) lo = mid;
            else hi = mid;
        }
        return e[lo];
    }
};
// The same in device memory (plans), with each chunk's entry written down.
template <typename E_>
struct Resident {
    using E = E_;
    const Entry<E>* e;
    const uint32_t* chunk;  // entry of each chunk
    unsigned* rep;
    __device__ __forceinline__ const Entry<E>& of(uint32_t c) const { return e[chunk[c]]; }
};

// one element's step: m, v and p in place; r = sqrt(v)
__device__ __forceinline__ void step1(float& p, float g, float& m, float& v, float& r, const AdamwScalars& k)
{
    g = __fmul_rn(g, k.gscale);
    m = __fadd_rn(__fmul_rn(m, k.b1), __fmul_rn(g, k.c1));
    v = __fadd_rn(__fmul_rn(v, k.b2), __fmul_rn(__fmul_rn(g, g), k.c2));
    r = __fsqrt_rn(v);
    const float q = __fdiv_rn(m, __fadd_rn(__fmul_rn(r, k.k2), k.eps));
    p = __fsub_rn(__fmul_rn(p, k.decay), __fmul_rn(q, k.lr));
}

// `copy16`: a 16-bit copy of f32 parameters is written beside them (1 bf16, 2 f16)
template <typename TP, bool FULL>
__device__ __forceinline__ void store_param(const trop_adamw_tensor& t, int64_t base, int at, int left, unsigned* rep,
                                            int copy16, const float (&p)[4])
{
    store4<TP, FULL>((TP*)t.param + base + at, left, span_bytes_dev(t.param, t.numel * sizeof(TP), rep), p);
    if (sizeof(TP) == 4 && t.copy) {
        const Span sp = span_bytes_dev(t.copy, t.numel * 2, rep);
        if (copy16 == 1) store4<__nv_bfloat16, FULL>((__nv_bfloat16*)t.copy + base + at, left, sp, p);
        else store4<__half, FULL>((__half*)t.copy + base + at, left, sp, p);
    }
}

// The chunk from `base` on, `size` of its elements existing.
template <typename TP, typename TG, bool FULL>
__device__ __forceinline__ void step_chunk(const trop_adamw_tensor& t, int64_t base, int size, const AdamwScalars& k,
                                           int copy16, unsigned* rep)
{
    const TP* pp = (const TP*)t.param + base;
    const TG* pg = (const TG*)t.grad + base;
    float* pm = (float*)t.exp_avg + base;
    float* pv = (float*)t.exp_avg_sq + base;
    const Span sp_p = span_bytes_dev(t.param, t.numel * sizeof(TP), rep), sp_g = span_bytes_dev(t.grad, t.numel * sizeof(TG), rep);
    const Span sp_m = span_bytes_dev(t.exp_avg, t.numel * 4, rep), sp_v = span_bytes_dev(t.exp_avg_sq, t.numel * 4, rep);
    const int i0 = threadIdx.x * 4;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float p[2][4], g[2][4], m[2][4], v[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + (half * 2 + u) * 1024;
            if (!FULL && i >= size) continue;
            load4<TP, FULL>(pp + i, size - i, sp_p, p[u]);
            load4<TG, FULL>(pg + i, size - i, sp_g, g[u]);
            load4<float, FULL>(pm + i, size - i, sp_m, m[u]);
            load4<float, FULL>(pv + i, size - i, sp_v, v[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + (half * 2 + u) * 1024;
            if (!FULL && i >= size) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float r;
                step1(p[u][q], g[u][q], m[u][q], v[u][q], r, k);
            }
            store_param<TP, FULL>(t, base, i, size - i, rep, copy16, p[u]);
            store4<float, FULL>(pm + i, size - i, sp_m, m[u]);
            store4<float, FULL>(pv + i, size - i, sp_v, v[u]);
        }
    }
}
template <typename TP, typename TG, typename TAB>
__global__ void __launch_bounds__(256) k_adamw(const __grid_constant__ TAB tab, const AdamwScalars k, int copy16)
{
    const Entry<trop_adamw_tensor>& x = tab.of(blockIdx.x);
    pdl_wait();  // (the table is older than the kernel before)
    pdl_signal();
    const int64_t base = (int64_t)(blockIdx.x - x.start) * CHUNK, left = x.e.numel - base;
    if (x.vec && left >= CHUNK) step_chunk<TP, TG, true>(x.e, base, CHUNK, k, copy16, tab.rep);
    else step_chunk<TP, TG, false>(x.e, base, (int)min(left, (int64_t)CHUNK), k, copy16, tab.rep);
}

// A warp per block of 256: lane l has elements 4 l .. and 128 + 4 l .., so that every access of the
// warp is contiguous.  The largest magnitude is taken over the values' bits, which order like the
// magnitudes and let a NaN win: a block with a NaN or an infinity has a scale of NaN (an infinite one
// would leave its largest entry infinite and make NaN of the others), so all of it reads back as NaN.
template <typename TP, typename TG>
struct Block8 {
    Raw<TP, 4> p[2];
    Raw<TG, 4> g[2];
    uint32_t cm[2], cr[2];
    float ms, rs;
};
template <typename T, bool FULL>
__device__ __forceinline__ void load_raw(const T* p, int left, const Span& sp, Raw<T, 4>& q)
{
    float v[4];
    if (FULL) {
        if (TROP_IN(p, 4 * sizeof(T), sp)) q.read(p);
        else q.zero();
    } else {
        load4<T, false>(p, left, sp, v);
        q.set(v);
    }
}
template <typename TP, typename TG, bool FULL>
__device__ __forceinline__ void load_block(const trop_adamw_tensor& t, int64_t base, int size, unsigned* rep, Block8<TP, TG>& x)
{
    const int lane = threadIdx.x & 31;
    const int64_t scales = (t.numel + BLOCK - 1) / BLOCK * 4;
    const float* ps = t.exp_avg_scale + base / BLOCK;
    const float* qs = t.exp_avg_sq_scale + base / BLOCK;
    x.ms = TROP_IN(ps, 4, span_bytes_dev(t.exp_avg_scale, scales, rep)) ? *ps : 0.f;
    x.rs = TROP_IN(qs, 4, span_bytes_dev(t.exp_avg_sq_scale, scales, rep)) ? *qs : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = h * 128 + lane * 4;
        load_raw<TP, FULL>((const TP*)t.param + base + i, size - i, span_bytes_dev(t.param, t.numel * sizeof(TP), rep), x.p[h]);
        load_raw<TG, FULL>((const TG*)t.grad + base + i, size - i, span_bytes_dev(t.grad, t.numel * sizeof(TG), rep), x.g[h]);
        x.cm[h] = load_codes<FULL>((const uint8_t*)t.exp_avg + base + i, size - i, span_bytes_dev(t.exp_avg, t.numel, rep));
        x.cr[h] = load_codes<FULL>((const uint8_t*)t.exp_avg_sq + base + i, size - i, span_bytes_dev(t.exp_avg_sq, t.numel, rep));
    }
    (void)scales;
}
template <typename TP, typename TG, bool FULL>
__device__ __forceinline__ void step_block(const trop_adamw_tensor& t, int64_t base, int size, const AdamwScalars& k,
                                           int copy16, unsigned* rep, const Block8<TP, TG>& x)
{
    const int lane = threadIdx.x & 31;
    float m[2][4], r[2][4];
    uint32_t mtop = 0, rtop = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = h * 128 + lane * 4;
        float p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float a = byte_to_f32<true>(x.cm[h], q), c = byte_to_f32<false>(x.cr[h], q);
            m[h][q] = __fmul_rn(__fmul_rn(a, fabsf(a)), x.ms);
            const float root = __fmul_rn(__fmul_rn(c, c), x.rs);
            float v = __fmul_rn(root, root);
            p[q] = x.p[h].get(q);
            step1(p[q], x.g[h].get(q), m[h][q], v, r[h][q], k);
            if (FULL || i + q < size) {
                mtop = max(mtop, __float_as_uint(m[h][q]) & 0x7fffffffu);
                rtop = max(rtop, __float_as_uint(r[h][q]) & 0x7fffffffu);
            }
        }
        store_param<TP, FULL>(t, base, i, size - i, rep, copy16, p);
    }
    const float mt = __uint_as_float(__reduce_max_sync(0xffffffffu, mtop));
    const float rt = __uint_as_float(__reduce_max_sync(0xffffffffu, rtop));
    const float mi = mt > 0.f ? __fdiv_rn(1.f, mt) : 0.f, ri = rt > 0.f ? __fdiv_rn(1.f, rt) : 0.f;
    float xm[2][4], xr[2][4], off = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            xm[h][q] = code_of(fminf(__fmul_rn(fabsf(m[h][q]), mi), 1.f), 127.f, off);
            xr[h][q] = code_of(fminf(__fmul_rn(r[h][q], ri), 1.f), 255.f, off);
        }
    if (off > 0.5f - NEAR) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                xm[h][q] = code_exact(fminf(__fmul_rn(fabsf(m[h][q]), mi), 1.f), 127.f);
                xr[h][q] = code_exact(fminf(__fmul_rn(r[h][q], ri), 1.f), 255.f);
            }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = h * 128 + lane * 4;
        uint32_t wm[4], wr[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            wm[q] = __float_as_uint(copysignf(xm[h][q] - TO_WHOLE, m[h][q]) + TO_WHOLE);
            wr[q] = __float_as_uint(xr[h][q]);
            if (r[h][q] > 0.f) wr[q] = max(wr[q], __float_as_uint(TO_WHOLE + 1.f));
        }
        store_codes<FULL>((uint8_t*)t.exp_avg + base + i, size - i, span_bytes_dev(t.exp_avg, t.numel, rep), low_bytes(wm));
        store_codes<FULL>((uint8_t*)t.exp_avg_sq + base + i, size - i, span_bytes_dev(t.exp_avg_sq, t.numel, rep), low_bytes(wr));
    }
    if (lane == 0) {
        const int64_t scales = (t.numel + BLOCK - 1) / BLOCK * 4;
        float* ps = t.exp_avg_scale + base / BLOCK;
        float* qs = t.exp_avg_sq_scale + base / BLOCK;
        if (TROP_IN(ps, 4, span_bytes_dev(t.exp_avg_scale, scales, rep))) *ps = mt < INFINITY ? __fmul_rn(mt, 1.f / 16129.f) : NAN;
        if (TROP_IN(qs, 4, span_bytes_dev(t.exp_avg_sq_scale, scales, rep))) *qs = rt < INFINITY ? __fmul_rn(rt, 1.f / 65025.f) : NAN;
        (void)scales;
    }
}
template <typename TP, typename TG, typename TAB>
__global__ void __launch_bounds__(256, 4)
    k_adamw8(const __grid_constant__ TAB tab, const AdamwScalars k, int copy16)
{
    const Entry<trop_adamw_tensor>& x = tab.of(blockIdx.x);
    const int64_t base = (int64_t)(blockIdx.x - x.start) * CHUNK + (threadIdx.x >> 5) * BLOCK, left = x.e.numel - base;
    constexpr int APART = CHUNK / 2;  // a warp's two blocks, both on their way before either is worked on
    pdl_wait();  // (the table is older than the kernel before)
    pdl_signal();
    if (x.vec && left >= APART + BLOCK) {
        Block8<TP, TG> a, b;
        load_block<TP, TG, true>(x.e, base, BLOCK, tab.rep, a);
        load_block<TP, TG, true>(x.e, base + APART, BLOCK, tab.rep, b);
        step_block<TP, TG, true>(x.e, base, BLOCK, k, copy16, tab.rep, a);
        step_block<TP, TG, true>(x.e, base + APART, BLOCK, k, copy16, tab.rep, b);
        return;
    }
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        const int64_t size = left - h * APART;
        if (size <= 0) break;
        Block8<TP, TG> a;
        load_block<TP, TG, false>(x.e, base + h * APART, (int)min(size, (int64_t)BLOCK), tab.rep, a);
        step_block<TP, TG, false>(x.e, base + h * APART, (int)min(size, (int64_t)BLOCK), k, copy16, tab.rep, a);
    }
}

// 8-bit states as the values they stand for
template <bool FULL>
__device__ __forceinline__ void values_chunk(const trop_adamw_state& t, int64_t base, int size, unsigned* rep)
{
    const uint8_t* pm = (const uint8_t*)t.exp_avg + base;
    const uint8_t* pr = (const uint8_t*)t.exp_avg_sq + base;
    const float* ps = t.exp_avg_scale + base / BLOCK;
    const float* qs = t.exp_avg_sq_scale + base / BLOCK;
    const Span sp_m = span_bytes_dev(t.exp_avg, t.numel, rep), sp_r = span_bytes_dev(t.exp_avg_sq, t.numel, rep);
    const int64_t scales = (t.numel + BLOCK - 1) / BLOCK * 4;
    const Span sp_ms = span_bytes_dev(t.exp_avg_scale, scales, rep), sp_rs = span_bytes_dev(t.exp_avg_sq_scale, scales, rep);
    const Span sp_a = span_bytes_dev(t.exp_avg_value, t.numel * 4, rep), sp_b = span_bytes_dev(t.exp_avg_sq_value, t.numel * 4, rep);
    (void)sp_ms, (void)sp_rs;
    const int i0 = threadIdx.x * 4;
    uint32_t cm[4], cr[4];
    float ms[4], rs[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 1024;
        if (!FULL && i >= size) continue;
        cm[u] = load_codes<FULL>(pm + i, size - i, sp_m);
        cr[u] = load_codes<FULL>(pr + i, size - i, sp_r);
        ms[u] = TROP_IN(ps + i / BLOCK, 4, sp_ms) ? ps[i / BLOCK] : 0.f;
        rs[u] = TROP_IN(qs + i / BLOCK, 4, sp_rs) ? qs[i / BLOCK] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * 1024;
        if (!FULL && i >= size) continue;
        float m[4], v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float a = byte_to_f32<true>(cm[u], q), c = byte_to_f32<false>(cr[u], q);
            m[q] = __fmul_rn(__fmul_rn(a, fabsf(a)), ms[u]);
            const float r = __fmul_rn(__fmul_rn(c, c), rs[u]);
            v[q] = __fmul_rn(r, r);
        }
        store4<float, FULL>(t.exp_avg_value + base + i, size - i, sp_a, m);
        store4<float, FULL>(t.exp_avg_sq_value + base + i, size - i, sp_b, v);
    }
}
template <typename TAB>
__global__ void __launch_bounds__(256) k_adamw_values(const __grid_constant__ TAB tab)
{
    const Entry<trop_adamw_state>& x = tab.of(blockIdx.x);
    pdl_wait();  // (the table is older than the kernel before)
    pdl_signal();
    const int64_t base = (int64_t)(blockIdx.x - x.start) * CHUNK, left = x.e.numel - base;
    if (x.vec && left >= CHUNK) values_chunk<true>(x.e, base, CHUNK, tab.rep);
    else values_chunk<false>(x.e, base, (int)min(left, (int64_t)CHUNK), tab.rep);
}

// ------------------------------------------------------------------ host
bool on(const void* p, size_t bytes) { return ((uintptr_t)p % bytes) == 0; }

bool is_vec(const trop_adamw_tensor& t, size_t pb, size_t gb, size_t sb)
{
    return on(t.param, 4 * pb) && on(t.grad, 4 * gb) && on(t.exp_avg, 4 * sb) && on(t.exp_avg_sq, 4 * sb) && on(t.copy, 8);
}

// Small tables for few tensors: a launch carries its table, and 3 KB cost less than 30.
constexpr int FEW = 28, MANY = 380;
constexpr int64_t MOST_CHUNKS = INT32_MAX;

unsigned* record()
{
#if TROP_DEBUG_BOUNDS
    return bounds_record();
#else
    return nullptr;
#endif
}

template <typename KERNEL, typename... A>
int launch_chunks(KERNEL kernel, int64_t chunks, cudaStream_t s, const A&... a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<void*>(static_cast<const void*>(&a))...};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
    if (e != cudaSuccess) return cuda_error(e, "AdamW launch");
    count_launches(1);
    return TROP_OK;
}

// Entries from e[*i] on, until `most` of them or a grid's chunks are taken: go(index, entry).
template <typename E, typename VEC, typename GO>
int take(int64_t n, const E* e, int64_t* i, int64_t most, VEC vec, int64_t* chunks, GO go)
{
    *chunks = 0;
    int64_t k = 0;
    for (; *i < n && k < most; ++*i) {
        const int64_t c = (e[*i].numel + CHUNK - 1) / CHUNK;
        if (c == 0) continue;
        if (c > MOST_CHUNKS) return set_error(TROP_ERR_UNSUPPORTED, "a tensor of %lld elements", (long long)e[*i].numel);
        if (*chunks + c > MOST_CHUNKS) break;
        go(k++, Entry<E>{e[*i], (uint32_t)*chunks, (uint32_t)vec(e[*i])}, c);
        *chunks += c;
    }
    return TROP_OK;
}

// All tensors through tables in the launches' parameters.
template <int CAP, typename E, typename VEC, typename GO>
int in_tables(int64_t n, const E* e, VEC vec, GO go)
{
    Table<E, CAP> tab;
    tab.rep = record();
    for (int64_t i = 0; i < n;) {
        int64_t chunks;
        tab.n = 0;
        TROP_TRY(take(n, e, &i, CAP, vec, &chunks, [&](int64_t k, const Entry<E>& x, int64_t) {
            tab.e[k] = x;
            tab.start[k] = x.start;
            tab.n = (int)k + 1;
        }));
        if (tab.n) TROP_TRY(go(tab, chunks));
    }
    return TROP_OK;
}

// All tensors laid out in one device allocation: per launch, its entries and its chunks' numbers.
template <typename E>
struct Laid {
    struct Part {
        Resident<E> tab;
        int64_t chunks;
    };
    std::vector<Part> parts;
    void* memory = nullptr;
    ~Laid()
    {
        if (memory) cudaFree(memory);
    }
    template <typename VEC>
    int fill(int64_t n, const E* e, VEC vec)
    {
        struct Host {
            std::vector<Entry<E>> e;
            std::vector<uint32_t> chunk;
        };
        std::vector<Host> host;
        size_t bytes = 0;
        for (int64_t i = 0; i < n;) {
            Host h;
            int64_t chunks;
            TROP_TRY(take(n, e, &i, INT32_MAX, vec, &chunks, [&](int64_t k, const Entry<E>& x, int64_t c) {
                h.e.push_back(x);
                h.chunk.insert(h.chunk.end(), (size_t)c, (uint32_t)k);
            }));
            if (h.e.empty()) continue;
            bytes += h.e.size() * sizeof(Entry<E>) + (h.chunk.size() * 4 + 15) / 16 * 16;
            host.push_back(std::move(h));
        }
        if (!bytes) return TROP_OK;
        std::vector<uint8_t> image(bytes);
        cudaError_t err = cudaMalloc(&memory, bytes);
        if (err != cudaSuccess) {
            cudaGetLastError();
            memory = nullptr;
            return set_error(TROP_ERR_OOM, "%zu bytes for the plan's table: %s", bytes, cudaGetErrorString(err));
        }
        size_t at = 0;
        for (const Host& h : host) {
            Part p;
            p.tab.rep = record();
            p.tab.e = (const Entry<E>*)((uint8_t*)memory + at);
            memcpy(&image[at], h.e.data(), h.e.size() * sizeof(Entry<E>));
            at += h.e.size() * sizeof(Entry<E>);
            p.tab.chunk = (const uint32_t*)((uint8_t*)memory + at);
            memcpy(&image[at], h.chunk.data(), h.chunk.size() * 4);
            at += (h.chunk.size() * 4 + 15) / 16 * 16;
            p.chunks = (int64_t)h.chunk.size();
            parts.push_back(p);
        }
        // The table is in device memory before the plan is handed out: its steps run on any stream, and read it
        // before they wait for the kernel ahead of them.  (A plain copy from pageable memory may return
        // while its last part is still on its way, in order with the legacy stream only.)
        cudaStream_t up = nullptr;
        err = cudaStreamCreateWithFlags(&up, cudaStreamNonBlocking);
        if (err != cudaSuccess) return cuda_error(err, "cudaStreamCreateWithFlags (the plan's table)");
        err = cudaMemcpyAsync(memory, image.data(), bytes, cudaMemcpyHostToDevice, up);
        const cudaError_t done = cudaStreamSynchronize(up);  // also before `image` goes
        cudaStreamDestroy(up);
        if (err == cudaSuccess) err = done;
        return err == cudaSuccess ? (int)TROP_OK : cuda_error(err, "copy of the plan's table");
    }
};

bool is_vec_state(const trop_adamw_state& x)
{
    return on(x.exp_avg, 4) && on(x.exp_avg_sq, 4) && on(x.exp_avg_value, 16) && on(x.exp_avg_sq_value, 16);
}

template <typename TP, typename TG, typename TAB>
int step_table(const TAB& tab, int64_t chunks, int state8, int copy16, const AdamwScalars& k, cudaStream_t s)
{
    return state8 ? launch_chunks(k_adamw8<TP, TG, TAB>, chunks, s, tab, k, copy16)
                  : launch_chunks(k_adamw<TP, TG, TAB>, chunks, s, tab, k, copy16);
}

// f(TP, TG) for the types' codes
template <typename F>
int by_types(int pdtype, int gdtype, F f)
{
    using bf16 = __nv_bfloat16;
    if (pdtype == TROP_F32) return gdtype == TROP_F32 ? f(0.f, 0.f) : gdtype == TROP_BF16 ? f(0.f, bf16()) : f(0.f, __half());
    if (pdtype == TROP_BF16) return gdtype == TROP_F32 ? f(bf16(), 0.f) : f(bf16(), bf16());
    return gdtype == TROP_F32 ? f(__half(), 0.f) : f(__half(), __half());
}

}  // namespace

struct AdamwTables {
    int pdtype, gdtype, state8, copy16;
    // few tensors: a table for the launches' parameters; more: in device memory
    std::vector<std::pair<Table<trop_adamw_tensor, FEW>, int64_t>> few;
    std::vector<std::pair<Table<trop_adamw_state, FEW>, int64_t>> few_states;
    Laid<trop_adamw_tensor> tensors;
    Laid<trop_adamw_state> states;
};
AdamwTables* adamw_tables() { return new AdamwTables(); }
void adamw_tables_free(AdamwTables* t) { delete t; }

int adamw_tables_fill(AdamwTables* a, int64_t n, const trop_adamw_tensor* t, int pdtype, int gdtype, int state8,
                      int copy_dtype)
{
    a->pdtype = pdtype;
    a->gdtype = gdtype;
    a->state8 = state8;
    a->copy16 = copy_dtype == TROP_F16 ? 2 : 1;
    const size_t pb = model_bytes(pdtype), gb = model_bytes(gdtype), sb = state8 ? 1 : 4;
    auto vec = [=](const trop_adamw_tensor& x) { return is_vec(x, pb, gb, sb); };
    if (n > FEW) return a->tensors.fill(n, t, vec);
    return in_tables<FEW>(n, t, vec, [&](const Table<trop_adamw_tensor, FEW>& tab, int64_t chunks) {
        a->few.emplace_back(tab, chunks);
        return (int)TROP_OK;
    });
}
int adamw_states_fill(AdamwTables* a, int64_t n, const trop_adamw_state* t)
{
    if (n > FEW) return a->states.fill(n, t, is_vec_state);
    return in_tables<FEW>(n, t, is_vec_state, [&](const Table<trop_adamw_state, FEW>& tab, int64_t chunks) {
        a->few_states.emplace_back(tab, chunks);
        return (int)TROP_OK;
    });
}

int launch_adamw_plan(const AdamwTables& a, const AdamwScalars& k, cudaStream_t s)
{
    return by_types(a.pdtype, a.gdtype, [&](auto tp, auto tg) {
        for (const auto& p : a.few)
            TROP_TRY((step_table<decltype(tp), decltype(tg)>(p.first, p.second, a.state8, a.copy16, k, s)));
        for (const auto& p : a.tensors.parts)
            TROP_TRY((step_table<decltype(tp), decltype(tg)>(p.tab, p.chunks, a.state8, a.copy16, k, s)));
        return (int)TROP_OK;
    });
}
int launch_adamw_plan_values(const AdamwTables& a, cudaStream_t s)
{
    for (const auto& p : a.few_states)
        TROP_TRY((launch_chunks(k_adamw_values<Table<trop_adamw_state, FEW>>, p.second, s, p.first)));
    for (const auto& p : a.states.parts) TROP_TRY(launch_chunks(k_adamw_values<Resident<trop_adamw_state>>, p.chunks, s, p.tab));
    return TROP_OK;
}

int launch_adamw(int64_t n, const trop_adamw_tensor* t, int pdtype, int gdtype, int state8, int copy_dtype,
                 const AdamwScalars& k, cudaStream_t s)
{
    const int copy16 = copy_dtype == TROP_F16 ? 2 : 1;
    return by_types(pdtype, gdtype, [&](auto tp, auto tg) {
        using TP = decltype(tp);
        using TG = decltype(tg);
        auto vec = [&](const trop_adamw_tensor& x) { return is_vec(x, sizeof(TP), sizeof(TG), state8 ? 1 : 4); };
        auto go = [&](const auto& tab, int64_t chunks) { return step_table<TP, TG>(tab, chunks, state8, copy16, k, s); };
        return n <= FEW ? in_tables<FEW>(n, t, vec, go) : in_tables<MANY>(n, t, vec, go);
    });
}
int launch_adamw_values(int64_t n, const trop_adamw_state* t, cudaStream_t s)
{
    auto go = [&](const auto& tab, int64_t chunks) {
        return launch_chunks(k_adamw_values<std::decay_t<decltype(tab)>>, chunks, s, tab);
    };
    return n <= FEW ? in_tables<FEW>(n, t, is_vec_state, go) : in_tables<MANY>(n, t, is_vec_state, go);
}

}  // namespace trop
