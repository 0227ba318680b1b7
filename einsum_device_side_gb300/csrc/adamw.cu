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
// an even code; r, not v, is what the update divides by, and no r > 0 is coded as 0, so a rounded
// state can damp an update but never blow it up.  The update itself uses the unrounded new m and v.
//
// The step moves 28 (f32) or 16 (8-bit, f32 parameters) bytes per element and is bound by memory.
// One launch covers hundreds of tensors: their addresses travel in the kernel's parameters, the
// grid has one block per 4096 elements of any tensor, and a block finds its tensor by bisection.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <vector>

#define TROP_TU 8  // this file's id in a bounds-violation record
#include "internal.h"
#include "train.h"

namespace trop {
namespace {

constexpr int CHUNK = 4096;   // elements of one block of threads
constexpr int BLOCK = 256;    // elements of one scale

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(int8_t v) { return (float)v; }
__device__ __forceinline__ float to_f32(uint8_t v) { return (float)v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ int8_t from_f32<int8_t>(float v) { return (int8_t)__float2int_rn(v); }
template <> __device__ __forceinline__ uint8_t from_f32<uint8_t>(float v) { return (uint8_t)__float2int_rn(v); }

template <typename T>
struct alignas(4 * sizeof(T)) Four {
    T e[4];
};

// Elements i .. i + 3 of a tensor of n: one access where the tensor is aligned and all four exist.
template <typename T>
__device__ __forceinline__ void load4(const void* base, int64_t i, int64_t n, bool vec, unsigned* rep, float (&v)[4])
{
    const T* p = (const T*)base + i;
    const Span sp = span_bytes_dev(base, n * sizeof(T), rep);
    if (vec && i + 4 <= n) {
        if (TROP_IN(p, 4 * sizeof(T), sp)) {
            const Four<T> q = *reinterpret_cast<const Four<T>*>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = to_f32(q.e[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k < n && TROP_IN(p + k, sizeof(T), sp) ? to_f32(p[k]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store4(void* base, int64_t i, int64_t n, bool vec, unsigned* rep, const float (&v)[4])
{
    T* p = (T*)base + i;
    const Span sp = span_bytes_dev(base, n * sizeof(T), rep);
    if (vec && i + 4 <= n) {
        Four<T> q;
#pragma unroll
        for (int k = 0; k < 4; ++k) q.e[k] = from_f32<T>(v[k]);
        if (TROP_IN(p, 4 * sizeof(T), sp)) *reinterpret_cast<Four<T>*>(p) = q;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n && TROP_IN(p + k, sizeof(T), sp)) p[k] = from_f32<T>(v[k]);
    }
}

// The tensors of one launch: chunk c belongs to the tensor i with start[i] <= c < start[i + 1].
template <typename E, int CAP>
struct Table {
    int n;
    unsigned* rep;  // the bounds-checked build's record
    uint32_t start[CAP + 1];
    uint8_t vec[CAP];
    E e[CAP];
};
template <typename TAB>
__device__ __forceinline__ int tensor_of(const TAB& t, uint32_t chunk)
{
    int lo = 0, hi = t.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.start[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

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

// `copy16`: a 16-bit copy of f32 parameters is written beside them (0 none, 1 bf16, 2 f16)
template <typename TP>
__device__ __forceinline__ void store_param(const trop_adamw_tensor& t, int64_t i, bool vec, unsigned* rep, int copy16,
                                            const float (&p)[4])
{
    store4<TP>(t.param, i, t.numel, vec, rep, p);
    if (sizeof(TP) == 4 && t.copy) {
        if (copy16 == 1) store4<__nv_bfloat16>(t.copy, i, t.numel, vec, rep, p);
        else store4<__half>(t.copy, i, t.numel, vec, rep, p);
    }
}

template <typename TP, typename TG, int CAP>
__global__ void __launch_bounds__(256)
    k_adamw(const __grid_constant__ Table<trop_adamw_tensor, CAP> tab, const AdamwScalars k, int copy16)
{
    pdl_wait();
    pdl_signal();
    const int at = tensor_of(tab, blockIdx.x);
    const trop_adamw_tensor& t = tab.e[at];
    const bool vec = tab.vec[at];
    const int64_t n = t.numel, i0 = (int64_t)(blockIdx.x - tab.start[at]) * CHUNK + threadIdx.x * 4;
    float p[4][4], g[4][4], m[4][4], v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * 1024;
        if (i >= n) continue;
        load4<TP>(t.param, i, n, vec, tab.rep, p[u]);
        load4<TG>(t.grad, i, n, vec, tab.rep, g[u]);
        load4<float>(t.exp_avg, i, n, vec, tab.rep, m[u]);
        load4<float>(t.exp_avg_sq, i, n, vec, tab.rep, v[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * 1024;
        if (i >= n) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float r;
            step1(p[u][q], g[u][q], m[u][q], v[u][q], r, k);
        }
        store_param<TP>(t, i, vec, tab.rep, copy16, p[u]);
        store4<float>(t.exp_avg, i, n, vec, tab.rep, m[u]);
        store4<float>(t.exp_avg_sq, i, n, vec, tab.rep, v[u]);
    }
}

// A warp per block of 256: lane l has elements 4 l .. and 128 + 4 l .., so that every access of the
// warp is contiguous.  The largest magnitude is taken over the values' bits, which order like the
// magnitudes and let a NaN win: a block with a NaN or an infinity has a scale that is not finite,
// and all of it reads back as NaN.
template <typename TP, typename TG, int CAP>
__global__ void __launch_bounds__(256)
    k_adamw8(const __grid_constant__ Table<trop_adamw_tensor, CAP> tab, const AdamwScalars k, int copy16)
{
    pdl_wait();
    pdl_signal();
    const int at = tensor_of(tab, blockIdx.x);
    const trop_adamw_tensor& t = tab.e[at];
    const bool vec = tab.vec[at];
    const int64_t n = t.numel;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Span sp_ms = span_bytes_dev(t.exp_avg_scale, (n + BLOCK - 1) / BLOCK * 4, tab.rep);
    const Span sp_vs = span_bytes_dev(t.exp_avg_sq_scale, (n + BLOCK - 1) / BLOCK * 4, tab.rep);
    float p[2][2][4], g[2][2][4], m[2][2][4], v[2][2][4], ms[2], vs[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int64_t block = (int64_t)(blockIdx.x - tab.start[at]) * (CHUNK / BLOCK) + b * 8 + warp;
        if (block * BLOCK >= n) continue;
        ms[b] = TROP_IN(t.exp_avg_scale + block, 4, sp_ms) ? t.exp_avg_scale[block] : 0.f;
        vs[b] = TROP_IN(t.exp_avg_sq_scale + block, 4, sp_vs) ? t.exp_avg_sq_scale[block] : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = block * BLOCK + h * 128 + lane * 4;
            load4<TP>(t.param, i, n, vec, tab.rep, p[b][h]);
            load4<TG>(t.grad, i, n, vec, tab.rep, g[b][h]);
            load4<int8_t>(t.exp_avg, i, n, vec, tab.rep, m[b][h]);
            load4<uint8_t>(t.exp_avg_sq, i, n, vec, tab.rep, v[b][h]);
        }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int64_t block = (int64_t)(blockIdx.x - tab.start[at]) * (CHUNK / BLOCK) + b * 8 + warp;
        if (block * BLOCK >= n) continue;
        float r[2][4];
        uint32_t mtop = 0, rtop = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = block * BLOCK + h * 128 + lane * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float& mm = m[b][h][q];
                const float c = v[b][h][q];
                mm = __fmul_rn(__fmul_rn(mm, fabsf(mm)), ms[b]);
                const float root = __fmul_rn(__fmul_rn(c, c), vs[b]);
                float vv = __fmul_rn(root, root);
                step1(p[b][h][q], g[b][h][q], mm, vv, r[h][q], k);
                if (i + q < n) {
                    mtop = max(mtop, __float_as_uint(mm) & 0x7fffffffu);
                    rtop = max(rtop, __float_as_uint(r[h][q]) & 0x7fffffffu);
                }
            }
            store_param<TP>(t, i, vec, tab.rep, copy16, p[b][h]);
        }
        const float mt = __uint_as_float(__reduce_max_sync(0xffffffffu, mtop));
        const float rt = __uint_as_float(__reduce_max_sync(0xffffffffu, rtop));
        const float mi = mt > 0.f ? __fdiv_rn(1.f, mt) : 0.f, ri = rt > 0.f ? __fdiv_rn(1.f, rt) : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = block * BLOCK + h * 128 + lane * 4;
            float cm[4], cv[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float a = m[b][h][q], z = r[h][q];
                cm[q] = copysignf(rintf(__fmul_rn(__fsqrt_rn(fminf(__fmul_rn(fabsf(a), mi), 1.f)), 127.f)), a);
                cv[q] = rintf(__fmul_rn(__fsqrt_rn(fminf(__fmul_rn(z, ri), 1.f)), 255.f));
                if (z > 0.f) cv[q] = fmaxf(cv[q], 1.f);
            }
            store4<int8_t>(t.exp_avg, i, n, vec, tab.rep, cm);
            store4<uint8_t>(t.exp_avg_sq, i, n, vec, tab.rep, cv);
        }
        if (lane == 0) {
            if (TROP_IN(t.exp_avg_scale + block, 4, sp_ms)) t.exp_avg_scale[block] = __fmul_rn(mt, 1.f / 16129.f);
            if (TROP_IN(t.exp_avg_sq_scale + block, 4, sp_vs)) t.exp_avg_sq_scale[block] = __fmul_rn(rt, 1.f / 65025.f);
        }
    }
}

// 8-bit states as the values they stand for
template <int CAP>
__global__ void __launch_bounds__(256) k_adamw_values(const __grid_constant__ Table<trop_adamw_state, CAP> tab)
{
    pdl_wait();
    pdl_signal();
    const int at = tensor_of(tab, blockIdx.x);
    const trop_adamw_state& t = tab.e[at];
    const bool vec = tab.vec[at];
    const int64_t n = t.numel;
    const int64_t i0 = (int64_t)(blockIdx.x - tab.start[at]) * CHUNK + threadIdx.x * 4;
    const Span sp_ms = span_bytes_dev(t.exp_avg_scale, (n + BLOCK - 1) / BLOCK * 4, tab.rep);
    const Span sp_vs = span_bytes_dev(t.exp_avg_sq_scale, (n + BLOCK - 1) / BLOCK * 4, tab.rep);
    float m[4][4], v[4][4], ms[4], vs[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * 1024;
        if (i >= n) continue;
        load4<int8_t>(t.exp_avg, i, n, vec, tab.rep, m[u]);
        load4<uint8_t>(t.exp_avg_sq, i, n, vec, tab.rep, v[u]);
        ms[u] = TROP_IN(t.exp_avg_scale + i / BLOCK, 4, sp_ms) ? t.exp_avg_scale[i / BLOCK] : 0.f;
        vs[u] = TROP_IN(t.exp_avg_sq_scale + i / BLOCK, 4, sp_vs) ? t.exp_avg_sq_scale[i / BLOCK] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * 1024;
        if (i >= n) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            m[u][q] = __fmul_rn(__fmul_rn(m[u][q], fabsf(m[u][q])), ms[u]);
            const float r = __fmul_rn(__fmul_rn(v[u][q], v[u][q]), vs[u]);
            v[u][q] = __fmul_rn(r, r);
        }
        store4<float>(t.exp_avg_value, i, n, vec, tab.rep, m[u]);
        store4<float>(t.exp_avg_sq_value, i, n, vec, tab.rep, v[u]);
    }
}

// ------------------------------------------------------------------ host
bool on(const void* p, size_t bytes) { return ((uintptr_t)p % bytes) == 0; }

bool is_vec(const trop_adamw_tensor& t, size_t pb, size_t gb, size_t sb)
{
    return on(t.param, 4 * pb) && on(t.grad, 4 * gb) && on(t.exp_avg, 4 * sb) && on(t.exp_avg_sq, 4 * sb) && on(t.copy, 8);
}

// Small tables for few tensors: a launch carries its table, and 2 KB cost less than 30.
constexpr int FEW = 28, MANY = 440;

// The tables of a call: as many tensors in each as it holds, and one launch for each.
template <typename E, int CAP>
struct Tables {
    std::vector<Table<E, CAP>> t;
    template <typename VEC>
    int fill(int64_t n, const E* e, VEC vec)
    {
        constexpr int64_t MOST = INT32_MAX;
        int64_t i = 0;
        while (i < n) {
            t.emplace_back();
            Table<E, CAP>& tab = t.back();
#if TROP_DEBUG_BOUNDS
            tab.rep = bounds_record();
#else
            tab.rep = nullptr;
#endif
            int64_t chunks = 0;
            int k = 0;
            for (; i < n && k < CAP; ++i) {
                const int64_t c = (e[i].numel + CHUNK - 1) / CHUNK;
                if (c == 0) continue;
                if (c > MOST) return set_error(TROP_ERR_UNSUPPORTED, "a tensor of %lld elements", (long long)e[i].numel);
                if (chunks + c > MOST) break;
                tab.e[k] = e[i];
                tab.vec[k] = vec(e[i]);
                tab.start[k++] = (uint32_t)chunks;
                chunks += c;
            }
            tab.n = k;
            tab.start[k] = (uint32_t)chunks;
            if (k == 0) t.pop_back();
        }
        return TROP_OK;
    }
    template <typename GO>
    int run(GO go) const
    {
        for (const Table<E, CAP>& tab : t) {
            const cudaError_t e = go(tab, dim3(tab.start[tab.n]));
            if (e != cudaSuccess) return cuda_error(e, "AdamW launch");
            count_launches(1);
        }
        return TROP_OK;
    }
};

template <typename KERNEL, typename... A>
cudaError_t launch_table(KERNEL kernel, dim3 grid, cudaStream_t s, const A&... a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<void*>(static_cast<const void*>(&a))...};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
}

template <typename TP, typename TG, int CAP>
int run_step(const Tables<trop_adamw_tensor, CAP>& t, int state8, int copy16, const AdamwScalars& k, cudaStream_t s)
{
    return t.run([&](const Table<trop_adamw_tensor, CAP>& tab, dim3 grid) {
        return state8 ? launch_table(k_adamw8<TP, TG, CAP>, grid, s, tab, k, copy16)
                      : launch_table(k_adamw<TP, TG, CAP>, grid, s, tab, k, copy16);
    });
}

}  // namespace

struct AdamwTables {
    int pdtype, gdtype, state8, copy16;
    Tables<trop_adamw_tensor, FEW> few;
    Tables<trop_adamw_tensor, MANY> many;
    Tables<trop_adamw_state, FEW> few_states;
    Tables<trop_adamw_state, MANY> many_states;

    template <typename TP, typename TG>
    int step(const AdamwScalars& k, cudaStream_t s) const
    {
        TROP_TRY((run_step<TP, TG, FEW>(few, state8, copy16, k, s)));
        return run_step<TP, TG, MANY>(many, state8, copy16, k, s);
    }
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
    return n <= FEW ? a->few.fill(n, t, vec) : a->many.fill(n, t, vec);
}

int adamw_states_fill(AdamwTables* a, int64_t n, const trop_adamw_state* t)
{
    auto vec = [](const trop_adamw_state& x) {
        return on(x.exp_avg, 4) && on(x.exp_avg_sq, 4) && on(x.exp_avg_value, 16) && on(x.exp_avg_sq_value, 16);
    };
    return n <= FEW ? a->few_states.fill(n, t, vec) : a->many_states.fill(n, t, vec);
}

int launch_adamw(const AdamwTables& a, const AdamwScalars& k, cudaStream_t s)
{
    using bf16 = __nv_bfloat16;
    if (a.pdtype == TROP_F32)
        return a.gdtype == TROP_F32    ? a.step<float, float>(k, s)
               : a.gdtype == TROP_BF16 ? a.step<float, bf16>(k, s)
                                       : a.step<float, __half>(k, s);
    if (a.pdtype == TROP_BF16) return a.gdtype == TROP_F32 ? a.step<bf16, float>(k, s) : a.step<bf16, bf16>(k, s);
    return a.gdtype == TROP_F32 ? a.step<__half, float>(k, s) : a.step<__half, __half>(k, s);
}

int launch_adamw_values(const AdamwTables& a, cudaStream_t s)
{
    TROP_TRY(a.few_states.run([&](const Table<trop_adamw_state, FEW>& tab, dim3 grid) {
        return launch_table(k_adamw_values<FEW>, grid, s, tab);
    }));
    return a.many_states.run([&](const Table<trop_adamw_state, MANY>& tab, dim3 grid) {
        return launch_table(k_adamw_values<MANY>, grid, s, tab);
    });
}

}  // namespace trop
