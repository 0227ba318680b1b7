// rows.h -- what the kernels over rows share (layer_norm.cu, residual_norm.cu): vectors of a row worked on in
// packed f32 pairs, sums over the group of threads that has a row, bulk copies into a ring, launches.
// Included once TROP_TU names the file's id.
#pragma once

#include <cuda_runtime.h>

#include <mutex>
#include <set>
#include <type_traits>
#include <utility>

#include "internal.h"
#include "packed.h"

namespace trop {
namespace {

// VEC elements that lie together, one access where they make 16 (or 8) bytes
template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float (&v)[VEC], const Span& sp)
{
    (void)sp;
    Raw<T, VEC> q;
    if (TROP_IN(p, VEC * sizeof(T), sp)) q.read(p);
    else q.zero();
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = q.get(i);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float (&v)[VEC], const Span& sp)
{
    (void)sp;
    Raw<T, VEC> q;
    q.set(v);
    if (TROP_IN(p, VEC * sizeof(T), sp)) q.write(p);
}

// Elements are worked on two at a time (packed f32 operations: with 16-bit rows the instructions per
// element, not memory, would bound these kernels); where elements come one by one, one at a time.
template <int VEC>
constexpr int pairs = VEC >= 2 ? VEC / 2 : 1;
template <int VEC>
using Pair = std::conditional_t<(VEC >= 2), float2, float>;
__device__ __forceinline__ float2 p_add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 p_mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 p_fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float p_sum(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float p_add(float a, float b) { return a + b; }
__device__ __forceinline__ float p_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float p_fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ float p_sum(float a) { return a; }
template <typename P>
__device__ __forceinline__ P p_of(float v)
{
    if constexpr (sizeof(P) == 8) return make_float2(v, v);
    else return v;
}
template <typename T, int VEC>
__device__ __forceinline__ Pair<VEC> pair_of(const Raw<T, VEC>& q, int i)
{
    if constexpr (VEC >= 2) return make_float2(q.get(2 * i), q.get(2 * i + 1));
    else return q.get(0);
}
template <int VEC>
__device__ __forceinline__ Pair<VEC> pair_at(const float (&v)[VEC], int i)
{
    if constexpr (VEC >= 2) return make_float2(v[2 * i], v[2 * i + 1]);
    else return v[0];
}
template <int VEC>
__device__ __forceinline__ void apart(const Pair<VEC> (&o)[pairs<VEC>], float (&v)[VEC])
{
    if constexpr (VEC >= 2) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i % 2 ? o[i / 2].y : o[i / 2].x;
    } else {
        v[0] = o[0];
    }
}
// Sums of K values over the group of a row: a warp (several rows per block), or the whole block.
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float (*sh)[K])
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (blockDim.x == 32) return;
    const int warps = blockDim.x >> 5;
    __syncthreads();  // the shared sums of the call before have been read
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) sh[threadIdx.x >> 5][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += sh[w][k];
}

template <int K>
__device__ __forceinline__ void warp_sum(float (&v)[K])
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}
// The same over a row's group with one barrier: callers alternate between two of `sh`.
template <int K>
__device__ __forceinline__ void group_sum_turn(float (&v)[K], float (*sh)[K])
{
    warp_sum<K>(v);
    if (blockDim.x == 32) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) sh[threadIdx.x >> 5][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += sh[w][k];
}
// `bytes` (a multiple of 16) between 16-byte boundaries, counted by the mbarrier
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

constexpr int RING_STAGES = 8;
// A copy did not land within its bounded wait: say so, and wait (bounded) for the others before the
// block leaves.
__device__ inline void ring_failed(uint64_t* full, int stages, int s, uint32_t phase, uint32_t* error)
{
    if (threadIdx.x != 0) return;
    *(volatile uint32_t*)error = 1;
    __threadfence_system();
    for (int i = 0; i < stages; ++i) {
        (void)mbar_wait(&full[s], phase);
        if (++s == stages) s = 0, phase ^= 1;
    }
}

// ------------------------------------------------------------------ host
inline bool aligned(const void* p, int64_t stride, size_t elem, int vec, int64_t rows)
{
    return !p || (((uintptr_t)p % (elem * vec)) == 0 && (rows <= 1 || stride % vec == 0));
}

#define TROP_LAUNCH(kernel, grid, block, smem, ...)                                   \
    do {                                                                              \
        const cudaError_t e_ = launch_pdl(kernel, grid, block, smem, s, __VA_ARGS__); \
        if (e_ != cudaSuccess) return cuda_error(e_, #kernel " launch");              \
        count_launches(1);                                                            \
    } while (0)

// Dynamic shared memory that needs no attribute: a block has 48 KB in all without it, of which static arrays take
// up to 2 KB (sh[2][32][8]).
constexpr size_t PLAIN_SMEM = 49152 - 2048;
// More of it.  The limit is state of the function, which every host thread shares: it is raised once for a kernel and
// a device, to all that the device has, and never set to one call's need, which another thread's smaller
// one could take back before the launch.
inline int allow_dynamic(const void* kernel)
{
    struct Raised {
        std::mutex mu;
        std::set<std::pair<int, const void*>> kernels;
    };
    static Raised* const raised = new Raised();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_error(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lk(raised->mu);
    if (raised->kernels.count({dev, kernel})) return TROP_OK;
    int most = 0;
    cudaFuncAttributes a;
    e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kernel);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)a.sharedSizeBytes);
    if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute (rows)");
    try {
        raised->kernels.insert({dev, kernel});
    } catch (...) {  // no memory to write it down: asked for again next time
    }
    return TROP_OK;
}

}  // namespace
}  // namespace trop
