// layer_norm.cu -- layer norm over the last axis, forward and backward.
//
//   mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps)
//   y  = (x - mean) rstd w + b                                     (per row)
//   with h = (x - mean) rstd and u = dy w:
//   dx = rstd (u - mean_c(u) - h mean_c(u h)),  dw = sum_r dy h,  db = sum_r dy.
//
// Rows of x, y, dy, dx in f32, bf16 or f16; every sum and statistic in f32 and one rounding per
// stored value.  The variance is taken of the centred values (a second pass over registers), not
// from sums of squares, so that a large mean costs no digits.
//
// Both directions are bound by memory: each reads its rows once, into registers.
//   k_norm          a row per group of 32 .. 1024 threads, each holding up to 16 vectors of it (16 bytes where
//                   the rows are aligned to them, else one element)
//   k_norm_short    short rows, many of them: a warp takes several at a time
//   k_norm_off      many rows that do not start on 16 bytes: whole vectors all the same, a block's rows all
//                   at one offset
//   k_norm_back, k_norm_back_off, k_norm_back_ring   the same backward; the ring brings the rows of x and dy
//                   by bulk copies ahead of their turn
//   k_norm_long, k_norm_back_long, k_norm_columns   rows longer than a block's registers: the row
//                   is walked again for each pass (it stays in L2)
// The weight's and bias's gradients are summed without atomics: a persistent block keeps the sums
// of its columns over all its rows and writes them once; k_norm_join adds the blocks'
// sums in block order, so results repeat bit for bit.
//
// Measured (device time, a copy runs at 6.8 TB/s):    forward               backward
//   16384x4096  f32                                   82 us, 6.6 TB/s       131 us, 6.2 TB/s
//   16384x4096  bf16                                  50 us, 5.4 TB/s        68 us, 5.9 TB/s
//   65536x256   f32                                   22 us, 6.1 TB/s        36 us, 5.5 TB/s
//   4096x16384  bf16                                  53 us, 5.1 TB/s       129 us, 3.1 TB/s (sums in shared memory)
//   65536x1001  f32 (rows off 16 bytes)              100 us, 5.3 TB/s       148 us, 5.3 TB/s
//   65536x1001  bf16                                  75 us, 3.5 TB/s       120 us, 3.3 TB/s
// With 16-bit rows the instructions per element come near the bound: they are worked on in packed pairs.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <set>
#include <type_traits>
#include <utility>

#define TROP_TU 7  // this file's id in a bounds-violation record
#include "internal.h"
#include "packed.h"
#include "train.h"

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
// one row's values: (x - mean)^2 summed, and the result
template <typename T, int VEC>
__device__ __forceinline__ Pair<VEC> squares(const Raw<T, VEC>& q, float mean, Pair<VEC> a)
{
#pragma unroll
    for (int i = 0; i < pairs<VEC>; ++i) {
        const Pair<VEC> d = p_add(pair_of<T, VEC>(q, i), p_of<Pair<VEC>>(-mean));
        a = p_fma(d, d, a);
    }
    return a;
}
template <typename TX, typename TY, int VEC>
__device__ __forceinline__ void normed(const Raw<TX, VEC>& q, float mean, float rstd, bool has_w, const float (&w)[VEC], bool has_b,
                                       const float (&b)[VEC], TY* y, const Span& sp)
{
    Pair<VEC> o[pairs<VEC>];
#pragma unroll
    for (int i = 0; i < pairs<VEC>; ++i) {
        o[i] = p_mul(p_add(pair_of<TX, VEC>(q, i), p_of<Pair<VEC>>(-mean)), p_of<Pair<VEC>>(rstd));
        if (has_w) o[i] = p_mul(o[i], pair_at<VEC>(w, i));
        if (has_b) o[i] = p_add(o[i], pair_at<VEC>(b, i));
    }
    float v[VEC];
    apart<VEC>(o, v);
    store<TY, VEC>(y, v, sp);
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
__device__ void ring_failed(uint64_t* full, int stages, int s, uint32_t phase, uint32_t* error)
{
    if (threadIdx.x != 0) return;
    *(volatile uint32_t*)error = 1;
    __threadfence_system();
    for (int i = 0; i < stages; ++i) {
        (void)mbar_wait(&full[s], phase);
        if (++s == stages) s = 0, phase ^= 1;
    }
}

struct NormJob {
    int64_t rows, cols;
    float inv_cols, eps;
    float n;  // cols
    const void *x, *dy, *w, *b;
    void *y, *dx;
    int64_t sx, sy, sdy, sdx;
    float *mean, *rstd;
    float *part_w, *part_b;  // [blocks][cols], null: not wanted
    Span sp_x, sp_y, sp_dy, sp_dx, sp_w, sp_b, sp_mean, sp_rstd, sp_pw, sp_pb;
};

// sum / n: the product with the rounded inverse alone misses a constant row's value by a last place, which the row's
// small deviation then magnifies.  One residual step makes it the nearest quotient (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990); a sum that is not finite stays as it is.  (The
// division itself costs short 16-bit rows 2 of 25 us.)
__device__ __forceinline__ float over_n(float sum, const NormJob& j)
{
    const float q = sum * j.inv_cols, better = __fmaf_rn(__fmaf_rn(-q, j.n, sum), j.inv_cols, q);
    return better == better ? better : q;
}

// Threads a block may have: where a thread holds more than 64 bytes of its row, registers allow 256.
template <typename T, int VEC, int NV>
constexpr int most_threads() { return VEC * NV * sizeof(T) <= 64 ? 1024 : 256; }

// One row in a group's registers: statistics, result.
template <typename TX, typename TY, typename TW, int VEC, int NV>
__device__ __forceinline__ void norm_row(const NormJob& j, int64_t row, Raw<TX, VEC> (&q)[NV], float (*sh)[32][1])
{
    const int cols = (int)j.cols;
    Pair<VEC> a = p_of<Pair<VEC>>(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) a = p_add(a, pair_of<TX, VEC>(q[k], i));
    float s[1] = {p_sum(a)};
    group_sum_turn<1>(s, sh[0]);
    const float mean = over_n(s[0], j);
    a = p_of<Pair<VEC>>(0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        q[k].again();
        if (c < cols) a = squares<TX, VEC>(q[k], mean, a);
    }
    s[0] = p_sum(a);
    group_sum_turn<1>(s, sh[1]);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(s[0], j.inv_cols, j.eps)));
    if (threadIdx.x == 0) {
        if (j.mean && TROP_IN(j.mean + row, 4, j.sp_mean)) j.mean[row] = mean;
        if (j.rstd && TROP_IN(j.rstd + row, 4, j.sp_rstd)) j.rstd[row] = rstd;
    }
    TY* y = (TY*)j.y + row * j.sy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (c < cols) {
            float w[VEC], b[VEC];
            q[k].again();
            if (j.w) load<TW, VEC>((const TW*)j.w + c, w, j.sp_w);
            if (j.b) load<TW, VEC>((const TW*)j.b + c, b, j.sp_b);
            normed<TX, TY, VEC>(q[k], mean, rstd, j.w, w, j.b, b, y + c, j.sp_y);
        }
    }
}

// Rows from global memory; a group that holds little of a row fetches its next row before it works
// on this one.
template <typename TX, typename TY, typename TW, int VEC, int NV>
__global__ void __launch_bounds__((most_threads<TX, VEC, NV>()),
                                  (most_threads<TX, VEC, NV>() == 1024 ? 1 : VEC * NV == 64 && sizeof(TX) == 2 ? 3 : 2))
    k_norm(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[2][32][1];
    constexpr bool AHEAD = VEC * NV * sizeof(TX) <= 32;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const int cols = (int)j.cols;
    auto fetch = [&](Raw<TX, VEC> (&q)[NV], int64_t row) {
        const TX* x = (const TX*)j.x + row * j.sx;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC;
            if (row < j.rows && c < cols && TROP_IN(x + c, VEC * sizeof(TX), j.sp_x)) q[k].read(x + c);
            else q[k].zero();
        }
    };
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    Raw<TX, VEC> q[NV], ahead[AHEAD ? NV : 1];
    if (AHEAD && row < j.rows) fetch(q, row);
    for (; row < j.rows; row += step) {
        if constexpr (AHEAD) {
            fetch(ahead, row + step);
            norm_row<TX, TY, TW, VEC, NV>(j, row, q, sh);
#pragma unroll
            for (int k = 0; k < NV; ++k) q[k] = ahead[k];
        } else {
            fetch(q, row);
            norm_row<TX, TY, TW, VEC, NV>(j, row, q, sh);
        }
    }
}

// Short rows, a warp per row and U of its rows at a time: U rows' loads are on their way together, and
// their sums' shuffles run side by side.
template <typename TX, typename TY, typename TW, int VEC, int NV, int U>
__global__ void __launch_bounds__(256, 4) k_norm_short(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    const int cols = (int)j.cols;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row0 < j.rows; row0 += step * U) {
        Raw<TX, VEC> q[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            const TX* x = (const TX*)j.x + row * j.sx;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * 32 + threadIdx.x) * VEC;
                if (row < j.rows && c < cols && TROP_IN(x + c, VEC * sizeof(TX), j.sp_x)) q[u][k].read(x + c);
                else q[u][k].zero();
            }
        }
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pair<VEC> a = p_of<Pair<VEC>>(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) a = p_add(a, pair_of<TX, VEC>(q[u][k], i));
            mean[u] = p_sum(a);
        }
        warp_sum<U>(mean);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[u] = over_n(mean[u], j);
            Pair<VEC> a = p_of<Pair<VEC>>(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if ((k * 32 + (int)threadIdx.x) * VEC < cols) a = squares<TX, VEC>(q[u][k], mean[u], a);
            rstd[u] = p_sum(a);
        }
        warp_sum<U>(rstd);
#pragma unroll
        for (int u = 0; u < U; ++u) rstd[u] = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(rstd[u], j.inv_cols, j.eps)));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * 32 + threadIdx.x) * VEC;
            if (c >= cols) continue;
            float w[VEC], b[VEC];
            if (j.w) load<TW, VEC>((const TW*)j.w + c, w, j.sp_w);
            if (j.b) load<TW, VEC>((const TW*)j.b + c, b, j.sp_b);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = row0 + u * step;
                if (row >= j.rows) break;
                normed<TX, TY, VEC>(q[u][k], mean[u], rstd[u], j.w, w, j.b, b, (TY*)j.y + row * j.sy + c, j.sp_y);
            }
        }
        if (threadIdx.x == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = row0 + u * step;
                if (row >= j.rows) break;
                if (j.mean && TROP_IN(j.mean + row, 4, j.sp_mean)) j.mean[row] = mean[u];
                if (j.rstd && TROP_IN(j.rstd + row, 4, j.sp_rstd)) j.rstd[row] = rstd[u];
            }
    }
}

// Rows that do not start on 16 bytes, as every row of an odd number of columns but one in VEC does: row r
// starts `off` elements into a 16-byte granule, and off repeats every `period` rows.  A block takes rows
// of one offset only, so that its threads' vectors, the granules of its rows, hold the same columns in
// all of them: thread's column c = vector * VEC - off.  A row's first and last vector may be partial; it
// is written element by element, so that nothing outside the row is touched.
struct Offset {
    int off, cls;
    int64_t first, step;  // of the block's rows: cls + period * (first + i * step)
};
template <typename T, int VEC>
__device__ __forceinline__ Offset offset_of(const void* base, int64_t stride, int period)
{
    Offset o;
    o.cls = blockIdx.x % period;
    o.off = (int)(((uintptr_t)((const T*)base + o.cls * stride) % 16) / sizeof(T));
    o.first = (int64_t)(blockIdx.x / period) * blockDim.y + threadIdx.y;
    o.step = (int64_t)(gridDim.x / period) * blockDim.y;
    return o;
}
template <int VEC>
__device__ __forceinline__ bool whole(int c, int cols) { return c >= 0 && c + VEC <= cols; }
template <typename T, int VEC>
__device__ __forceinline__ void load_part(const T* row, int c, int cols, float (&v)[VEC], const Span& sp)
{
    (void)sp;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const bool in = c + i >= 0 && c + i < cols && TROP_IN(row + c + i, sizeof(T), sp);
        v[i] = in ? to_f32(row[c + i]) : 0.f;
    }
}
// (Of 16-bit rows a granule inside the matrix is read whole and the neighbouring rows' elements are put to
// zero: forward of 65536x1001 bf16 94 us, element by element 118 us.  Of f32 rows, whose granules have four
// elements, that costs more registers than it saves: backward of 65536x1001 348 us, element by element 148 us.)
template <typename T, int VEC>
__device__ __forceinline__ void load_off(const T* row, int c, int cols, const T* begin, const T* end, Raw<T, VEC>& q,
                                         const Span& sp)
{
    (void)sp;
    if (sizeof(T) == 2 ? row + c >= begin && row + c + VEC <= end : whole<VEC>(c, cols)) {
        if (TROP_IN(row + c, VEC * sizeof(T), sp)) q.read(row + c);
        else q.zero();
        if (sizeof(T) == 2 && !whole<VEC>(c, cols)) {
            constexpr int E = 4 / sizeof(T);  // elements of a word
#pragma unroll
            for (int i = 0; i < Raw<T, VEC>::N; ++i) {
                uint32_t keep = 0;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (c + i * E + e >= 0 && c + i * E + e < cols) keep |= (E == 1 ? 0xffffffffu : 0xffffu) << 16 * e;
                q.w[i] &= keep;
            }
        }
    } else {
        float v[VEC];
        load_part<T, VEC>(row, c, cols, v, sp);
        q.set(v);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_off(T* row, int c, int cols, const float (&v)[VEC], const Span& sp)
{
    if (whole<VEC>(c, cols)) {
        store<T, VEC>(row + c, v, sp);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i >= 0 && c + i < cols && TROP_IN(row + c + i, sizeof(T), sp)) row[c + i] = from_f32<T>(v[i]);
    }
}

// U rows of a group at a time; the weight and bias lie in shared memory, moved by the block's offset.
template <typename T, typename TW, int VEC, int NV, int U>
__global__ void __launch_bounds__(NV == 4 ? 672 : 256) k_norm_off(const NormJob j, int period)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float sh[2][32][U];
    const int cols = (int)j.cols, span = (cols + VEC - 1 + VEC) / VEC * VEC;  // (off + cols at most)
    const Offset o = offset_of<T, VEC>(j.x, j.sx, period);
    const T* const end = (const T*)j.x + (j.rows - 1) * j.sx + cols;
    TW* sw = reinterpret_cast<TW*>(dyn);
    TW* sb = sw + span;
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < span; i += blockDim.x * blockDim.y) {
        const int c = i - o.off;
        const bool in = c >= 0 && c < cols;
        if (j.w) sw[i] = in && TROP_IN((const TW*)j.w + c, sizeof(TW), j.sp_w) ? ((const TW*)j.w)[c] : from_f32<TW>(0.f);
        if (j.b) sb[i] = in && TROP_IN((const TW*)j.b + c, sizeof(TW), j.sp_b) ? ((const TW*)j.b)[c] : from_f32<TW>(0.f);
    }
    __syncthreads();
    for (int64_t n = o.first; o.cls + period * n < j.rows; n += o.step * U) {
        Raw<T, VEC> q[U][NV];
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = o.cls + period * (n + u * o.step);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * blockDim.x + threadIdx.x) * VEC - o.off;
                if (row < j.rows && c < cols)
                    load_off<T, VEC>((const T*)j.x + row * j.sx, c, cols, (const T*)j.x, end, q[u][k], j.sp_x);
                else
                    q[u][k].zero();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pair<VEC> a = p_of<Pair<VEC>>(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) a = p_add(a, pair_of<T, VEC>(q[u][k], i));
            mean[u] = p_sum(a);
        }
        group_sum_turn<U>(mean, sh[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mean[u] = over_n(mean[u], j);
            Pair<VEC> a = p_of<Pair<VEC>>(0.f);
            float edge = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * blockDim.x + threadIdx.x) * VEC - o.off;
                if (whole<VEC>(c, cols)) {
                    a = squares<T, VEC>(q[u][k], mean[u], a);
                } else if (c < cols) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float d = c + i >= 0 && c + i < cols ? q[u][k].get(i) - mean[u] : 0.f;
                        edge = __fmaf_rn(d, d, edge);
                    }
                }
            }
            rstd[u] = p_sum(a) + edge;
        }
        group_sum_turn<U>(rstd, sh[1]);
#pragma unroll
        for (int u = 0; u < U; ++u) rstd[u] = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(rstd[u], j.inv_cols, j.eps)));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (k * blockDim.x + threadIdx.x) * VEC, c = at - o.off;
            if (c >= cols) continue;
            Raw<TW, VEC> w, b;
            if (j.w) w.read(sw + at);
            if (j.b) b.read(sb + at);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = o.cls + period * (n + u * o.step);
                if (row >= j.rows) break;
                Pair<VEC> r[pairs<VEC>];
                float v[VEC];
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) {
                    r[i] = p_mul(p_add(pair_of<T, VEC>(q[u][k], i), p_of<Pair<VEC>>(-mean[u])), p_of<Pair<VEC>>(rstd[u]));
                    if (j.w) r[i] = p_mul(r[i], pair_of<TW, VEC>(w, i));
                    if (j.b) r[i] = p_add(r[i], pair_of<TW, VEC>(b, i));
                }
                apart<VEC>(r, v);
                store_off<T, VEC>((T*)j.y + row * j.sy, c, cols, v, j.sp_y);
            }
        }
        if (threadIdx.x == 0)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = o.cls + period * (n + u * o.step);
                if (row >= j.rows) break;
                if (j.mean && TROP_IN(j.mean + row, 4, j.sp_mean)) j.mean[row] = mean[u];
                if (j.rstd && TROP_IN(j.rstd + row, 4, j.sp_rstd)) j.rstd[row] = rstd[u];
            }
    }
}

// Rows longer than a block's registers: one block per row, three walks over it.
template <typename TX, typename TY, typename TW>
__global__ void __launch_bounds__(1024) k_norm_long(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[32][1];
    const int64_t row = blockIdx.x;
    const TX* x = (const TX*)j.x + row * j.sx;
    TY* y = (TY*)j.y + row * j.sy;
    float s[1] = {0.f}, v[1], w[1] = {1.f}, b[1] = {0.f};
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        load<TX, 1>(x + c, v, j.sp_x);
        s[0] += v[0];
    }
    group_sum<1>(s, sh);
    const float mean = over_n(s[0], j);
    s[0] = 0.f;
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        load<TX, 1>(x + c, v, j.sp_x);
        s[0] = __fmaf_rn(v[0] - mean, v[0] - mean, s[0]);
    }
    group_sum<1>(s, sh);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(s[0], j.inv_cols, j.eps)));
    if (threadIdx.x == 0) {
        if (j.mean && TROP_IN(j.mean + row, 4, j.sp_mean)) j.mean[row] = mean;
        if (j.rstd && TROP_IN(j.rstd + row, 4, j.sp_rstd)) j.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        load<TX, 1>(x + c, v, j.sp_x);
        if (j.w) load<TW, 1>((const TW*)j.w + c, w, j.sp_w);
        if (j.b) load<TW, 1>((const TW*)j.b + c, b, j.sp_b);
        float o[1] = {(v[0] - mean) * rstd};
        if (j.w) o[0] *= w[0];
        if (j.b) o[0] += b[0];
        store<TY, 1>(y + c, o, j.sp_y);
    }
}

// One row of the backward pass in a group's registers: h and dy, then u in its place, the weight's and
// bias's sums, and the row's two sums.
template <int VEC, int NV>
using Pairs = Pair<VEC>[NV][pairs<VEC>];
template <typename TX, typename TY, int VEC, int NV>
__device__ __forceinline__ void back_row(const Raw<TX, VEC> (&qx)[NV], const Raw<TY, VEC> (&qd)[NV], float mean, float rstd,
                                         Pairs<VEC, NV>& h, Pairs<VEC, NV>& d)
{
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) {
            h[k][i] = p_mul(p_add(pair_of<TX, VEC>(qx[k], i), p_of<Pair<VEC>>(-mean)), p_of<Pair<VEC>>(rstd));
            d[k][i] = pair_of<TY, VEC>(qd[k], i);
        }
}
// A thread's column sums, in registers, or where 1024 threads leave too few of those, in its own words
// of shared memory (16 bytes a pair; no other thread touches them).
template <int VEC, int NV, bool SHARED>
struct Sums {
    Pairs<VEC, NV> w, b;
    __device__ __forceinline__ void init(void*)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) w[k][i] = b[k][i] = p_of<Pair<VEC>>(0.f);
    }
    __device__ __forceinline__ void add(int k, int i, Pair<VEC> d, Pair<VEC> h)
    {
        w[k][i] = p_fma(d, h, w[k][i]);
        b[k][i] = p_add(b[k][i], d);
    }
    __device__ __forceinline__ Pair<VEC> get(int k, int i, int which) const { return which ? b[k][i] : w[k][i]; }
};
template <int VEC, int NV>
struct Sums<VEC, NV, true> {
    Pair<VEC>* at;
    __device__ __forceinline__ Pair<VEC>& word(int k, int i, int which) const
    {
        return at[((k * pairs<VEC> + i) * 2 + which) * blockDim.x + threadIdx.x];
    }
    __device__ __forceinline__ void init(void* shared)
    {
        at = reinterpret_cast<Pair<VEC>*>(shared);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) word(k, i, 0) = word(k, i, 1) = p_of<Pair<VEC>>(0.f);
    }
    __device__ __forceinline__ void add(int k, int i, Pair<VEC> d, Pair<VEC> h)
    {
        word(k, i, 0) = p_fma(d, h, word(k, i, 0));
        word(k, i, 1) = p_add(word(k, i, 1), d);
    }
    __device__ __forceinline__ Pair<VEC> get(int k, int i, int which) const { return word(k, i, which); }
};
// The weight's values: kept in registers, or read again for every row.
template <typename TW, int VEC, int NV, bool KEPT>
struct Weights {
    Pairs<VEC, NV> w;
    __device__ __forceinline__ void init(const NormJob& j)
    {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC;
            float v[VEC];
            const bool has = j.w && c < (int)j.cols;
            if (has) load<TW, VEC>((const TW*)j.w + c, v, j.sp_w);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) w[k][i] = has ? pair_at<VEC>(v, i) : p_of<Pair<VEC>>(1.f);
        }
    }
    // d times the weight
    __device__ __forceinline__ void times(const NormJob&, int k, Pair<VEC> (&d)[pairs<VEC>]) const
    {
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) d[i] = p_mul(d[i], w[k][i]);
    }
};
template <typename TW, int VEC, int NV>
struct Weights<TW, VEC, NV, false> {
    __device__ __forceinline__ void init(const NormJob&) {}
    __device__ __forceinline__ void times(const NormJob& j, int k, Pair<VEC> (&d)[pairs<VEC>]) const
    {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (!j.w || c >= (int)j.cols) return;
        float v[VEC];
        load<TW, VEC>((const TW*)j.w + c, v, j.sp_w);
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) d[i] = p_mul(d[i], pair_at<VEC>(v, i));
    }
};
// `times(k, d)` multiplies vector k by the weight.
template <int VEC, int NV, typename W, typename S>
__device__ __forceinline__ void back_sums(const Pairs<VEC, NV>& h, Pairs<VEC, NV>& d, const W& times, S& acc, float (&s)[2])
{
    Pair<VEC> flat = p_of<Pair<VEC>>(0.f), along = flat;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) acc.add(k, i, d[k][i], h[k][i]);
        times(k, d[k]);
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) {
            flat = p_add(flat, d[k][i]);
            along = p_fma(d[k][i], h[k][i], along);
        }
    }
    s[0] = p_sum(flat);
    s[1] = p_sum(along);
}
template <typename TX, int VEC, int NV>
__device__ __forceinline__ void back_store(const NormJob& j, int64_t row, const Pairs<VEC, NV>& h, const Pairs<VEC, NV>& d,
                                           float rstd, const float (&s)[2])
{
    const Pair<VEC> flat = p_of<Pair<VEC>>(-s[0] * j.inv_cols), along = p_of<Pair<VEC>>(-s[1] * j.inv_cols);
    TX* dx = (TX*)j.dx + row * j.sdx;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * VEC;
        if (c < (int)j.cols) {
            Pair<VEC> o[pairs<VEC>];
            float v[VEC];
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i)
                o[i] = p_mul(p_fma(h[k][i], along, p_add(d[k][i], flat)), p_of<Pair<VEC>>(rstd));
            apart<VEC>(o, v);
            store<TX, VEC>(dx + c, v, j.sp_dx);
        }
    }
}
// The block's column sums into its row of the partial sums.  Blocks of several warps that each took
// rows of their own (blockDim.y > 1) add theirs in warp order, through `across` [warps][cols].
template <int VEC, int NV, typename S>
__device__ __forceinline__ void back_partials(const NormJob& j, const S& acc, float* across, int off = 0)
{
    const int cols = (int)j.cols;
    for (int which = 0; which < 2; ++which) {
        float* part = which ? j.part_b : j.part_w;
        if (!part) continue;
        const Span& sp = which ? j.sp_pb : j.sp_pw;
        (void)sp;
        part += (int64_t)blockIdx.x * cols;
        if (blockDim.y > 1) __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC - off;
            if (c >= cols) continue;
            Pair<VEC> o[pairs<VEC>];
            float v[VEC];
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) o[i] = acc.get(k, i, which);
            apart<VEC>(o, v);
            if (blockDim.y > 1 || cols % VEC != 0 || off != 0) {
                float* to = blockDim.y > 1 ? across + threadIdx.y * cols : part;
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i >= 0 && c + i < cols && (blockDim.y > 1 || TROP_IN(part + c + i, 4, sp))) to[c + i] = v[i];
            } else {
                store<float, VEC>(part + c, v, sp);
            }
        }
        if (blockDim.y > 1) {
            __syncthreads();
            for (int c = threadIdx.y * 32 + threadIdx.x; c < cols; c += 32 * blockDim.y) {
                float a = 0.f;
                for (int r = 0; r < (int)blockDim.y; ++r) a += across[r * cols + c];
                if (TROP_IN(part + c, 4, sp)) part[c] = a;
            }
        }
    }
}

// Rows from global memory, U of a group's rows on their way at a time.  TX: x and dx; TY: dy.
template <typename TX, typename TY, typename TW, int VEC, int NV, int U, int MAXT>
__global__ void __launch_bounds__(MAXT) k_norm_back(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float sh[2][32][2 * U];
    constexpr bool WIDE = MAXT > 512;  // sums in shared memory, weights read again
    Sums<VEC, NV, WIDE> acc;
    Weights<TW, VEC, NV, !WIDE> w;
    acc.init(dyn);
    w.init(j);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    const int cols = (int)j.cols;
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row0 < j.rows; row0 += step * U) {
        Raw<TX, VEC> qx[U][NV];
        Raw<TY, VEC> qd[U][NV];
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            const bool live = row < j.rows;
            mean[u] = live && TROP_IN(j.mean + row, 4, j.sp_mean) ? j.mean[row] : 0.f;
            rstd[u] = live && TROP_IN(j.rstd + row, 4, j.sp_rstd) ? j.rstd[row] : 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * blockDim.x + threadIdx.x) * VEC;
                const TX* x = (const TX*)j.x + row * j.sx + c;
                const TY* dy = (const TY*)j.dy + row * j.sdy + c;
                if (live && c < cols && TROP_IN(x, VEC * sizeof(TX), j.sp_x) && TROP_IN(dy, VEC * sizeof(TY), j.sp_dy)) {
                    qx[u][k].read(x);
                    qd[u][k].read(dy);
                } else {  // dy = 0: nothing in any sum
                    qx[u][k].zero();
                    qd[u][k].zero();
                }
            }
        }
        // the U rows' sums, joined at once; h and u are formed again for the result
        float sums[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pairs<VEC, NV> h, d;
            float s[2];
            back_row<TX, TY, VEC, NV>(qx[u], qd[u], mean[u], rstd[u], h, d);
            back_sums<VEC, NV>(h, d, [&](int k, Pair<VEC>(&e)[pairs<VEC>]) { w.times(j, k, e); }, acc, s);
            sums[2 * u] = s[0], sums[2 * u + 1] = s[1];
        }
        if (!j.dx) continue;
        group_sum_turn<2 * U>(sums, sh[turn]);
        turn ^= 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            if (row >= j.rows) break;
            Pairs<VEC, NV> h, d;
#pragma unroll
            for (int k = 0; k < NV; ++k) qx[u][k].again(), qd[u][k].again();
            back_row<TX, TY, VEC, NV>(qx[u], qd[u], mean[u], rstd[u], h, d);
#pragma unroll
            for (int k = 0; k < NV; ++k) w.times(j, k, d[k]);
            const float s[2] = {sums[2 * u], sums[2 * u + 1]};
            back_store<TX, VEC, NV>(j, row, h, d, rstd[u], s);
        }
    }
    if (j.part_w || j.part_b) back_partials<VEC, NV>(j, acc, reinterpret_cast<float*>(dyn));
}

// The same for rows that do not start on 16 bytes: a block's rows share one offset (see k_norm_off), so
// its threads' columns, and with them their sums, stay the same ones.  WIDE: up to 1024 threads of 64
// registers, the sums and the weight (moved by the offset) in shared memory.
template <typename T, typename TW, int VEC, int NV, int U, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 1024 : 512) k_norm_back_off(const NormJob j, int period)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float sh[2][32][2 * U];
    const int cols = (int)j.cols;
    const Offset o = offset_of<T, VEC>(j.x, j.sx, period);
    const T *const end_x = (const T*)j.x + (j.rows - 1) * j.sx + cols, *const end_dy = (const T*)j.dy + (j.rows - 1) * j.sdy + cols;
    Sums<VEC, NV, WIDE> acc;
    acc.init(dyn);
    TW* const sw = reinterpret_cast<TW*>(dyn + (size_t)blockDim.x * NV * VEC * 8);
    Pairs<VEC, WIDE ? 1 : NV> w;
    if (WIDE) {
        for (int i = threadIdx.x; i < NV * VEC * (int)blockDim.x; i += blockDim.x) {
            const int c = i - o.off;
            const bool in = j.w && c >= 0 && c < cols && TROP_IN((const TW*)j.w + c, sizeof(TW), j.sp_w);
            sw[i] = in ? ((const TW*)j.w)[c] : from_f32<TW>(j.w ? 0.f : 1.f);
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC - o.off;
            float v[VEC];
            if (j.w) load_part<TW, VEC>((const TW*)j.w, c, cols, v, j.sp_w);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) w[WIDE ? 0 : k][i] = j.w ? pair_at<VEC>(v, i) : p_of<Pair<VEC>>(1.f);
        }
    }
    const auto times = [&](int k, Pair<VEC>(&d)[pairs<VEC>]) {
        if (WIDE) {
            Raw<TW, VEC> q;
            q.read(sw + (k * blockDim.x + threadIdx.x) * VEC);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) d[i] = p_mul(d[i], pair_of<TW, VEC>(q, i));
        } else {
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) d[i] = p_mul(d[i], w[WIDE ? 0 : k][i]);
        }
    };
    int turn = 0;
    for (int64_t n = o.first; o.cls + period * n < j.rows; n += o.step * U) {
        Raw<T, VEC> qx[U][NV], qd[U][NV];
        float mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = o.cls + period * (n + u * o.step);
            const bool live = row < j.rows;
            mean[u] = live && TROP_IN(j.mean + row, 4, j.sp_mean) ? j.mean[row] : 0.f;
            rstd[u] = live && TROP_IN(j.rstd + row, 4, j.sp_rstd) ? j.rstd[row] : 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * blockDim.x + threadIdx.x) * VEC - o.off;
                if (live && c < cols) {
                    load_off<T, VEC>((const T*)j.x + row * j.sx, c, cols, (const T*)j.x, end_x, qx[u][k], j.sp_x);
                    load_off<T, VEC>((const T*)j.dy + row * j.sdy, c, cols, (const T*)j.dy, end_dy, qd[u][k], j.sp_dy);
                } else {  // dy = 0: nothing in any sum
                    qx[u][k].zero();
                    qd[u][k].zero();
                }
            }
        }
        float sums[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Pairs<VEC, NV> h, d;
            float s[2];
            back_row<T, T, VEC, NV>(qx[u], qd[u], mean[u], rstd[u], h, d);
            back_sums<VEC, NV>(h, d, times, acc, s);
            sums[2 * u] = s[0], sums[2 * u + 1] = s[1];
        }
        if (!j.dx) continue;
        group_sum_turn<2 * U>(sums, sh[turn]);
        turn ^= 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = o.cls + period * (n + u * o.step);
            if (row >= j.rows) break;
            Pairs<VEC, NV> h, d;
#pragma unroll
            for (int k = 0; k < NV; ++k) qx[u][k].again(), qd[u][k].again();
            back_row<T, T, VEC, NV>(qx[u], qd[u], mean[u], rstd[u], h, d);
            const Pair<VEC> flat = p_of<Pair<VEC>>(-sums[2 * u] * j.inv_cols);
            const Pair<VEC> along = p_of<Pair<VEC>>(-sums[2 * u + 1] * j.inv_cols);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                times(k, d[k]);
                const int c = (k * blockDim.x + threadIdx.x) * VEC - o.off;
                if (c >= cols) continue;
                Pair<VEC> r[pairs<VEC>];
                float v[VEC];
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i)
                    r[i] = p_mul(p_fma(h[k][i], along, p_add(d[k][i], flat)), p_of<Pair<VEC>>(rstd[u]));
                apart<VEC>(r, v);
                store_off<T, VEC>((T*)j.dx + row * j.sdx, c, cols, v, j.sp_dx);
            }
        }
    }
    if (j.part_w || j.part_b) back_partials<VEC, NV>(j, acc, reinterpret_cast<float*>(dyn), o.off);
}

// Rows through shared memory: a ring of `stages` rows of x and dy, each brought by two bulk copies, so
// that several rows per block are on their way whatever the block is doing; the barrier of a row's
// sums also says that its stage has been read.
template <typename TX, typename TY, typename TW, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) k_norm_back_ring(const NormJob j, int stages, uint32_t* error)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float sh[2][32][2];
    __shared__ __align__(8) uint64_t full[RING_STAGES];
    const int cols = (int)j.cols;
    const uint32_t xb = cols * sizeof(TX), db = cols * sizeof(TY);
    const int64_t first = blockIdx.x, step = gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    auto fetch = [&](int s, int64_t row) {
        const TX* x = (const TX*)j.x + row * j.sx;
        const TY* dy = (const TY*)j.dy + row * j.sdy;
        if (TROP_IN(x, (int)xb, j.sp_x) && TROP_IN(dy, (int)db, j.sp_dy)) {
            mbar_expect_tx(&full[s], xb + db);
            bulk_load(dyn + (size_t)s * (xb + db), x, xb, &full[s]);
            bulk_load(dyn + (size_t)s * (xb + db) + xb, dy, db, &full[s]);
        } else {
            mbar_expect_tx(&full[s], 0);
        }
    };
    int64_t ahead = first;  // the next row to fetch (thread 0)
    if (threadIdx.x == 0)
        for (int s = 0; s < stages && ahead < j.rows; ++s, ahead += step) fetch(s, ahead);
    Sums<VEC, NV, false> acc;
    Weights<TW, VEC, NV, true> w;
    acc.init(nullptr);
    w.init(j);
    int s = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    float mean = 0.f, rstd = 0.f;
    if (first < j.rows && TROP_IN(j.mean + first, 4, j.sp_mean) && TROP_IN(j.rstd + first, 4, j.sp_rstd))
        mean = j.mean[first], rstd = j.rstd[first];
    for (int64_t row = first; row < j.rows; row += step) {
        float mean2 = 0.f, rstd2 = 0.f;  // the next row's
        if (row + step < j.rows && TROP_IN(j.mean + row + step, 4, j.sp_mean) && TROP_IN(j.rstd + row + step, 4, j.sp_rstd))
            mean2 = j.mean[row + step], rstd2 = j.rstd[row + step];
        ok = mbar_wait(&full[s], phase);
        const uint8_t* at = dyn + (size_t)s * (xb + db);
        Raw<TX, VEC> qx[NV];
        Raw<TY, VEC> qd[NV];
        Pairs<VEC, NV> h, d;
        float sum[2];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * VEC;
            qx[k].zero();  // past the row dy = 0: nothing in any sum
            qd[k].zero();
            if (c < cols) {
                qx[k].read(reinterpret_cast<const TX*>(at) + c);
                qd[k].read(reinterpret_cast<const TY*>(at + xb) + c);
            }
        }
        back_row<TX, TY, VEC, NV>(qx, qd, mean, rstd, h, d);
        back_sums<VEC, NV>(h, d, [&](int k, Pair<VEC>(&e)[pairs<VEC>]) { w.times(j, k, e); }, acc, sum);
        warp_sum<2>(sum);
        if ((threadIdx.x & 31) == 0) sh[turn][threadIdx.x >> 5][0] = sum[0], sh[turn][threadIdx.x >> 5][1] = sum[1];
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (threadIdx.x == 0 && ahead < j.rows) fetch(s, ahead), ahead += step;
        if (j.dx) {
            sum[0] = sum[1] = 0.f;
            for (int q = 0; q < (int)(blockDim.x >> 5); ++q) sum[0] += sh[turn][q][0], sum[1] += sh[turn][q][1];
            back_store<TX, VEC, NV>(j, row, h, d, rstd, sum);
        }
        turn ^= 1;
        mean = mean2, rstd = rstd2;
        if (++s == stages) s = 0, phase ^= 1;
    }
    if (!ok) {
        ring_failed(full, stages, s, phase, error);
        return;
    }
    if (j.part_w || j.part_b) back_partials<VEC, NV>(j, acc, nullptr);
}

template <typename TX, typename TY, typename TW>
__global__ void __launch_bounds__(1024) k_norm_back_long(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[32][2];
    const int64_t row = blockIdx.x;
    const TX* x = (const TX*)j.x + row * j.sx;
    const TY* dy = (const TY*)j.dy + row * j.sdy;
    TX* dx = (TX*)j.dx + row * j.sdx;
    const float mean = TROP_IN(j.mean + row, 4, j.sp_mean) ? j.mean[row] : 0.f;
    const float rstd = TROP_IN(j.rstd + row, 4, j.sp_rstd) ? j.rstd[row] : 0.f;
    float s[2] = {0.f, 0.f}, v[1], d[1], w[1] = {1.f};
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        load<TX, 1>(x + c, v, j.sp_x);
        load<TY, 1>(dy + c, d, j.sp_dy);
        if (j.w) load<TW, 1>((const TW*)j.w + c, w, j.sp_w);
        const float u = d[0] * w[0];
        s[0] += u;
        s[1] = __fmaf_rn(u, (v[0] - mean) * rstd, s[1]);
    }
    group_sum<2>(s, sh);
    const float flat = s[0] * j.inv_cols, along = s[1] * j.inv_cols;
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        load<TX, 1>(x + c, v, j.sp_x);
        load<TY, 1>(dy + c, d, j.sp_dy);
        if (j.w) load<TW, 1>((const TW*)j.w + c, w, j.sp_w);
        const float o[1] = {rstd * (d[0] * w[0] - flat - (v[0] - mean) * rstd * along)};
        store<TX, 1>(dx + c, o, j.sp_dx);
    }
}

// Column sums of rows blockIdx.y, + gridDim.y, ...: one thread per column.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) k_norm_columns(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= j.cols) return;
    float aw = 0.f, ab = 0.f, v[1], d[1];
    for (int64_t row = blockIdx.y; row < j.rows; row += gridDim.y) {
        load<TX, 1>((const TX*)j.x + row * j.sx + c, v, j.sp_x);
        load<TY, 1>((const TY*)j.dy + row * j.sdy + c, d, j.sp_dy);
        const float mean = TROP_IN(j.mean + row, 4, j.sp_mean) ? j.mean[row] : 0.f;
        const float rstd = TROP_IN(j.rstd + row, 4, j.sp_rstd) ? j.rstd[row] : 0.f;
        aw = __fmaf_rn(d[0], (v[0] - mean) * rstd, aw);
        ab += d[0];
    }
    const int64_t at = blockIdx.y * j.cols + c;
    if (j.part_w && TROP_IN(j.part_w + at, 4, j.sp_pw)) j.part_w[at] = aw;
    if (j.part_b && TROP_IN(j.part_b + at, 4, j.sp_pb)) j.part_b[at] = ab;
}

// The blocks' column sums: 32 columns per block of threads, 32 warps taking every 32nd block's sums
// in block order, blockIdx.y choosing the weight or the bias.
template <typename TW>
__global__ void __launch_bounds__(1024) k_norm_join(const float* part_w, const float* part_b, int blocks, int64_t cols,
                                                    TW* dw, TW* db, Span sp_pw, Span sp_pb, Span sp_dw, Span sp_db)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[32][33];
    const bool bias = dw == nullptr || blockIdx.y == 1;
    const float* part = bias ? part_b : part_w;
    const Span sp = bias ? sp_pb : sp_pw;
    (void)sp;
    TW* out = bias ? db : dw;
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < cols) {
        float v[4];
        int b = threadIdx.y;
        for (; b + 96 < blocks; b += 128) {  // four loads on their way
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float* p = part + (b + 32 * k) * cols + c;
                v[k] = TROP_IN(p, 4, sp) ? *p : 0.f;
            }
            a += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; b < blocks; b += 32)
            if (TROP_IN(part + b * cols + c, 4, sp)) a += part[b * cols + c];
    }
    sh[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    // warp y sums column y's 32 values
    a = sh[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < cols) {
        const float o[1] = {a};
        store<TW, 1>(out + col, o, bias ? sp_db : sp_dw);
    }
}
template <typename TW>
__global__ void __launch_bounds__(256) k_fill_zero(TW* p, int64_t n, Span sp)
{
    pdl_wait();
    pdl_signal();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n && TROP_IN(p + i, sizeof(TW), sp)) p[i] = from_f32<TW>(0.f);
}

// ------------------------------------------------------------------ host
bool aligned(const void* p, int64_t stride, size_t elem, int vec, int64_t rows)
{
    return !p || (((uintptr_t)p % (elem * vec)) == 0 && (rows <= 1 || stride % vec == 0));
}

// After how many rows the rows' places in 16-byte granules repeat, the same for all the matrices: 0 where
// they differ, or an element straddles granules.
struct Rows {
    const void* p;
    int64_t stride;
};
int offset_period(size_t elem, int64_t rows, std::initializer_list<Rows> all)
{
    const int64_t v = 16 / elem;
    int64_t base = -1, stride = 0;
    for (const Rows& m : all) {
        if (!m.p) continue;
        if ((uintptr_t)m.p % elem) return 0;
        const int64_t b = ((uintptr_t)m.p % 16) / elem, s = rows > 1 ? m.stride % v : 0;
        if (base < 0) base = b, stride = s;
        else if (b != base || s != stride) return 0;
    }
    int period = 1;
    while (period * stride % v) period *= 2;
    return period;
}

#define TROP_LAUNCH(kernel, grid, block, smem, ...)                                   \
    do {                                                                              \
        const cudaError_t e_ = launch_pdl(kernel, grid, block, smem, s, __VA_ARGS__); \
        if (e_ != cudaSuccess) return cuda_error(e_, #kernel " launch");              \
        count_launches(1);                                                            \
    } while (0)

// A row's group of the forward pass: as many vectors per thread as still leave 8 warps per SM at
// work, so that long batches put a row into one warp (no barrier, up to 16 loads on their way per
// thread) and a few rows are spread over many threads: 16384x4096 bf16, two warps per row; 16x512 f32,
// 128 threads per row.
template <typename TX, int VEC>
bool forward_shape(int64_t units, int64_t rows, int sm, int* nv, dim3* block)
{
    for (int n = VEC == 8 ? 8 : 16; n >= 1; n /= 2) {
        const int64_t most = VEC * n * sizeof(TX) <= 64 ? 1024 : 256;
        const int64_t g = ((units + n - 1) / n + 31) / 32 * 32;
        if (g > most) break;
        *nv = n;
        *block = g == 32 ? dim3(32, 8) : dim3((unsigned)g, 1);
        if (rows * (g / 32) >= (int64_t)sm * 8) return true;
    }
    return *nv > 0;
}

template <typename TX, typename TY, typename TW, int VEC>
int norm_rows(const NormJob& j, int nv, dim3 grid, dim3 block, cudaStream_t s)
{
    switch (nv) {
    case 1: TROP_LAUNCH((k_norm<TX, TY, TW, VEC, 1>), grid, block, 0, j); break;
    case 2: TROP_LAUNCH((k_norm<TX, TY, TW, VEC, 2>), grid, block, 0, j); break;
    case 4: TROP_LAUNCH((k_norm<TX, TY, TW, VEC, 4>), grid, block, 0, j); break;
    case 8: TROP_LAUNCH((k_norm<TX, TY, TW, VEC, 8>), grid, block, 0, j); break;
    default: TROP_LAUNCH((k_norm<TX, TY, TW, VEC, VEC == 8 ? 8 : 16>), grid, block, 0, j);
    }
    return TROP_OK;
}

// Dynamic shared memory that needs no attribute: a block has 48 KB in all without it, of which static arrays take
// up to 2 KB (sh[2][32][8]).
constexpr size_t PLAIN_SMEM = 49152 - 2048;
// More of it.  The limit is state of the function, which every host thread shares: it is raised once for a kernel and
// a device, to all that the device has, and never set to one call's need, which another thread's smaller
// one could take back before the launch.
int allow_dynamic(const void* kernel)
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
    if (e != cudaSuccess) return cuda_error(e, "cudaFuncSetAttribute (layer norm)");
    try {
        raised->kernels.insert({dev, kernel});
    } catch (...) {  // no memory to write it down: asked for again next time
    }
    return TROP_OK;
}

// Bytes of an SM's rings.
constexpr size_t RING_BYTES = 196608;

template <typename TX, typename TY, typename TW>
int norm_forward(const NormJob& j, int sm, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(TX);
    const bool vec = j.cols % V == 0 && aligned(j.x, j.sx, sizeof(TX), V, j.rows) &&
                     aligned(j.y, j.sy, sizeof(TY), V, j.rows) && aligned(j.w, 0, sizeof(TW), V, 1) &&
                     aligned(j.b, 0, sizeof(TW), V, 1);
    const int64_t units = j.cols / V;
    // many short rows (65536x512 f32: 46 us, a warp per row and one row at a time 81 us; bf16 26 us and 50 us; on the device at
    // the rule's 2432 rows: 512 f32 2.8 us and 3.8 us, 256 bf16 3.0 us and 2.9 us)
    if (vec && units <= 128 && j.rows >= (int64_t)sm * 16) {
        const int nv = units <= 32 ? 1 : units <= 64 ? 2 : 4;
        const dim3 block(32, 8);
        const int64_t blocks = std::min<int64_t>((j.rows * nv + 31) / 32, (int64_t)sm * 4);
        const auto kernel = nv == 1   ? k_norm_short<TX, TY, TW, V, 1, 4>
                            : nv == 2 ? k_norm_short<TX, TY, TW, V, 2, 2>
                                      : k_norm_short<TX, TY, TW, V, 4, 1>;
        TROP_LAUNCH(kernel, dim3((unsigned)blocks), block, 0, j);
        return TROP_OK;
    }
    if constexpr (std::is_same<TX, TY>::value) {
        const int period = vec ? 0 : offset_period(sizeof(TX), j.rows, {{j.x, j.sx}, {j.y, j.sy}});
        const int64_t vecs = (j.cols + V - 1) / V + 1;
        const int nv = vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4;
        const int64_t g = ((vecs + nv - 1) / nv + 31) / 32 * 32;
        // Two f32 rows at a time (65536x1001 100 us, one 120 us, the scalar kernel 135 us), one 16-bit row (75 us; two
        // spill: 104 us; scalar 158 us).  Near the rule's number of rows it comes out even: 1216x1001 bf16 4.3 us and 6.4 us,
        // 608x4001 bf16 10.8 us and 7.8 us, 2432x1001 f32 8.2 us and 7.1 us on the device.
        if (period > 0 && vecs <= 2048 && j.rows * (g / 32) >= (int64_t)sm * 16) {
            const dim3 block((unsigned)g, g == 32 ? 8 : 1);
            const size_t smem = 2 * (size_t)(j.cols + 2 * V) * sizeof(TW);
            const auto kernel = nv == 1   ? k_norm_off<TX, TW, V, 1, 4>
                                : nv == 2 ? k_norm_off<TX, TW, V, 2, 2>
                                          : k_norm_off<TX, TW, V, 4, sizeof(TX) == 2 ? 1 : 2>;
            if (smem > PLAIN_SMEM) TROP_TRY(allow_dynamic((const void*)kernel));
            int per_sm = 0;  // as many blocks as run at once: none waits for a place
            const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, (int)(g * block.y), smem);
            if (e != cudaSuccess) return cuda_error(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor(k_norm_off)");
            int64_t blocks = std::min<int64_t>((j.rows + block.y - 1) / block.y, (int64_t)sm * std::max(1, per_sm));
            blocks = std::max<int64_t>(1, blocks / period) * period;
            TROP_LAUNCH(kernel, dim3((unsigned)blocks), block, smem, j, period);
            return TROP_OK;
        }
    }
    int nv = 0;
    dim3 block;
    const bool fits = vec ? forward_shape<TX, V>(units, j.rows, sm, &nv, &block)
                          : forward_shape<TX, 1>(j.cols, j.rows, sm, &nv, &block);
    if (!fits) {
        TROP_LAUNCH((k_norm_long<TX, TY, TW>), dim3((unsigned)j.rows), dim3(1024), 0, j);
        return TROP_OK;
    }
    // blocks that fetch ahead walk over the rows; the others take one row each
    int64_t blocks = (j.rows + block.y - 1) / block.y;
    if ((vec ? 16 : sizeof(TX)) * nv <= 32)
        blocks = std::min<int64_t>(blocks, (int64_t)sm * std::max<int>(1, 2048 / (int)(block.x * block.y)));
    const dim3 grid((unsigned)blocks);
    return vec ? norm_rows<TX, TY, TW, V>(j, nv, grid, block, s) : norm_rows<TX, TY, TW, 1>(j, nv, grid, block, s);
}

// A row's group of the backward pass, whose threads keep the column sums too: 16 elements at most.  Few
// rows: the fewest vectors per thread that keep the group at 256 threads or less, then wider groups.
// `many` rows: as many elements per thread as leave a warp or two per row, since what a row costs beside
// its elements (sums, barrier) is the group's: 65536x1024 f32 with 256 threads per row 213 us, with 64
// 134 us; on the device at the 2432 rows from which it applies 10.6 us and 9.7 us.
bool backward_shape(int64_t units, int most_nv, bool many, int* nv, dim3* block)
{
    int n = 1;
    if (many && units > 32 && units <= 64) n = 2;
    else if (many)
        for (n = most_nv; n > 1 && units < (int64_t)n * 48; n /= 2) {
        }
    else
        while (n < most_nv && units > (int64_t)n * 256) n *= 2;
    const int64_t g = ((units + n - 1) / n + 31) / 32 * 32;
    if (g > 1024) return false;
    *nv = n;
    *block = g == 32 ? dim3(32, 4) : dim3((unsigned)g, 1);
    return true;
}

template <typename TX, typename TY, typename TW>
int norm_backward(NormJob j, const NormVec& dw, const NormVec& db, int sm, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(TX);
    constexpr int MOST = sizeof(TX) == 2 ? 2 : 4;  // vectors per thread: 16 elements
    const bool vec = j.cols % V == 0 && aligned(j.x, j.sx, sizeof(TX), V, j.rows) &&
                     aligned(j.dx, j.sdx, sizeof(TX), V, j.rows) && aligned(j.dy, j.sdy, sizeof(TY), V, j.rows) &&
                     aligned(j.w, 0, sizeof(TW), V, 1);
    int nv = 0;
    dim3 block;
    const bool fits = backward_shape(vec ? j.cols / V : j.cols, vec ? MOST : 16, vec && j.rows >= 16 * sm, &nv, &block);
    const bool sums = dw.p || db.p;
    // Many rows off the 16-byte granules: eight elements a thread, four rows at a time, where that fills an
    // SM's 512 threads of 128 registers; else sixteen a thread, one row at a time, and so for 16-bit rows too
    // where a block gets eight rows or more: 65536x1001 bf16 119 us, with eight a thread 186 us, but
    // 2999x1001 23.5 us, with eight 16.3 us (partial sums of more blocks).  On the device near the rule's 1216 rows, against the
    // scalar kernel: 1216x1001 f32 8.6 us and 8.3 us, 2432x1001 f32 10.2 us and 11.5 us, bf16 14.1 us and 11.8 us.
    int period = 0;
    if constexpr (std::is_same<TX, TY>::value)
        if (!vec && j.rows >= (int64_t)sm * 8 && j.cols + V > 8 * V && j.cols + V <= 16384)
            period = offset_period(sizeof(TX), j.rows, {{j.x, j.sx}, {j.dy, j.sdy}, {j.dx, j.sdx}});
    const int64_t off_vecs = (j.cols + V - 1) / V + 1;
    int64_t off_g = ((off_vecs * V + 7) / 8 + 31) / 32 * 32, off_per_sm = 512 / (off_g == 32 ? 128 : off_g);
    const int64_t wide_g = ((off_vecs * V + 15) / 16 + 31) / 32 * 32;
    const bool off_many = sizeof(TX) == 2 && j.rows * wide_g >= (int64_t)sm * 1024 * 8;
    const bool off_wide = wide_g > 32 && (off_g * off_per_sm < 384 || off_many);
    if (off_wide) {
        off_g = wide_g;
        off_per_sm = std::min<int64_t>(1024 / off_g, 220000 / (off_g * 16 * (8 + sizeof(TW))));
    }
    const dim3 off_block((unsigned)off_g, off_g == 32 ? 4 : 1);  // (a wide block has one group: off_g >= 64)
    const size_t pair = j.cols * (sizeof(TX) + sizeof(TY));
    const int per_sm = block.x > 256 ? 1 : std::max<int>(2, 512 / (int)block.x);  // blocks that share an SM
    const int stages = (int)std::min<size_t>(RING_STAGES, RING_BYTES / per_sm / pair);
    // Rows of x and dy that bulk copies can bring (16-byte granules), and enough of them to fill a ring:
    // 16384x4096 bf16 69 us, loaded by the threads themselves 129 us; f32 130 us and 138 us.  On the device at the rule's
    // 608 rows: 4096 bf16 9.8 us and 10.1 us, 1024 f32 6.2 us and 6.5 us.
    const bool ring = fits && vec && block.y == 1 && block.x >= 64 && block.x <= 512 && j.cols * sizeof(TY) % 16 == 0 &&
                      aligned(j.dy, j.sdy * sizeof(TY), 1, 16, j.rows) && j.rows >= 4 * sm && stages >= 2;
    int blocks = 0;
    if (period > 0) {
        blocks = (int)std::min<int64_t>((j.rows + off_block.y - 1) / off_block.y, sm * off_per_sm);
        blocks = std::max(1, blocks / period) * period;
    } else if (ring) blocks = (int)std::min<int64_t>(j.rows, (int64_t)sm * per_sm);
    else if (fits)
        blocks = (int)std::min<int64_t>((j.rows + block.y - 1) / block.y,
                                        (int64_t)sm * std::max<int>(1, 512 / (int)(block.x * block.y)));
    else blocks = (int)std::min<int64_t>(j.rows, std::max<int64_t>(1, (int64_t)sm * 8 * 256 / j.cols));
    const size_t bytes = (size_t)blocks * j.cols * 4, spaced = (bytes + 255) / 256 * 256;
    Workspace ws(s);
    if (sums) {
        ws.add(2 * spaced);
        TROP_TRY(ws.take());
    }
    char* const part = ws.base;
    void* const pw = dw.p ? part : nullptr;
    void* const pb = db.p ? part + spaced : nullptr;
    j.part_w = (float*)pw;
    j.part_b = (float*)pb;
    j.sp_pw = span_bytes(pw, bytes);
    j.sp_pb = span_bytes(pb, bytes);
    if (period > 0) {
        if constexpr (std::is_same<TX, TY>::value) {
            const size_t smem = off_wide ? off_g * 16 * (8 + sizeof(TW)) : off_block.y > 1 ? off_block.y * (size_t)j.cols * 4 : 0;
            const auto kernel = off_wide ? k_norm_back_off<TX, TW, V, 16 / V, 1, true>
                                         : k_norm_back_off<TX, TW, V, 8 / V, 4, false>;
            if (smem > PLAIN_SMEM) TROP_TRY(allow_dynamic((const void*)kernel));
            TROP_LAUNCH(kernel, dim3((unsigned)blocks), off_block, smem, j, period);
        }
    } else if (!fits) {
        if (j.dx) TROP_LAUNCH((k_norm_back_long<TX, TY, TW>), dim3((unsigned)j.rows), dim3(1024), 0, j);
        if (sums)
            TROP_LAUNCH((k_norm_columns<TX, TY>), dim3((unsigned)((j.cols + 255) / 256), (unsigned)blocks), dim3(256), 0, j);
    } else if (ring) {
        uint32_t* error;
        TROP_TRY(device_error_word(&error));
        const dim3 grid((unsigned)blocks);
        const size_t smem = stages * pair;
        const auto kernel = nv == 1   ? k_norm_back_ring<TX, TY, TW, V, 1, 512>
                            : nv == 2 ? k_norm_back_ring<TX, TY, TW, V, 2, 512>
                                      : k_norm_back_ring<TX, TY, TW, V, MOST, 512>;
        TROP_TRY(allow_dynamic((const void*)kernel));
        TROP_LAUNCH(kernel, grid, block, smem, j, stages, error);
    } else {
        const dim3 grid((unsigned)blocks);
        const bool wide = block.x > 512;
        const auto kernel = !vec ? (nv <= 2  ? k_norm_back<TX, TY, TW, 1, 2, 4, 512>
                                    : nv == 4 ? k_norm_back<TX, TY, TW, 1, 4, 4, 512>
                                    : wide    ? k_norm_back<TX, TY, TW, 1, 16, 1, 1024>
                                              : k_norm_back<TX, TY, TW, 1, 16, 1, 512>)
                            : nv == 1         ? k_norm_back<TX, TY, TW, V, 1, 4, 512>
                            : nv == 2 && wide ? k_norm_back<TX, TY, TW, V, 2, 1, 1024>
                            : block.y > 1     ? k_norm_back<TX, TY, TW, V, 2, 2, 512>
                            : nv == 2         ? k_norm_back<TX, TY, TW, V, 2, 1, 512>
                            : wide            ? k_norm_back<TX, TY, TW, V, MOST, 1, 1024>
                                              : k_norm_back<TX, TY, TW, V, MOST, 1, 512>;
        // warps' sums to add up, or all sums of a wide block: 16 elements a thread, two floats each
        const size_t smem = wide ? (size_t)block.x * 16 * 8 : block.y > 1 ? block.y * (size_t)j.cols * 4 : 0;
        if (smem > PLAIN_SMEM) TROP_TRY(allow_dynamic((const void*)kernel));
        TROP_LAUNCH(kernel, grid, block, smem, j);
    }
    if (sums) {
        const dim3 grid((unsigned)((j.cols + 31) / 32), dw.p && db.p ? 2 : 1);
        TROP_LAUNCH((k_norm_join<TW>), grid, dim3(32, 32), 0, (const float*)pw, (const float*)pb, blocks, j.cols,
                    (TW*)dw.p, (TW*)db.p, j.sp_pw, j.sp_pb, span_bytes(dw.p, j.cols * sizeof(TW)),
                    span_bytes(db.p, j.cols * sizeof(TW)));
    }
    return TROP_OK;
}

template <typename TW>
int zero_vec(const NormVec& v, int64_t n, cudaStream_t s)
{
    if (v.p)
        TROP_LAUNCH((k_fill_zero<TW>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, (TW*)v.p, n,
                    span_bytes(v.p, n * sizeof(TW)));
    return TROP_OK;
}

NormJob job_of(int64_t rows, int64_t cols, const NormMat& x, const NormVec& w)
{
    NormJob j = {};
    j.rows = rows;
    j.cols = cols;
    j.inv_cols = (float)(1.0 / (double)cols);
    j.n = (float)cols;
    j.x = x.p;
    j.sx = x.sr;
    j.w = w.p;
    const int64_t size[2] = {rows, cols}, stride[2] = {x.sr, 1};
    j.sp_x = span_of(x.p, model_bytes(x.dtype), 2, size, stride);
    j.sp_w = span_bytes(w.p, cols * model_bytes(w.dtype));
    return j;
}
Span rows_span(const NormMat& m, int64_t rows, int64_t cols)
{
    const int64_t size[2] = {rows, cols}, stride[2] = {m.sr, 1};
    return span_of(m.p, model_bytes(m.dtype), 2, size, stride);
}

using bf16 = __nv_bfloat16;

}  // namespace

int launch_layer_norm(int64_t rows, int64_t cols, const NormMat& x, const NormVec& w, const NormVec& b, double eps,
                      const NormMat& y, float* mean, float* rstd, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const int sm = dev->sm_count;
    NormJob j = job_of(rows, cols, x, w);
    j.eps = (float)eps;
    j.b = b.p;
    j.y = y.p;
    j.sy = y.sr;
    j.mean = mean;
    j.rstd = rstd;
    j.sp_b = span_bytes(b.p, cols * model_bytes(b.dtype));
    j.sp_y = rows_span(y, rows, cols);
    j.sp_mean = span_bytes(mean, rows * 4);
    j.sp_rstd = span_bytes(rstd, rows * 4);
    const int tw = w.p ? w.dtype : b.p ? b.dtype : x.dtype;
    if (x.dtype == TROP_F32)
        return y.dtype == TROP_F32    ? norm_forward<float, float, float>(j, sm, s)
               : y.dtype == TROP_BF16 ? norm_forward<float, bf16, float>(j, sm, s)
                                      : norm_forward<float, __half, float>(j, sm, s);
    if (x.dtype == TROP_BF16)
        return tw == TROP_F32 ? norm_forward<bf16, bf16, float>(j, sm, s) : norm_forward<bf16, bf16, bf16>(j, sm, s);
    return tw == TROP_F32 ? norm_forward<__half, __half, float>(j, sm, s) : norm_forward<__half, __half, __half>(j, sm, s);
}

int launch_layer_norm_backward(int64_t rows, int64_t cols, const NormMat& dy, const NormMat& x, const float* mean,
                               const float* rstd, const NormVec& w, const NormMat& dx, const NormVec& dw,
                               const NormVec& db, cudaStream_t s)
{
    const int tw = w.p ? w.dtype : dw.p ? dw.dtype : db.p ? db.dtype : x.dtype;
    if (rows == 0) {  // sums over no rows
        for (const NormVec& v : {dw, db})
            TROP_TRY(tw == TROP_F32    ? zero_vec<float>(v, cols, s)
                     : tw == TROP_BF16 ? zero_vec<bf16>(v, cols, s)
                                       : zero_vec<__half>(v, cols, s));
        return TROP_OK;
    }
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    NormJob j = job_of(rows, cols, x, w);
    j.dy = dy.p;
    j.sdy = dy.sr;
    j.dx = dx.p;
    j.sdx = dx.sr;
    j.mean = const_cast<float*>(mean);
    j.rstd = const_cast<float*>(rstd);
    j.sp_dy = rows_span(dy, rows, cols);
    j.sp_dx = rows_span(dx, rows, cols);
    j.sp_mean = span_bytes(mean, rows * 4);
    j.sp_rstd = span_bytes(rstd, rows * 4);
    const int sm = dev->sm_count;
    if (x.dtype == TROP_F32)
        return dy.dtype == TROP_F32    ? norm_backward<float, float, float>(j, dw, db, sm, s)
               : dy.dtype == TROP_BF16 ? norm_backward<float, bf16, float>(j, dw, db, sm, s)
                                       : norm_backward<float, __half, float>(j, dw, db, sm, s);
    if (x.dtype == TROP_BF16)
        return tw == TROP_F32 ? norm_backward<bf16, bf16, float>(j, dw, db, sm, s)
                              : norm_backward<bf16, bf16, bf16>(j, dw, db, sm, s);
    return tw == TROP_F32 ? norm_backward<__half, __half, float>(j, dw, db, sm, s)
                          : norm_backward<__half, __half, __half>(j, dw, db, sm, s);
}

}  // namespace trop
