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
//   k_norm, k_norm_back   a row per group of 32 .. 1024 threads, each holding up to 16 (32)
//                         elements of it, as 16-byte vectors where rows are aligned to them
//   k_norm_long, k_norm_back_long, k_norm_columns   rows longer than a block's registers: the row
//                         is walked again for each pass (it stays in L2)
// The weight's and bias's gradients are summed without atomics: a persistent block keeps the sums
// of its columns over all its rows in registers and writes them once; k_norm_join adds the blocks'
// sums in block order, so results repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#define TROP_TU 7  // this file's id in a bounds-violation record
#include "internal.h"
#include "train.h"

namespace trop {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// VEC elements that lie together, moved as 16-byte (or one 8-byte, or scalar) accesses
template <typename T, int VEC>
struct alignas(VEC * sizeof(T) >= 16 ? 16 : VEC * sizeof(T)) Pack {
    T e[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float (&v)[VEC], const Span& sp)
{
    if (TROP_IN(p, VEC * sizeof(T), sp)) {
        const Pack<T, VEC> q = *reinterpret_cast<const Pack<T, VEC>*>(p);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f32(q.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.f;
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float (&v)[VEC], const Span& sp)
{
    Pack<T, VEC> q;
#pragma unroll
    for (int i = 0; i < VEC; ++i) q.e[i] = from_f32<T>(v[i]);
    if (TROP_IN(p, VEC * sizeof(T), sp)) *reinterpret_cast<Pack<T, VEC>*>(p) = q;
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

struct NormJob {
    int64_t rows, cols;
    float inv_cols, eps;
    const void *x, *dy, *w, *b;
    void *y, *dx;
    int64_t sx, sy, sdy, sdx;
    float *mean, *rstd;
    float *part_w, *part_b;  // [blocks][cols], null: not wanted
    Span sp_x, sp_y, sp_dy, sp_dx, sp_w, sp_b, sp_mean, sp_rstd, sp_pw, sp_pb;
};

template <typename TX, typename TY, typename TW, int VEC, int NV>
__global__ void __launch_bounds__(1024) k_norm(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[32][1];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= j.rows) return;  // (a block of several rows has one warp per row)
    const TX* x = (const TX*)j.x + row * j.sx;
    float v[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
        if (c < j.cols) {
            load<TX, VEC>(x + c, v[k], j.sp_x);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[k][i] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[0] += v[k][i];
    group_sum<1>(s, sh);
    const float mean = s[0] * j.inv_cols;
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
        if (c < j.cols)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                v[k][i] -= mean;
                s[0] = __fmaf_rn(v[k][i], v[k][i], s[0]);
            }
    }
    group_sum<1>(s, sh);
    const float rstd = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(s[0], j.inv_cols, j.eps)));
    if (threadIdx.x == 0) {
        if (j.mean && TROP_IN(j.mean + row, 4, j.sp_mean)) j.mean[row] = mean;
        if (j.rstd && TROP_IN(j.rstd + row, 4, j.sp_rstd)) j.rstd[row] = rstd;
    }
    TY* y = (TY*)j.y + row * j.sy;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
        if (c < j.cols) {
            float w[VEC], b[VEC], o[VEC];
            if (j.w) load<TW, VEC>((const TW*)j.w + c, w, j.sp_w);
            if (j.b) load<TW, VEC>((const TW*)j.b + c, b, j.sp_b);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                o[i] = v[k][i] * rstd;
                if (j.w) o[i] *= w[i];
                if (j.b) o[i] += b[i];
            }
            store<TY, VEC>(y + c, o, j.sp_y);
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
    const float mean = s[0] * j.inv_cols;
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

// TX: x and dx; TY: dy.
template <typename TX, typename TY, typename TW, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) k_norm_back(const NormJob j)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ float across[];  // blocks of several rows: [rows][cols]
    __shared__ float sh[32][2];
    float aw[NV][VEC], ab[NV][VEC], w[NV][VEC];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) aw[k][i] = ab[k][i] = 0.f, w[k][i] = 1.f;
        if (j.w && c < j.cols) load<TW, VEC>((const TW*)j.w + c, w[k], j.sp_w);
    }
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < j.rows;
         row += (int64_t)gridDim.x * blockDim.y) {
        const TX* x = (const TX*)j.x + row * j.sx;
        const TY* dy = (const TY*)j.dy + row * j.sdy;
        float h[NV][VEC], d[NV][VEC];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            if (c < j.cols) {
                load<TX, VEC>(x + c, h[k], j.sp_x);
                load<TY, VEC>(dy + c, d[k], j.sp_dy);
            }
        }
        const float mean = TROP_IN(j.mean + row, 4, j.sp_mean) ? j.mean[row] : 0.f;
        const float rstd = TROP_IN(j.rstd + row, 4, j.sp_rstd) ? j.rstd[row] : 0.f;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            if (c < j.cols)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    h[k][i] = (h[k][i] - mean) * rstd;
                    aw[k][i] = __fmaf_rn(d[k][i], h[k][i], aw[k][i]);
                    ab[k][i] += d[k][i];
                    d[k][i] *= w[k][i];
                    s[0] += d[k][i];
                    s[1] = __fmaf_rn(d[k][i], h[k][i], s[1]);
                }
        }
        if (!j.dx) continue;
        group_sum<2>(s, sh);
        const float flat = s[0] * j.inv_cols, along = s[1] * j.inv_cols;
        TX* dx = (TX*)j.dx + row * j.sdx;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            if (c < j.cols) {
                float o[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] = rstd * (d[k][i] - flat - h[k][i] * along);
                store<TX, VEC>(dx + c, o, j.sp_dx);
            }
        }
    }
    if (!j.part_w && !j.part_b) return;
    for (int which = 0; which < 2; ++which) {
        float* part = which ? j.part_b : j.part_w;
        if (!part) continue;
        const Span& sp = which ? j.sp_pb : j.sp_pw;
        part += (int64_t)blockIdx.x * j.cols;
        if (blockDim.y > 1) {  // the block's rows were shared by several warps: add theirs in warp order
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
                if (c < j.cols)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        across[threadIdx.y * j.cols + c + i] = which ? ab[k][i] : aw[k][i];
            }
            __syncthreads();
            for (int64_t c = threadIdx.y * 32 + threadIdx.x; c < j.cols; c += 32 * blockDim.y) {
                float a = 0.f;
                for (int r = 0; r < (int)blockDim.y; ++r) a += across[r * j.cols + c];
                if (TROP_IN(part + c, 4, sp)) part[c] = a;
            }
        } else {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
                if (c < j.cols)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (TROP_IN(part + c + i, 4, sp)) part[c + i] = which ? ab[k][i] : aw[k][i];
            }
        }
    }
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

// The blocks' column sums added in block order: 32 columns per block, eight warps taking every
// eighth block's sums, blockIdx.y choosing the weight or the bias.
template <typename TW>
__global__ void __launch_bounds__(256) k_norm_join(const float* part_w, const float* part_b, int blocks, int64_t cols,
                                                   TW* dw, TW* db, Span sp_pw, Span sp_pb, Span sp_dw, Span sp_db)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[8][33];
    const bool bias = dw == nullptr || blockIdx.y == 1;
    const float* part = bias ? part_b : part_w;
    const Span sp = bias ? sp_pb : sp_pw;
    TW* out = bias ? db : dw;
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int b = threadIdx.y; b < blocks; b += 8)
            if (TROP_IN(part + b * cols + c, 4, sp)) a += part[b * cols + c];
    sh[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && c < cols) {
        for (int w = 1; w < 8; ++w) a += sh[w][threadIdx.x];
        const float o[1] = {a};
        store<TW, 1>(out + c, o, bias ? sp_db : sp_dw);
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

#define TROP_LAUNCH(kernel, grid, block, smem, ...)                                   \
    do {                                                                              \
        const cudaError_t e_ = launch_pdl(kernel, grid, block, smem, s, __VA_ARGS__); \
        if (e_ != cudaSuccess) return cuda_error(e_, #kernel " launch");              \
        count_launches(1);                                                            \
    } while (0)

// A row's group: 32 threads (four rows per block), or one block per row.  Vectors per thread: the
// fewest that keep the group at 256 threads or less, then wider groups.
bool shape_of(int64_t units, int most_nv, int* nv, dim3* block)
{
    int n = 1;
    while (n < most_nv && units > (int64_t)n * 256) n *= 2;
    const int64_t g = ((units + n - 1) / n + 31) / 32 * 32;
    if (g > 1024) return false;
    *nv = n;
    *block = g == 32 ? dim3(32, 4) : dim3((unsigned)g, 1);
    return true;
}

template <typename TX, typename TY, typename TW>
int norm_forward(const NormJob& j, cudaStream_t s)
{
    constexpr int V = 16 / sizeof(TX);
    const bool vec = j.cols % V == 0 && aligned(j.x, j.sx, sizeof(TX), V, j.rows) &&
                     aligned(j.y, j.sy, sizeof(TY), V, j.rows) && aligned(j.w, 0, sizeof(TW), V, 1) &&
                     aligned(j.b, 0, sizeof(TW), V, 1);
    int nv;
    dim3 block;
    if (!shape_of(vec ? j.cols / V : j.cols, vec ? 4 : 16, &nv, &block)) {
        TROP_LAUNCH((k_norm_long<TX, TY, TW>), dim3((unsigned)j.rows), dim3(1024), 0, j);
        return TROP_OK;
    }
    const dim3 grid((unsigned)((j.rows + block.y - 1) / block.y));
    if (vec) {
        if (nv == 1) TROP_LAUNCH((k_norm<TX, TY, TW, V, 1>), grid, block, 0, j);
        else if (nv == 2) TROP_LAUNCH((k_norm<TX, TY, TW, V, 2>), grid, block, 0, j);
        else TROP_LAUNCH((k_norm<TX, TY, TW, V, 4>), grid, block, 0, j);
    } else if (nv <= 2) {
        TROP_LAUNCH((k_norm<TX, TY, TW, 1, 2>), grid, block, 0, j);
    } else if (nv == 4) {
        TROP_LAUNCH((k_norm<TX, TY, TW, 1, 4>), grid, block, 0, j);
    } else {
        TROP_LAUNCH((k_norm<TX, TY, TW, 1, 16>), grid, block, 0, j);
    }
    return TROP_OK;
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
    const bool fits = shape_of(vec ? j.cols / V : j.cols, vec ? MOST : 16, &nv, &block);
    const bool sums = dw.p || db.p;
    int blocks = 0;
    if (fits) {
        blocks = (int)std::min<int64_t>((j.rows + block.y - 1) / block.y,
                                        (int64_t)sm * std::max<int>(1, 512 / (int)(block.x * block.y)));
    } else {
        blocks = (int)std::min<int64_t>(j.rows, std::max<int64_t>(1, (int64_t)sm * 8 * 256 / j.cols));
    }
    void *pw = nullptr, *pb = nullptr;
    const size_t bytes = (size_t)blocks * j.cols * 4;
    if (dw.p) TROP_TRY(pool_alloc(bytes, s, &pw));
    struct Give {
        void* p;
        cudaStream_t s;
        ~Give() { if (p) pool_retire(p, s); }
    } give_w{pw, s};
    if (db.p) TROP_TRY(pool_alloc(bytes, s, &pb));
    Give give_b{pb, s};
    j.part_w = (float*)pw;
    j.part_b = (float*)pb;
    j.sp_pw = span_bytes(pw, bytes);
    j.sp_pb = span_bytes(pb, bytes);
    if (!fits) {
        if (j.dx) TROP_LAUNCH((k_norm_back_long<TX, TY, TW>), dim3((unsigned)j.rows), dim3(1024), 0, j);
        if (sums)
            TROP_LAUNCH((k_norm_columns<TX, TY>), dim3((unsigned)((j.cols + 255) / 256), (unsigned)blocks), dim3(256), 0, j);
    } else {
        const dim3 grid((unsigned)blocks);
        const size_t smem = block.y > 1 ? block.y * (size_t)j.cols * 4 : 0;
        const bool wide = block.x > 512;
        if (vec) {
            if (nv == 1) TROP_LAUNCH((k_norm_back<TX, TY, TW, V, 1, 512>), grid, block, smem, j);
            else if (nv == 2 && !wide) TROP_LAUNCH((k_norm_back<TX, TY, TW, V, 2, 512>), grid, block, smem, j);
            else if (nv == 2) TROP_LAUNCH((k_norm_back<TX, TY, TW, V, 2, 1024>), grid, block, smem, j);
            else if (!wide) TROP_LAUNCH((k_norm_back<TX, TY, TW, V, MOST, 512>), grid, block, smem, j);
            else TROP_LAUNCH((k_norm_back<TX, TY, TW, V, MOST, 1024>), grid, block, smem, j);
        } else if (nv <= 2) {
            TROP_LAUNCH((k_norm_back<TX, TY, TW, 1, 2, 512>), grid, block, smem, j);
        } else if (nv == 4) {
            TROP_LAUNCH((k_norm_back<TX, TY, TW, 1, 4, 512>), grid, block, smem, j);
        } else if (!wide) {
            TROP_LAUNCH((k_norm_back<TX, TY, TW, 1, 16, 512>), grid, block, smem, j);
        } else {
            TROP_LAUNCH((k_norm_back<TX, TY, TW, 1, 16, 1024>), grid, block, smem, j);
        }
    }
    if (sums) {
        const dim3 grid((unsigned)((j.cols + 31) / 32), dw.p && db.p ? 2 : 1);
        TROP_LAUNCH((k_norm_join<TW>), grid, dim3(32, 8), 0, (const float*)pw, (const float*)pb, blocks, j.cols,
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
        return y.dtype == TROP_F32    ? norm_forward<float, float, float>(j, s)
               : y.dtype == TROP_BF16 ? norm_forward<float, bf16, float>(j, s)
                                      : norm_forward<float, __half, float>(j, s);
    if (x.dtype == TROP_BF16)
        return tw == TROP_F32 ? norm_forward<bf16, bf16, float>(j, s) : norm_forward<bf16, bf16, bf16>(j, s);
    return tw == TROP_F32 ? norm_forward<__half, __half, float>(j, s) : norm_forward<__half, __half, __half>(j, s);
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
