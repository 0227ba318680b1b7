// linear_ce.cu -- softmax cross entropy of a linear head, without keeping its logits.
//
// Tokens x [N, D], weights w [V, D] (bf16 or f16), targets t [N]:
//   l[i, v]  = sum_d x[i, d] w[v, d]                 (products exact, sums in f32)
//   lse[i]   = log sum_v exp l[i, v]
//   loss[i]  = lse[i] - l[i, t[i]]
// and, given g[i] = d(total)/d(loss[i]):
//   P[i, v]  = g[i] (exp(l[i, v] - lse[i]) - [v = t[i]])
//   dx       = P w,   dw = P^T x.
// The logits are the ordinary (+, x) product under a log-sum-exp, the smooth form of the library's
// max-plus contraction; unlike that one they are multiply-accumulates and run on the tensor cores.
//
// One kernel, k_tile, computes all four products as tiles in tensor memory; what differs is where an
// accumulator goes:
//   LSE   a tile's logits are folded into each row's running maximum and sum of exponentials in
//         registers; the logits of a unit of tiles leave as one (maximum, sum) pair per row
//   GRAD  the logits are formed again and leave as P (scaled, in the operands' type), for a piece of
//         the vocabulary at a time, so that P takes a bounded workspace whatever V is
//   DX    P w over a piece (added to the pieces before it in f32)
//   DW    P^T x: the piece's rows of dw, whole
// Operand tiles come by TMA into a ring of 128-byte-swizzled stages; one thread issues the
// products, eight warps empty one accumulator while the next one fills.
//
// Tiles of 256 x 256 by pairs of CTAs: each CTA loads half of each operand tile, so that a stage's 64 KB feed
// twice the products of a CTA alone (8192x2048x65536 forward: CTAs alone 1433 us, pairs 1265 us).  The largest
// cases are bound by the tensor cores at the clock that the power limit leaves them, small ones by the chain of
// launches, few tokens by reading the weights (measured, bf16):
//   8192x2048x65536   forward 1265 us, 1738 TFLOP/s; backward 3960 us, 1666 TFLOP/s of the three products
//   16x4096x131072    forward 180 us, 6.0 TB/s; backward 572 us (w read for the logits and again, a gigabyte later, for dx)
//   1021x1000x32003   forward 53 us, backward 169 us
//   16x512x2000       forward 13 us, backward 26 us (per call, back to back)
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#define TROP_TU 9  // this file's id in a bounds-violation record
#include "internal.h"
#include "operands.h"
#include "packed.h"
#include "tcgen05.h"
#include "train.h"

namespace trop {

namespace {

enum { LSE = 0, GRAD = 1, DX = 2, DW = 3 };

constexpr int TK = 64;                 // depth of a stage: one 128-byte row of 16-bit elements
constexpr int A_BYTES = 128 * TK * 2;  // of one CTA
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;

// A tile's shape: CG CTAs share it, each with 128 of its rows and all TN columns in tensor memory,
// NACC accumulators taking the stages of the depth in turn.  A stage holds SUB slices of TK.
template <int CG_, int TN_, int NACC_, int SUB_ = 1>
struct Shape {
    static constexpr int CG = CG_, TN = TN_, NACC = NACC_, SUB = SUB_;
    static constexpr int TM = 128 * CG;
    static constexpr int B_BYTES = TN / CG * TK * 2;
    static constexpr int STAGE_BYTES = SUB * (A_BYTES + B_BYTES);
    static constexpr int STAGES = 196608 / STAGE_BYTES;
    static constexpr int RING = STAGES * STAGE_BYTES;
    static constexpr int BUFS = NACC * TN == 512 ? 1 : 2;  // tiles in tensor memory at a time
};
constexpr int BOX_BYTES = 4096;  // 32 rows of 128 bytes: what a result warp hands to one store
// dynamic shared memory: the ring, the result warps' boxes (LSE has none), room to align
template <int MODE, typename S>
constexpr int smem_bytes() { return S::RING + (MODE == LSE ? 0 : EPI_WARPS * BOX_BYTES) + 1024; }
using Pair = Shape<2, 256, 1>;   // products bound by the tensor cores
using Deep = Shape<2, 256, 2>;   // long logits: half the depth per accumulator
// Few tokens: bound by reading the weights, in two slices at a time so that a row's 256 bytes are
// asked for together (16x4096x131072: one slice 181 us, two 178 us, three 185 us).
using Few = Shape<1, 128, 2, 2>;
using Few1 = Shape<1, 128, 1>;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NO_MAX = -3.0e38f;  // running maximum before any logit (finite: 2^(NO_MAX - M) = 0)

// The target of row i: its column, -1 where the row is left out, -2 where it lies outside the vocabulary.
struct Targets {
    const void* p;
    int64_t stride, ignore, V;
    int wide;  // int64, else int32
    Span sp;
};
__device__ __forceinline__ int64_t target_of(const Targets& t, int64_t i)
{
    int64_t v;
    if (t.wide) {
        const int64_t* q = (const int64_t*)t.p + i * t.stride;
        v = TROP_IN(q, 8, t.sp) ? *q : t.ignore;
    } else {
        const int32_t* q = (const int32_t*)t.p + i * t.stride;
        v = TROP_IN(q, 4, t.sp) ? *q : t.ignore;
    }
    return v == t.ignore ? -1 : v < 0 || v >= t.V ? -2 : v;
}

// The tokens' gradients g[i * sg] (over *count, where that is given), and how P is stored for the 16-bit
// products: times `top` / max |g| over the tokens that count, undone in f32 when the products leave.  A
// target's entry, g (p - 1), is then close to -top when p is small, a value the type holds; g itself would be
// rounded by the same factor for every token of a batch (0.3 % of all gradients for an unlucky 1 / 7783).  In
// f16 top = 2^14 besides lifts P's entries of g / V into the type's range.
struct GradScale {
    const float* g;
    int64_t sg;
    const float* count;
    const float* given;  // {factor of P, factor of the products}; null with one g for all tokens
    float top;
    Span sp;
};
__device__ __forceinline__ float2 scale_of(float m, float top)
{
    const bool fine = m > 0.f && m < INFINITY;  // nothing kept, all zero, or not finite: P as it is
    m = fmaxf(m, 7.888609e-31f);  // 2^-100: top / m stays finite; products of smaller gradients round to f16's zero anyway
    return fine ? make_float2(__fdiv_rn(top, m), __fdiv_rn(m, top)) : make_float2(1.f, 1.f);
}
__device__ __forceinline__ float grad_of(const GradScale& q, int64_t i)
{
    const float v = TROP_IN(q.g + i * q.sg, 4, q.sp) ? q.g[i * q.sg] : 0.f;
    return q.count ? __fdiv_rn(v, *q.count) : v;
}
__device__ __forceinline__ float2 grad_scale(const GradScale& q)
{
    if (q.given) return make_float2(q.given[0], q.given[1]);
    return scale_of(fabsf(grad_of(q, 0)), q.top);
}

struct Job {
    int mt, nt, inner;      // tiles along rows and columns; column tiles of a unit
    int kt, kper;           // depth in stages, and of one split
    int units, band;
    int a_bytes;            // of A in a stage
    int a0, ak0, b0, bk0;   // first row / depth of A and of B in their tensor maps
    int pad_rows;           // rows of one split's f32 sums
    int rows, cols;         // of the output (cols: LSE the vocabulary, GRAD the piece)
    uint32_t* error;
    Targets tgt;
    // LSE
    float2* part;           // [2 * (units / mt)][mt * TM]
    float* at;              // [rows]: the logit of the target
    // GRAD
    int64_t v0;             // the piece's first column
    const float* lse;
    GradScale grad;
    // DX, DW
    void* out;              // null: f32 sums, through map_c
    int64_t ldo;
    int vec;                // rows of out start on 16 bytes: through map_c
    int add;                // f32 sums: added to the pieces before
    Span sp_part, sp_at, sp_lse, sp_out;
};

// `yes` where i == d, else `no`, as one select: written out so that 32 of them in a row do not
// become an indexed array, which would put the logits into local memory (128 bytes a thread; the
// loss of a tile then took 18,000 cycles against the 8,000 of its products at D = 1000).
__device__ __forceinline__ float where(int i, int d, float yes, float no)
{
    float r;
    asm("{\n .reg .pred p;\n setp.eq.s32 p, %1, %2;\n selp.f32 %0, %3, %4, p;\n}" : "=f"(r) : "r"(i), "r"(d), "f"(yes), "f"(no));
    return r;
}

struct Unit {
    int m, n, k0, k1;  // row tile, first column tile, stages
};
template <int MODE>
__device__ __forceinline__ Unit unit_of(const Job& j, int u)
{
    Unit r;
    if (MODE == LSE || MODE == GRAD) {
        // groups of `band` row tiles, rows fastest: the units that run together cover about as many
        // row tiles as column tiles, so each operand tile is fetched by many of them at a time
        const int groups = j.units / j.mt, per = j.band * groups;
        const int g = u / per, m0 = g * j.band, wide = min(j.band, j.mt - m0);
        u -= g * per;
        r.m = m0 + u % wide;
        r.n = (u / wide) * j.inner;
        r.k0 = 0;
        r.k1 = j.kt;
    } else {
        r.n = u % j.nt;
        u /= j.nt;
        r.m = u % j.mt;
        r.k0 = (u / j.mt) * j.kper;
        r.k1 = min(j.kt, r.k0 + j.kper);
    }
    return r;
}

// ------------------------------------------------------------------ what becomes of an accumulator tile
// A thread has one row and 128 of the tile's columns, in four loads of 32.

// 2^n of a whole n <= 0, exactly (zero from 2^-127 down)
__device__ __forceinline__ float pow2_whole(float n) { return __int_as_float(((int)fmaxf(n, -127.f) + 127) << 23); }

struct RowState {
    float M, s;        // LSE: integer reference (in log2 units) and the sum of 2^(l log2e - M)
    int64_t t;         // target column
    float nlse, g;     // GRAD: -lse log2e, gradient
};

__device__ __forceinline__ void lse_chunk(RowState& r, float (&v)[32], int left, int64_t col, float* at, const Job& j)
{
    if (left < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i >= left) v[i] = -INFINITY;
    }
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = fmaxf(v[i], v[i + 4]);
#pragma unroll
        for (int k = 8; k < 32; k += 4) m[i] = fmaxf(m[i], v[i + k]);
    }
    const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    // The reference is the maximum rounded up to a whole power of two: rescaling by a change of it
    // is exact, so the sum's only roundings are its own.
    const float M = fmaxf(r.M, ceilf(top * LOG2E));
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) a[i & 3] += ex2(__fmaf_rn(v[i], LOG2E, -M));
    r.s = r.s * pow2_whole(r.M - M) + ((a[0] + a[1]) + (a[2] + a[3]));
    r.M = M;
    const int64_t d = r.t - col;
    if (d >= 0 && d < 32) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) x = where(i, (int)d, v[i], x);
        if (TROP_IN(at, 4, j.sp_at)) *at = x;
    }
}

template <bool BF16>
__device__ __forceinline__ void grad_chunk(const RowState& r, float (&v)[32], int64_t col, uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = ex2(__fmaf_rn(v[i], LOG2E, r.nlse));
    const int64_t d = r.t - col;
    if (d >= 0 && d < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] -= where(i, (int)d, 1.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = r.t == -1 ? 0u : pack2<BF16>(v[2 * i] * r.g, v[2 * i + 1] * r.g);
}

// ------------------------------------------------------------------ joining the units' pairs
// lse and loss of `rows` tokens from their units' (reference, sum) pairs; the losses' sum.
struct JoinJob {
    const float2* part;
    int64_t stride;  // of one unit's pairs
    int G;
    int64_t rows;
    const float* at;
    Targets tgt;
    float* loss;   // nullable [rows]
    float* lse;    // [rows]
    float* total;  // {sum or mean of the losses, rows kept}: nullable
    float* kept;
    int mean;
    float2* sums;  // [CTAs]
    uint32_t* ticket;
    Span sp_part, sp_at, sp_loss, sp_lse, sp_total, sp_kept;
};
__device__ __forceinline__ void join_pair(float& M, float& s, float2 q)
{
    const float m = fmaxf(M, q.x);
    s = s * pow2_whole(M - m) + q.y * pow2_whole(q.x - m);
    M = m;
}
// 32 rows' pairs shared out to `parts` warps: the lane's row, its pairs part, part + parts, ... in that order.
__device__ __forceinline__ float2 join_part(const JoinJob& j, int64_t row, int part, int parts)
{
    float M = NO_MAX, s = 0.f;
    if (row < j.rows) {
        int g = part;
        for (; g + 3 * parts < j.G; g += 4 * parts) {  // four loads on their way
            float2 q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2* p = j.part + (int64_t)(g + k * parts) * j.stride + row;
                q[k] = TROP_IN(p, 8, j.sp_part) ? __ldcg(p) : make_float2(NO_MAX, 0.f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) join_pair(M, s, q[k]);
        }
        for (; g < j.G; g += parts) {
            const float2* p = j.part + (int64_t)g * j.stride + row;
            if (TROP_IN(p, 8, j.sp_part)) join_pair(M, s, __ldcg(p));
        }
    }
    return make_float2(M, s);
}
// The parts' pairs of 32 rows, joined in part order by one warp; {sum of the rows' losses, rows kept} in every lane.
__device__ __forceinline__ float2 join_rows(const JoinJob& j, int64_t row, const float2 (*sh)[33], int parts)
{
    const int lane = threadIdx.x & 31;
    float M = NO_MAX, s = 0.f, loss = 0.f, keep = 0.f;
    for (int w = 0; w < parts; ++w) join_pair(M, s, sh[w][lane]);
    if (row < j.rows) {
        // M is a whole number of powers of two: M ln 2 + log s in two pieces of ln 2
        const float lse = __fmaf_rn(M, LN2, __fmaf_rn(M, -1.9046542121259335e-09f, logf(s)));
        const int64_t t = target_of(j.tgt, row);
        if (TROP_IN(j.lse + row, 4, j.sp_lse)) j.lse[row] = lse;
        if (t >= 0 && TROP_IN(j.at + row, 4, j.sp_at)) loss = lse - __ldcg(j.at + row);
        if (t == -2) loss = NAN;
        keep = t == -1 ? 0.f : 1.f;
        if (j.loss && TROP_IN(j.loss + row, 4, j.sp_loss)) j.loss[row] = loss;
    }
    for (int o = 16; o > 0; o >>= 1) {
        loss += __shfl_xor_sync(0xffffffffu, loss, o);
        keep += __shfl_xor_sync(0xffffffffu, keep, o);
    }
    return make_float2(loss, keep);
}
__device__ __forceinline__ void join_total(const JoinJob& j, float loss, float keep)
{
    if (j.total && TROP_IN(j.total, 4, j.sp_total)) *j.total = j.mean ? __fdiv_rn(loss, keep) : loss;
    if (j.kept && TROP_IN(j.kept, 4, j.sp_kept)) *j.kept = keep;
}

// Many tokens: 32 rows per CTA; the CTAs leave their sums and the last one to arrive adds them in CTA
// order.
__global__ void __launch_bounds__(256) k_lse_join(const __grid_constant__ JoinJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float2 sh[8][33];
    __shared__ float red[2][32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + lane;
    sh[warp][lane] = join_part(j, row, warp, 8);
    __syncthreads();
    if (warp == 0) {
        const float2 mine = join_rows(j, row, sh, 8);
        if (lane == 0) {
            j.sums[blockIdx.x] = mine;
            __threadfence();
            last = atomicAdd(j.ticket, 1u) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    float a = 0.f, b = 0.f;
    for (int i = threadIdx.x; i < gridDim.x; i += 256) {
        const float2 q = __ldcg(&j.sums[i]);
        a += q.x;
        b += q.y;
    }
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0) red[0][warp] = a, red[1][warp] = b;
    __syncthreads();
    if (threadIdx.x == 0) {
        a = b = 0.f;
        for (int w = 0; w < 8; ++w) a += red[0][w], b += red[1][w];
        join_total(j, a, b);
        *j.ticket = 0;
    }
}

// ------------------------------------------------------------------ the kernel
template <int MODE, bool BF16, typename S>
__global__ void __launch_bounds__(THREADS, 1)
    k_tile(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const __grid_constant__ CUtensorMap map_c, const __grid_constant__ Job j, const __grid_constant__ JoinJob join)
{
    constexpr bool A_MN = MODE == DW, B_MN = MODE == DX || MODE == DW;
    constexpr int CG = S::CG, TM = S::TM, TN = S::TN, NACC = S::NACC, STAGES = S::STAGES;
    constexpr int STAGE_BYTES = S::STAGE_BYTES, BUFS = S::BUFS, SUB = S::SUB;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp == 1 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
        for (int b = 0; b < 2; ++b) mbar_init(&tfull[b], 1), mbar_init(&tempty[b], EPI_WARPS * CG);
        mbar_init(&drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) tma_prefetch_map(&map_a), tma_prefetch_map(&map_b);
    if (warp == 2) tmem_alloc_all<CG>(&tmem_slot);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {  // loads
            int s = 0;
            uint32_t phase = 0, issued = 0;
            for (int u = first; u < j.units && ok; u += step) {
                const Unit t = unit_of<MODE>(j, u);
                const int n_end = min(j.nt, t.n + (MODE == LSE ? j.inner : 1));
                for (int n = t.n; n < n_end && ok; ++n)
                    for (int k = t.k0; k < t.k1; ++k) {
                        if (!(ok = mbar_wait(&empty[s], phase ^ 1))) break;
                        if (rank == 0) mbar_expect_tx(&full[s], SUB * (j.a_bytes + S::B_BYTES) * CG);
                        const uint32_t bar = CG == 2 ? mapa(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
                        const int am = j.a0 + t.m * TM + rank * 128, bm = j.b0 + n * TN + rank * (TN / CG);
#pragma unroll
                        for (int sub = 0; sub < SUB; ++sub) {
                            const uint32_t sa = ring + s * STAGE_BYTES + sub * A_BYTES;
                            const uint32_t sb = ring + s * STAGE_BYTES + SUB * A_BYTES + sub * S::B_BYTES;
                            const int ak = j.ak0 + (k * SUB + sub) * TK, bk = j.bk0 + (k * SUB + sub) * TK;
                            if (A_MN) {
#pragma unroll
                                for (int c = 0; c < 2; ++c) tma_load_2d<CG>(sa + c * 8192, &map_a, am + 64 * c, ak, bar);
                            } else {
                                tma_load_2d<CG>(sa, &map_a, ak, am, bar);
                            }
                            if (B_MN) {
#pragma unroll
                                for (int c = 0; c < TN / CG / 64; ++c)
                                    tma_load_2d<CG>(sb + c * 8192, &map_b, bm + 64 * c, bk, bar);
                            } else {
#pragma unroll
                                for (int c = 0; c < (TN / CG + 127) / 128; ++c)
                                    tma_load_2d<CG>(sb + c * 16384, &map_b, bk, bm + 128 * c, bar);
                            }
                        }
                        ++issued;
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
            }
            if (!ok && rank == 0)  // no copy may land after the CTA has left
                for (uint32_t i = 0; i < min(issued, (uint32_t)STAGES); ++i) {
                    if (--s < 0) s = STAGES - 1, phase ^= 1;
                    (void)mbar_wait(&full[s], phase);
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {  // products
            constexpr uint32_t idesc = mma_desc(BF16, A_MN, B_MN, TM, TN);
            int s = 0;
            uint32_t phase = 0, tile = 0;
            for (int u = first; u < j.units && ok; u += step) {
                const Unit t = unit_of<MODE>(j, u);
                const int n_end = min(j.nt, t.n + (MODE == LSE ? j.inner : 1));
                for (int n = t.n; n < n_end && ok; ++n, ++tile) {
                    const uint32_t b = tile % BUFS, acc = tmem + b * (NACC * TN);
                    if (!(ok = mbar_wait_cluster(&tempty[b], ((tile / BUFS) & 1) ^ 1))) break;
                    tc_fence_after();
                    for (int k = t.k0; k < t.k1; ++k) {
                        if (!(ok = mbar_wait_cluster(&full[s], phase))) break;
                        tc_fence_after();
#pragma unroll
                        for (int sub = 0; sub < SUB; ++sub) {
                            const uint32_t sa = ring + s * STAGE_BYTES + sub * A_BYTES;
                            const uint32_t sb = ring + s * STAGE_BYTES + SUB * A_BYTES + sub * S::B_BYTES;
                            const uint64_t da = smem_desc(sa, A_MN ? 8192 : 16), db = smem_desc(sb, B_MN ? 8192 : 16);
#pragma unroll
                            for (int i = 0; i < TK / 16; ++i)  // 16 k: 32 bytes along a row, or 16 rows
                                tc_mma<CG>(acc + (NACC == 2 ? ((k - t.k0) & 1) * TN : 0), da + i * (A_MN ? 128 : 2),
                                           db + i * (B_MN ? 128 : 2), idesc, k >= t.k0 + NACC || i > 0 || sub > 0);
                        }
                        tc_commit<CG>(&empty[s]);
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
                    if (ok) tc_commit<CG>(&tfull[b]);
                }
            }
            if (!ok) {  // no product may run after the CTA has left
                tc_commit<CG>(&drain);
                (void)mbar_wait(&drain, 0);
            }
        }
    } else if (warp >= 4) {  // results
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t box = ring + S::RING + (warp - 4) * BOX_BYTES;
        uint32_t tile = 0;
        const float2 scale = MODE == LSE ? make_float2(1.f, 1.f) : grad_scale(j.grad);
        for (int u = first; u < j.units && ok; u += step) {
            const Unit t = unit_of<MODE>(j, u);
            const int n_end = min(j.nt, t.n + (MODE == LSE ? j.inner : 1));
            const int64_t row = (int64_t)t.m * TM + rank * 128 + quad * 32 + lane;
            const bool live = row < j.rows;
            RowState r;
            r.M = NO_MAX;
            r.s = 0.f;
            r.t = -1;
            if (MODE == LSE || MODE == GRAD) {
                if (live) r.t = target_of(j.tgt, row);
            }
            if (MODE == GRAD) {
                r.nlse = 0.f;
                r.g = 0.f;
                if (live && TROP_IN(j.lse + row, 4, j.sp_lse)) {
                    r.nlse = -j.lse[row] * LOG2E;
                    r.g = r.t == -2 ? NAN : grad_of(j.grad, row) * scale.x;
                }
            }
            for (int n = t.n; n < n_end && ok; ++n, ++tile) {
                const uint32_t b = tile % BUFS;
                ok = mbar_wait(&tfull[b], (tile / BUFS) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                constexpr int HALF = TN / 2, CHUNKS = HALF / 32;  // columns of a warp, loads of 32
                const uint32_t src = tmem + b * (NACC * TN) + half * HALF + ((uint32_t)(quad * 32) << 16);
                const bool both = NACC == 2 && t.k1 - t.k0 > 1;  // a single stage left the second one unwritten
                uint32_t v[2][32];
                tmem_ld32(src, v[0]);
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c) {
                    float f[32];
                    if (NACC == 2) {
                        if (both) tmem_ld32(src + TN + c * 32, v[1]);
                        tmem_wait_ld(v[0]);
                        tmem_wait_ld(v[1]);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            f[i] = both ? __uint_as_float(v[0][i]) + __uint_as_float(v[1][i]) : __uint_as_float(v[0][i]);
                        if (c < CHUNKS - 1) tmem_ld32(src + (c + 1) * 32, v[0]);
                    } else {
                        tmem_wait_ld(v[c & 1]);
                        if (c < CHUNKS - 1) tmem_ld32(src + (c + 1) * 32, v[(c + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[c & 1][i]);
                    }
                    if (c == CHUNKS - 1) {  // the accumulator is in registers: the next tile may fill it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&tempty[b]), 0));
                    }
                    const int col = n * TN + half * HALF + c * 32;
                    if (MODE == LSE) {
                        lse_chunk(r, f, j.cols - col, col, j.at + row, j);
                        continue;
                    }
                    const int row0 = t.m * TM + rank * 128 + quad * 32;
                    if (MODE != GRAD && !j.out) {  // f32 sums: a box of 32 columns
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(f[i]);
                        box_free(lane);
                        to_box<32>(box, lane, 0, w);
                        store_box(&map_c, box, lane, col, (t.k0 / j.kper) * j.pad_rows + row0, j.cols,
                                  (t.k0 / j.kper) * j.pad_rows + j.rows, j.add);
                        continue;
                    }
                    uint32_t w[16];
                    if (MODE == GRAD) {
                        grad_chunk<BF16>(r, f, j.v0 + col, w);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack2<BF16>(f[2 * i] * scale.y, f[2 * i + 1] * scale.y);
                    }
                    if (c % 2 == 0) box_free(lane);  // a box of 64 columns, in two halves
                    to_box<16>(box, lane, (c % 2) * 4, w);
                    if (c % 2 == 0) continue;
                    if (MODE == GRAD || j.vec) store_box(&map_c, box, lane, col - 32, row0, j.cols, j.rows, false);
                    else copy_box<uint16_t>(box, lane, col - 32, row0, j.rows, j.cols, j.out, j.ldo, j.sp_out);
                }
            }
            if (MODE == LSE && ok) {
                float2* q = j.part + ((int64_t)(t.n / j.inner) * 2 + half) * ((int64_t)j.mt * TM) + row;
                if (TROP_IN(q, 8, j.sp_part)) *q = make_float2(r.M, r.s);
            }
        }
    }
    if (MODE != LSE && warp >= 4 && lane == 0) tma_store_wait();
    if (!ok && lane == 0) {
        *(volatile uint32_t*)j.error = 1;
        __threadfence_system();
    }
    __syncwarp();
    pdl_signal();
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();
    if (warp == 2) tmem_free_all<CG>(tmem);
    if constexpr (MODE == LSE && CG == 1) {
        // Few tokens: the last CTA to arrive joins the pairs here, which spares a launch (about 3 us).
        __shared__ float2 sh[THREADS / 32][33];
        __shared__ uint32_t arrived;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) arrived = atomicAdd(join.ticket, 1u);
        __syncthreads();
        if (arrived != gridDim.x - 1) return;
        __threadfence();
        // 32 rows to a group of warps, all groups at once
        __shared__ float2 red[THREADS / 32];
        const int groups = (int)((join.rows + 31) / 32), parts = THREADS / 32 / groups, group = warp / parts;
        if (group < groups) sh[warp][lane] = join_part(join, group * 32 + lane, warp % parts, parts);
        __syncthreads();
        if (warp < groups) {
            const float2 q = join_rows(join, warp * 32 + lane, sh + warp * parts, parts);
            if (lane == 0) red[warp] = q;
        }
        __syncthreads();
        float loss = 0.f, keep = 0.f;
        for (int w = 0; w < groups; ++w) loss += red[w].x, keep += red[w].y;
        if (threadIdx.x == 0) {
            join_total(join, loss, keep);
            *join.ticket = 0;
        }
    }
}

// ------------------------------------------------------------------ the largest gradient of a batch
// Of the tokens that count (an ignored one's P is zero whatever its gradient) and of finite values: one infinite
// gradient spoils its own token's row, not the others' digits.
__global__ void __launch_bounds__(1024) k_gscale(const GradScale q, const Targets t, int64_t n, float* scale)
{
    pdl_wait();
    pdl_signal();
    __shared__ float red[32];
    float m = 0.f;
    for (int64_t i = threadIdx.x; i < n; i += 1024) {
        const float v = fabsf(grad_of(q, i));
        if (target_of(t, i) >= 0 && v < INFINITY) m = fmaxf(m, v);
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w) m = fmaxf(m, red[w]);
        const float2 r = scale_of(m, q.top);
        scale[0] = r.x;
        scale[1] = r.y;
    }
}

// ------------------------------------------------------------------ sums of the depth's splits
// Four columns of a row per thread and step where rows allow 16-byte loads.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) k_split_join(const float* acc, int ks, int64_t slice, int64_t lda, int64_t rows,
                                                    int64_t cols, uint16_t* out, int64_t ldo, const GradScale grad, Span sp_acc, Span sp_out)
{
    pdl_wait();
    pdl_signal();
    constexpr int W = VEC ? 4 : 1;
    const float alpha = grad_scale(grad).y;
    const int64_t n = rows * cols / W, per_row = cols / W;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per_row, c = (i - r * per_row) * W;
        float s[W];
#pragma unroll
        for (int w = 0; w < W; ++w) s[w] = 0.f;
#pragma unroll 4
        for (int k = 0; k < ks; ++k) {
            const float* p = acc + k * slice + r * lda + c;
            if (!TROP_IN(p, 4 * W, sp_acc)) continue;
            if (VEC) {
                const float4 q = *reinterpret_cast<const float4*>(p);
                s[0] += q.x, s[1] += q.y, s[2] += q.z, s[3] += q.w;
            } else {
                s[0] += *p;
            }
        }
        uint16_t* dst = out + r * ldo + c;
        if (VEC) {
            if (TROP_IN(dst, 8, sp_out))
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(s[0] * alpha, s[1] * alpha), pack2<BF16>(s[2] * alpha, s[3] * alpha));
        } else if (TROP_IN(dst, 2, sp_out)) {
            *dst = (uint16_t)(pack2<BF16>(s[0] * alpha, 0.f) & 0xffff);
        }
    }
}

__global__ void __launch_bounds__(256) k_zero16(uint16_t* out, int64_t sr, int64_t rows, int64_t cols, Span sp)
{
    pdl_wait();
    pdl_signal();
    const int64_t n = rows * cols;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        uint16_t* p = out + (i / cols) * sr + i % cols;
        if (TROP_IN(p, 2, sp)) *p = 0;
    }
}

// ------------------------------------------------------------------ host
int grid_for(int64_t n, int sm) { return (int)std::min<int64_t>((n + 255) / 256, (int64_t)sm * 8); }

template <int MODE, bool BF16, typename S>
int launch_tile(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const Job& j, const JoinJob& join, int sm,
                cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(j.units, sm / S::CG) * S::CG);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<MODE, S>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S::CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S::CG == 2 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_tile<MODE, BF16, S>, a, b, c, j, join);
    if (e != cudaSuccess) return cuda_error(e, "k_tile launch");
    count_launches(1);
    return TROP_OK;
}
template <int MODE, typename S>
int launch_tile(bool bf16, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const Job& j, int sm,
                cudaStream_t s, const JoinJob& join = JoinJob())
{
    return bf16 ? launch_tile<MODE, true, S>(a, b, c, j, join, sm, s) : launch_tile<MODE, false, S>(a, b, c, j, join, sm, s);
}

// Up to this many tokens one row tile of one CTA holds them all, and reading the weights is the work.  Forward
// against pairs of CTAs and a join of its own (back to back): 8 tokens x 4096 x 65536 93 us and 121 us; 64 x 512 x 8000
// 13.5 us and 16.5 us; 64 x 2048 x 32000 33.6 us and 34.8 us; at 128 tokens 37.7 us and 34.7 us there, 13.6 us and 16.3 us
// with 512 x 8000, 187 us and 191 us with 4096 x 131072.  Backward, 128x4096x131072: 648 us and 658 us; 128x2048x32000 104 us and
// 108 us.
constexpr int64_t FEW_TOKENS = 128;
// A logit's sum loses up to a last place of its accumulator every 16 products; past this depth two
// accumulators share it, which halves lse's error and leaves no room for a second tile.  8192 x depth x 32768, lse's
// relative error and time in one and in two accumulators: 1024 3.1e-7, 342 us and 1.5e-7, 419 us; 2048 6.2e-7, 610 us and
// 3.0e-7, 690 us; 2304 7.1e-7, 679 us and 3.4e-7, 760 us; 4096 1.3e-6, 1166 us and 6.2e-7, 1236 us.  The rule lets the error of
// 2048 products stand and pays the second accumulator where it would grow past that.  The backward pass forms
// its logits in one at every depth: what its probabilities are off by for that (2e-5 relative at 4096) is far
// below their rounding to 16 bits (2^-9, 2^-12).
constexpr int64_t DEEP_LOGITS = 2048;
// Rows of such a tile's box: the tokens' only.  The tile's other rows keep what shared memory holds,
// and so do the accumulator's, which nobody reads.
int few_rows(int64_t rows) { return (int)((rows + 7) / 8 * 8); }

// Row tiles of a band: as many as keep their operand (a row tile's whole depth) in about 48 MB of
// the L2, so that the other operand is read from memory once per band.  8192x2048x65536: all 32 row
// tiles (33 MB) 1269 us, bands of 16 / 12 / 8 / 4 1293 / 1305 / 1330 / 1378 us.
int band_of(int mt, int64_t tile_bytes) { return (int)std::min<int64_t>(mt, std::max<int64_t>(8, (48 << 20) / tile_bytes)); }

Targets targets_of(const LinearCe& q)
{
    const int64_t size[1] = {q.x.rows}, stride[1] = {q.starget};
    return {q.target, q.starget, q.ignore, q.w.rows, q.target_wide, span_of(q.target, q.target_wide ? 8 : 4, 1, size, stride)};
}

// The join of the pairs of `rows` tokens (G = 0: no pair, the sums of no token).
int launch_join(JoinJob t, float2* sums, cudaStream_t s)
{
    const int ctas = std::max(1, cdiv(t.rows, 32));
    t.sums = sums;
    const cudaError_t e = launch_pdl(k_lse_join, dim3(ctas), dim3(256), 0, s, t);
    if (e != cudaSuccess) return cuda_error(e, "k_lse_join launch");
    count_launches(1);
    return TROP_OK;
}

template <int MODE, typename S>
cudaError_t allow_smem()
{
    constexpr cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t e = cudaFuncSetAttribute(k_tile<MODE, true, S>, most, smem_bytes<MODE, S>());
    return e != cudaSuccess ? e : cudaFuncSetAttribute(k_tile<MODE, false, S>, most, smem_bytes<MODE, S>());
}

}  // namespace

int register_linear_ce_kernels()
{
    const cudaError_t e[] = {allow_smem<LSE, Pair>(), allow_smem<LSE, Deep>(), allow_smem<LSE, Few>(),
                             allow_smem<GRAD, Pair>(), allow_smem<GRAD, Few1>(), allow_smem<DX, Pair>(),
                             allow_smem<DX, Few1>(), allow_smem<DW, Pair>()};
    for (const cudaError_t r : e)
        if (r != cudaSuccess) return cuda_error(r, "cudaFuncSetAttribute(k_tile)");
    return TROP_OK;
}

int launch_linear_ce(const LinearCe& q, float* loss, float* lse, float* total, float* kept, int mean, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const int sm = dev->sm_count;
    Workspace ws(s);
    JoinJob t = {};
    t.rows = q.x.rows;
    t.tgt = targets_of(q);
    t.loss = loss;
    t.lse = lse;
    t.total = total;
    t.kept = kept;
    t.mean = mean;
    t.sp_loss = span_bytes(t.loss, (size_t)t.rows * 4);
    t.sp_lse = span_bytes(t.lse, (size_t)t.rows * 4);
    t.sp_total = span_bytes(t.total, 4);
    t.sp_kept = span_bytes(t.kept, 4);
    const size_t sums = (size_t)std::max(1, cdiv(t.rows, 32)) * sizeof(float2);
    const size_t at_sums = ws.add(sums);
    if (t.rows == 0) {
        TROP_TRY(ws.take());
        TROP_TRY(ws.ticket(&t.ticket));
        return launch_join(t, (float2*)(ws.base + at_sums), s);
    }
    Operand ox(q.x, ws), ow(q.w, ws);
    const Matrix16 &x = ox.m, &w = ow.m;
    const bool few = x.rows <= FEW_TOKENS;
    const int type = q.bf16 ? TROP_BF16 : TROP_F16;
    const int TM = few ? Few::TM : Pair::TM, TN = few ? Few::TN : Pair::TN, CG = few ? 1 : 2;
    Job j = {};
    TROP_TRY(device_error_word(&j.error));
    j.rows = (int)x.rows;
    j.cols = (int)w.rows;
    j.mt = cdiv(x.rows, TM);
    j.nt = cdiv(w.rows, TN);
    j.kt = cdiv(x.cols, few ? Few::SUB * TK : TK);
    j.kper = j.kt;
    // column tiles of a unit: the fewest rounds of tiles, then the fewest pairs to join
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 32 && c <= j.nt; ++c) {
        const int64_t cost = (int64_t)cdiv((int64_t)j.mt * cdiv(j.nt, c), sm / CG) * c;
        if (cost <= best) best = cost, j.inner = c;
    }
    const int groups = cdiv(j.nt, j.inner);
    j.units = j.mt * groups;
    j.band = band_of(j.mt, TM * x.cols * 2);
    j.tgt = t.tgt;
    t.stride = (int64_t)j.mt * TM;
    t.G = 2 * groups;
    const size_t pairs = (size_t)t.G * t.stride * sizeof(float2), at = (size_t)(x.rows + 63) / 64 * 64 * 4;
    const size_t at_part = ws.add(pairs), at_logit = ws.add(at);
    TROP_TRY(ws.take());
    TROP_TRY(ws.ticket(&t.ticket));
    TROP_TRY(pack(ox, ow, ws, sm));
    t.part = j.part = (float2*)(ws.base + at_part);
    t.at = j.at = (float*)(ws.base + at_logit);
    t.sp_part = j.sp_part = span_bytes(j.part, pairs);
    t.sp_at = j.sp_at = span_bytes(j.at, (size_t)x.rows * 4);
    const int a_rows = few ? few_rows(x.rows) : 128;
    j.a_bytes = a_rows * TK * 2;
    CUtensorMap ma, mb;
    TROP_TRY(make_map(&ma, type, x.p, x.cols, x.rows, x.ld, a_rows));
    TROP_TRY(make_map(&mb, type, w.p, w.cols, w.rows, w.ld, 128));
    if (few) return launch_tile<LSE, Few>(q.bf16, ma, mb, ma, j, sm, s, t);
    TROP_TRY((x.cols > DEEP_LOGITS ? launch_tile<LSE, Deep>(q.bf16, ma, mb, ma, j, sm, s)
                                   : launch_tile<LSE, Pair>(q.bf16, ma, mb, ma, j, sm, s)));
    return launch_join(t, (float2*)(ws.base + at_sums), s);
}

// The splits' f32 sums [ks][slab rows][lda], added in order, into rows of 16-bit elements.
int launch_split_join(bool bf16, const float* acc, int ks, int64_t slab, int64_t lda, int64_t rows, int64_t D, uint16_t* out,
                      int64_t ldo, const GradScale& grad, int sm, cudaStream_t s)
{
    const int64_t size[2] = {rows, D}, stride[2] = {ldo, 1};
    const Span sp_out = span_of(out, 2, 2, size, stride), sp_acc = span_bytes(acc, (size_t)ks * slab * lda * 4);
    const bool vec = D % 4 == 0 && ldo % 4 == 0 && ((uintptr_t)out & 7) == 0;
    const auto kernel = bf16 ? (vec ? k_split_join<true, true> : k_split_join<true, false>)
                             : (vec ? k_split_join<false, true> : k_split_join<false, false>);
    const cudaError_t e = launch_pdl(kernel, dim3(grid_for(rows * D / (vec ? 4 : 1), sm)), dim3(256), 0, s, acc, ks, slab * lda, lda,
                                     rows, D, out, ldo, grad, sp_acc, sp_out);
    if (e != cudaSuccess) return cuda_error(e, "k_split_join launch");
    count_launches(1);
    return TROP_OK;
}

int launch_linear_ce_backward(const LinearCe& q, const float* g, int64_t sg, const float* lse, const float* kept,
                              const Mat16* dx, const Mat16* dw, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const int64_t N = q.x.rows, D = q.x.cols, V = q.w.rows;
    const bool few = N <= FEW_TOKENS;
    const int type = q.bf16 ? TROP_BF16 : TROP_F16;
    const int TM = few ? Few1::TM : Pair::TM, TN = few ? Few1::TN : Pair::TN;  // of the logits and of dx
    const int sm = dev->sm_count, teams = few ? sm : sm / 2;
    const int a_rows = few ? few_rows(N) : 128;
    Workspace ws(s);
    Operand ox(q.x, ws), ow(q.w, ws);
    const Matrix16 &x = ox.m, &w = ow.m;

    // A piece of the vocabulary: P takes at most 512 MiB (and at least 4096 columns).
    const int64_t whole = (V + 255) / 256 * 256;
    int64_t piece = ((int64_t)1 << 28) / N / 256 * 256;
    piece = std::min(whole, std::max<int64_t>(piece, 4096));
    const int pieces = cdiv(V, piece);
    const int dx_mt = cdiv(N, TM), dx_nt = cdiv(D, TN), dx_kt = cdiv(std::min(piece, V), TK);
    const int dw_mt = cdiv(std::min(piece, V), Pair::TM), dw_nt = cdiv(D, Pair::TN), dw_kt = cdiv(N, TK);
    const int ks = dx ? splits(dx_mt * dx_nt, dx_kt, teams, N * D * 4) : 1;
    const int ks_w = dw ? splits(dw_mt * dw_nt, dw_kt, sm / 2, std::min(piece, V) * D * 4) : 1;
    const size_t p_bytes = (size_t)N * piece * 2;
    const bool summed = dx && (ks > 1 || pieces > 1);  // f32 sums, [ks][pad_rows][lda]
    const int64_t lda = (D + 3) / 4 * 4, pad_rows = (N + 31) / 32 * 32;
    const size_t acc_bytes = summed ? (size_t)ks * pad_rows * lda * 4 : 0;
    const int64_t pad_cols = (std::min(piece, V) + 31) / 32 * 32;
    const size_t accw_bytes = ks_w > 1 ? (size_t)ks_w * pad_cols * lda * 4 : 0;
    const size_t at_p = ws.add(p_bytes), at_acc = ws.add(acc_bytes), at_accw = ws.add(accw_bytes), at_scale = ws.add(8);
    TROP_TRY(ws.take());
    TROP_TRY(pack(ox, ow, ws, sm));
    void* const P = ws.base + at_p;
    float* const acc = (float*)(ws.base + at_acc);
    float* const accw = (float*)(ws.base + at_accw);
    float* const scale = (float*)(ws.base + at_scale);
    const int64_t gsize[1] = {N}, gstride[1] = {sg};
    GradScale grad = {g, sg, kept, nullptr, q.bf16 ? 1.f : 16384.f, span_of(g, 4, 1, gsize, gstride)};
    if (sg != 0) {
        const cudaError_t e = launch_pdl(k_gscale, dim3(1), dim3(1024), 0, s, grad, targets_of(q), N, scale);
        if (e != cudaSuccess) return cuda_error(e, "k_gscale launch");
        count_launches(1);
        grad.given = scale;
    }
    CUtensorMap x_k, w_k, x_mn, w_mn, p_k, p_mn, c;
    TROP_TRY(make_map(&x_k, type, x.p, D, N, x.ld, a_rows));
    TROP_TRY(make_map(&w_k, type, w.p, D, V, w.ld, 128));
    TROP_TRY(make_map(&x_mn, type, x.p, D, N, x.ld, 64));
    TROP_TRY(make_map(&w_mn, type, w.p, D, V, w.ld, 64));
    for (int i = 0; i < pieces; ++i) {
        const int64_t v0 = i * piece, cols = std::min(piece, V - v0);
        TROP_TRY(make_map(&p_k, type, P, cols, N, piece, a_rows));
        TROP_TRY(make_map(&p_mn, type, P, cols, N, piece, 64));
        Job j = {};
        TROP_TRY(device_error_word(&j.error));
        j.inner = 1;
        j.a_bytes = a_rows * TK * 2;
        j.grad = grad;
        {
            Job t = j;
            t.rows = (int)N;
            t.cols = (int)cols;
            t.mt = cdiv(N, TM);
            t.nt = cdiv(cols, TN);
            t.kt = t.kper = cdiv(D, TK);
            t.units = t.mt * t.nt;
            t.band = band_of(t.mt, TM * D * 2);
            t.b0 = (int)v0;
            t.v0 = v0;
            t.tgt = targets_of(q);
            t.lse = lse;
            t.sp_lse = span_bytes(lse, (size_t)N * 4);
            TROP_TRY(make_map(&c, type, P, cols, N, piece, 32));
            TROP_TRY((few ? launch_tile<GRAD, Few1>(q.bf16, x_k, w_k, c, t, sm, s)
                           : launch_tile<GRAD, Pair>(q.bf16, x_k, w_k, c, t, sm, s)));
        }
        if (dw) {
            Job t = j;
            t.rows = (int)cols;
            t.cols = (int)D;
            t.mt = cdiv(cols, Pair::TM);
            t.nt = dw_nt;
            t.kt = dw_kt;
            t.kper = cdiv(dw_kt, ks_w);
            t.a_bytes = A_BYTES;
            t.units = t.mt * t.nt * ks_w;
            uint16_t* const out = (uint16_t*)dw->p + v0 * dw->sr;
            if (ks_w > 1) {
                t.pad_rows = (int)pad_cols;
                TROP_TRY(make_map(&c, TROP_F32, accw, D, ks_w * pad_cols, lda, 32));
            } else {
                t.out = out;
                t.ldo = dw->sr;
                t.vec = ((uintptr_t)t.out & 15) == 0 && dw->sr % 8 == 0;
                const int64_t size[2] = {cols, D}, stride[2] = {dw->sr, 1};
                t.sp_out = span_of(t.out, 2, 2, size, stride);
                if (t.vec) TROP_TRY(make_map(&c, type, t.out, D, cols, t.ldo, 32));
            }
            TROP_TRY((launch_tile<DW, Pair>(q.bf16, p_mn, x_mn, ks_w > 1 || t.vec ? c : p_mn, t, sm, s)));
            if (ks_w > 1) TROP_TRY(launch_split_join(q.bf16, accw, ks_w, pad_cols, lda, cols, D, out, dw->sr, grad, sm, s));
        }
        if (dx) {
            Job t = j;
            t.rows = (int)N;
            t.cols = (int)D;
            t.mt = dx_mt;
            t.nt = dx_nt;
            t.kt = cdiv(cols, TK);
            t.kper = cdiv(dx_kt, ks);  // the last piece may have fewer splits: those it lacks stay as they are
            t.units = t.mt * t.nt * cdiv(t.kt, t.kper);
            t.bk0 = (int)v0;
            if (summed) {
                t.pad_rows = (int)pad_rows;
                t.add = i > 0;
                TROP_TRY(make_map(&c, TROP_F32, acc, D, ks * pad_rows, lda, 32));
            } else {
                t.out = dx->p;
                t.ldo = dx->sr;
                t.vec = ((uintptr_t)t.out & 15) == 0 && dx->sr % 8 == 0;
                const int64_t size[2] = {N, D}, stride[2] = {dx->sr, 1};
                t.sp_out = span_of(t.out, 2, 2, size, stride);
                if (t.vec) TROP_TRY(make_map(&c, type, t.out, D, N, t.ldo, 32));
            }
            const CUtensorMap& to = summed || t.vec ? c : p_k;
            TROP_TRY((few ? launch_tile<DX, Few1>(q.bf16, p_k, w_mn, to, t, sm, s)
                           : launch_tile<DX, Pair>(q.bf16, p_k, w_mn, to, t, sm, s)));
        }
    }
    if (summed) TROP_TRY(launch_split_join(q.bf16, acc, ks, pad_rows, lda, N, D, (uint16_t*)dx->p, dx->sr, grad, sm, s));
    return TROP_OK;
}

// Rows of 16-bit elements set to zero (gradients of an empty sum).
int launch_zero16(const Mat16& m, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const int64_t size[2] = {m.rows, m.cols}, stride[2] = {m.sr, 1};
    const cudaError_t e = launch_pdl(k_zero16, dim3(grid_for(m.rows * m.cols, dev->sm_count)), dim3(256), 0, s,
                                     (uint16_t*)m.p, m.sr, m.rows, m.cols, span_of(m.p, 2, 2, size, stride));
    if (e != cudaSuccess) return cuda_error(e, "k_zero16 launch");
    count_launches(1);
    return TROP_OK;
}

}  // namespace trop
