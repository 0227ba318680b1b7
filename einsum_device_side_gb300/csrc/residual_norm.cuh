// residual_norm.cuh -- the norms after and before a block, fused with its gate, its residual scale and the addition to the
// residual stream; forward and backward.
//
//   v = N(u) pw + pb  (or u),   r = alpha x + s a(g) v,   y = N(r) w + b              (per row)
//   N(t) = (t - mean) rstd  with  rstd = 1 / sqrt(mean_c (t - mean)^2 + eps);  of the rms norm mean = 0.
// With h = N(r), e = dy w, uh = N(u) (or u), d the whole gradient of r and J the norm's transposed Jacobian,
//   J(e, h, rstd) = rstd (e - mean_c e - h mean_c(e h))   (no middle term of the rms norm):
//   d = dr + J(e, h, rstd),  dx = alpha d,  dg = d s v a'(g),  du = J(d s a pw, uh, rstd_u)  (or d s a),
//   dw = sum_r dy h,  db = sum_r dy,  and with A1 = sum_r d a uh, A2 = sum_r d a:
//   dpw = s A1,  dpb = s A2,  ds = pw A1 + pb A2  (A1 without a norm of u).
//
// x, r and their gradients have one type (S), u, gate and theirs another (U), y and dy a third (Y): f32, bf16 or f16;
// sums, statistics and the stream inside a row are f32, and each stored value is rounded once.  y is the norm of the
// unrounded r.  The backward pass reads r, u and gate as they are or as 8-bit copies (pack8.h), which forward leaves in
// the same pass: of the stored, rounded r, so that they are what a separate call would make of it.
// Included by one file for each set of types (residual_types_*.cu), which are compiled side by side; residual_norm.cu lays
// out the jobs and chooses among them.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "residual_job.h"
#include "pack8.h"
#include "rows.h"
#include "tcgen05.h"

namespace trop {
namespace {

// A row's statistics from two passes over registers: a first mean, then the sums of the deviations from it and of their
// squares, which correct each other (Chan, Golub and LeVeque, "Algorithms for computing the sample variance", 1983): the
// first mean's error, some last places, is what the deviations' mean says, so that a constant row's mean is its value and
// its norm zero, whatever the deviation is divided by.  Squares that pass f32's range make the deviation infinite and the norm zero, as
// layer_norm's do; a NaN stays.
__device__ __forceinline__ void finish_stats(float sum, float squares, const ResJob& j, float& mean, float& rstd)
{
    const bool finite = squares < __uint_as_float(0x7f800000u);
    const float off = finite ? sum * j.inv_cols : 0.f, var = finite ? fmaxf(__fmaf_rn(-off, sum, squares), 0.f) : squares;
    mean += off;
    rstd = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(var, j.inv_cols, j.eps)));
}

// The gate's value and slope, for gates of type U.  Of 16 bits: the hardware's exponential of a rounded product, whose error grows
// with |g| (2^-22 near 0, 3.7e-6 at -85) and is far below half a step of theirs.  Of 32 bits that would lose five bits of a strongly
// negative gate's value: expf, good to 2 units in the last place (f32 silu: 16384x4096 forward 220 us, backward 388 us, with the
// product 222 and 382; 60000x1001 312 and 400 us, 300 and 385).  The reciprocal is good to one.
template <typename U>
__device__ __forceinline__ float sigmoid(float g)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + (sizeof(U) == 4 ? expf(-g) : ex2(g * -1.4426950408889634f))));
    return r;
}
template <typename U>
__device__ __forceinline__ float gate_value(float g, int act)
{
    if (act == 0) return g;
    const float s = sigmoid<U>(g);
    return act == 1 ? s : g * s;
}
template <typename U>
__device__ __forceinline__ void gate_both(float g, int act, float& value, float& slope)
{
    value = g, slope = 1.f;
    if (act == 0) return;
    const float s = sigmoid<U>(g), t = s * (1.f - s);
    value = act == 1 ? s : g * s;
    slope = act == 1 ? t : __fmaf_rn(g, t, s);
}

// ------------------------------------------------------------------ vectors of a row
// A thread's vector k of a row.  OFF: rows that do not start on 16 bytes.  A block then takes rows of one offset only
// (which repeats every `period` rows, and is the same for every tensor), so that its threads' vectors, the 16-byte granules of
// its rows, hold the same columns in all of them: column c = vector * VEC - off, and a row's first and last vector may lie
// partly outside it.
template <int VEC>
__device__ __forceinline__ int column(int k, int off) { return (int)(k * blockDim.x + threadIdx.x) * VEC - off; }
// (of the CTAs that share a row, each has a part of its vectors: `off` is then less by the parts before)
template <int VEC>
__device__ __forceinline__ bool whole(int c, int cols) { return c >= 0 && c + VEC <= cols; }

struct Walk {  // a group's rows: first, + step, ...  (rows are below 2^31, and no step passes 2^31)
    int off;
    uint32_t first, step;
};
template <typename T, int VEC, bool OFF>
__device__ __forceinline__ Walk walk_of(const void* base, int64_t stride, int period, int block, int blocks)
{
    Walk w = {0, 0, 0};
    int cls = 0;
    if (OFF) {
        cls = block % period;
        w.off = (int)(((uintptr_t)((const T*)base + cls * stride) / sizeof(T)) % VEC);
    } else {
        period = 1;
    }
    w.first = cls + period * ((uint32_t)(block / period) * blockDim.y + threadIdx.y);
    w.step = period * ((uint32_t)(blocks / period) * blockDim.y);
    return w;
}
// A row's element c.  Rows lie less than 2^32 bytes apart here, which makes their address one wide multiplication: with
// 64-bit strides the addresses were a third of the backward pass's instructions.
template <typename T>
__device__ __forceinline__ T* elem(const RowsAt& a, uint32_t row, int c)
{
    return reinterpret_cast<T*>((char*)a.p + (uint64_t)row * a.sb) + c;
}
__device__ __forceinline__ int8_t* codes_at(const Rows8& a, uint32_t row, int c) { return a.codes + (uint64_t)row * a.sb + c; }
__device__ __forceinline__ uint8_t* scales_at(const Rows8& a, uint32_t row, int group) { return a.scales + (uint64_t)row * a.ssb + group; }

template <typename T, int VEC, bool OFF>
__device__ __forceinline__ void put(const RowsAt& a, uint32_t row, int c, const Raw<T, VEC>& q, int cols)
{
    T* p = elem<T>(a, row, c);
    if (!OFF || whole<VEC>(c, cols)) {
        if (c < cols && TROP_IN(p, VEC * sizeof(T), a.sp)) q.write(p);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i >= 0 && c + i < cols && TROP_IN(p + i, sizeof(T), a.sp)) p[i] = from_f32<T>(q.get(i));
    }
}
template <typename T, int VEC, bool OFF>
__device__ __forceinline__ void put(const RowsAt& a, uint32_t row, int c, const Pair<VEC> (&o)[pairs<VEC>], int cols)
{
    float v[VEC];
    apart<VEC>(o, v);
    Raw<T, VEC> q;
    q.set(v);
    put<T, VEC, OFF>(a, row, c, q, cols);
}

// VEC elements of a vector over the columns: f32, or of type T; `none` where it is absent, zero outside the row.  SHARED: from
// the block's shared copies (five, in the order of the job's), moved by the row's offset.  They spare the address and the checks of
// every row's five loads; 32-bit vectors of on-grid rows stay in L1, which has the room that the copies would take.  Forward, where
// an SM has four blocks, each with copies of its own, that holds for all but blocks of several rows (65536x512 bf16 67 us
// against 79; 4096x8192 f16 with copies 146 us against 108).
template <typename T, int VEC, bool OFF, bool SHARED>
struct Vectors {
    const uint8_t* shared;
    int span;  // bytes of one
    template <typename V>
    __device__ __forceinline__ void read(const V* p, float (&v)[VEC]) const
    {
        Raw<V, VEC> q;
        q.read(p);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = q.get(i);
    }
    __device__ __forceinline__ void fetch(const VecAt& a, int c, const ResJob& j, float none, float (&v)[VEC]) const
    {
        if (!a.p || c >= (int)j.cols) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = c < (int)j.cols ? none : 0.f;
        } else if (j.wide_w) {
            load<float, VEC>((const float*)a.p + c, v, a.sp);
        } else {
            load<T, VEC>((const T*)a.p + c, v, a.sp);
        }
    }
    __device__ __forceinline__ void get(int which, const VecAt& a, int k, int c, const ResJob& j, float none, Pair<VEC> (&o)[pairs<VEC>]) const
    {
        float v[VEC];
        if (SHARED) {
            const int at = (k * blockDim.x + threadIdx.x) * VEC;
            if (j.wide_w) read((const float*)(shared + which * span) + at, v);
            else read((const T*)(shared + which * span) + at, v);
        } else {
            fetch(a, c, j, none, v);
        }
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) o[i] = pair_at<VEC>(v, i);
    }
    // all of the block; five of NV * blockDim.x vectors each
    template <int NV>
    __device__ __forceinline__ void init(uint8_t* dyn, int off, const ResJob& j)
    {
        shared = dyn;
        span = NV * blockDim.x * VEC * (j.wide_w ? 4 : (int)sizeof(T));
        if constexpr (!SHARED) return;
        const VecAt all[5] = {j.w, j.b, j.pw, j.pb, j.s};
        const float none[5] = {1.f, 0.f, 1.f, 0.f, 1.f};
        if constexpr (!OFF) {
            if (threadIdx.y == 0)
#pragma unroll
                for (int which = 0; which < 5; ++which)
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        float v[VEC];
                        fetch(all[which], column<VEC>(k, off), j, none[which], v);
                        const int at = (k * blockDim.x + threadIdx.x) * VEC;
                        if (j.wide_w) {
                            Raw<float, VEC> q;
                            q.set(v);
                            q.write((float*)(dyn + which * span) + at);
                        } else {
                            Raw<T, VEC> q;
                            q.set(v);
                            q.write((T*)(dyn + which * span) + at);
                        }
                    }
        } else {
            for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < NV * VEC * (int)blockDim.x; i += blockDim.x * blockDim.y) {
                const int c = i - off;
                const bool in = c >= 0 && c < (int)j.cols;
                float v[5];
#pragma unroll
                for (int which = 0; which < 5; ++which) {
                    const VecAt& a = all[which];
                    v[which] = !in ? 0.f : !a.p ? none[which] : j.wide_w ? (TROP_IN((const float*)a.p + c, 4, a.sp) ? ((const float*)a.p)[c] : 0.f)
                               : TROP_IN((const T*)a.p + c, sizeof(T), a.sp) ? to_f32(((const T*)a.p)[c]) : 0.f;
                }
#pragma unroll
                for (int which = 0; which < 5; ++which) {
                    if (j.wide_w) ((float*)(dyn + which * span))[i] = v[which];
                    else ((T*)(dyn + which * span))[i] = from_f32<T>(v[which]);
                }
            }
        }
        __syncthreads();
    }
};
// (a number's scale may need more digits than T has: it is a factor of its own where there is no vector of it)

// ------------------------------------------------------------------ rows on their way
// A group's rows come through shared memory ahead of their turn: a stage of the ring holds a row of every tensor, and the
// barrier of a later sum says that it has been read.  Rows on 16 bytes come by one bulk copy a tensor, which an mbarrier counts.
// Of the others (OFF) every thread copies its own vectors and waits for those alone.
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes, bool in)
{
    const int n = in ? bytes : 0;  // (what is not there arrives as zeros; its address has to be aligned all the same)
    if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
    else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait(int stages)  // the oldest of `stages` groups
{
    if (stages >= 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// a row with `n` others before it and after it
__device__ __forceinline__ bool amid(uint32_t row, uint32_t n, const ResJob& j) { return row >= n && row + n < (uint32_t)j.rows; }

// One tensor's part of a stage: BYTES for each vector of each thread.  OFF: a piece of every thread's beside the others'.  `to`:
// the part's shared address; `t` of `threads`.
template <typename T, int VEC, bool CODED, bool OFF>
struct In {
    static constexpr int BYTES = VEC * sizeof(T), PIECE = BYTES < 16 ? BYTES : 16;
    // Whether the vector lies in the matrix, whatever row of it: all in its row, or over the edge of a row with others on both sides
    // that lie far enough off.  (By 32-bit comparisons that the tensors
    // share: 65536x1001 bf16 backward 370 us; by those of their 64-bit addresses 425 us.)
    static __device__ __forceinline__ bool inside(uint32_t row, int c, const RowsAt& a, const ResJob& j)
    {
        return !OFF || whole<VEC>(c, (int)j.cols) || (amid(row, 1, j) && a.sb >= VEC * sizeof(T));
    }
    static __device__ __forceinline__ void issue(uint32_t to, int t, int threads, const RowsAt& a, const Rows8&, uint32_t row, int c, const ResJob& j)
    {
        if (c >= (int)j.cols) return;
        const T* p = elem<T>(a, row, c);
        const bool in = inside(row, c, a, j) && TROP_IN(p, BYTES, a.sp);
#pragma unroll
        for (int i = 0; i < BYTES / PIECE; ++i)
            copy_async(to + (i * threads + t) * PIECE, reinterpret_cast<const char*>(p) + i * PIECE, PIECE, in);
    }
    static __device__ __forceinline__ void take(Raw<T, VEC>& q, uint32_t to, int t, int threads, const RowsAt& a, uint32_t row, int c, const ResJob& j)
    {
        const int cols = (int)j.cols;
        q.zero();
        if (c >= cols) return;
#pragma unroll
        for (int i = 0; i < BYTES / PIECE; ++i) {
            const uint32_t from = OFF ? to + (i * threads + t) * PIECE : to + t * BYTES + i * PIECE;
            if constexpr (PIECE == 16)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(q.w[4 * i]), "=r"(q.w[4 * i + 1]), "=r"(q.w[4 * i + 2]), "=r"(q.w[4 * i + 3])
                             : "r"(from)
                             : "memory");
            else
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(q.w[0]), "=r"(q.w[1]) : "r"(from) : "memory");
        }
        if (OFF && !whole<VEC>(c, cols)) {
            const T* p = elem<T>(a, row, c);
            if (inside(row, c, a, j)) {
                constexpr int E = 4 / sizeof(T);  // elements of a word
#pragma unroll
                for (int i = 0; i < Raw<T, VEC>::N; ++i) {
                    uint32_t mask = 0;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (c + i * E + e >= 0 && c + i * E + e < cols) mask |= (E == 1 ? 0xffffffffu : 0xffffu) << 16 * e;
                    q.w[i] &= mask;
                }
            } else {  // at the matrix's own ends: one by one
                float v[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = c + i >= 0 && c + i < cols && TROP_IN(p + i, sizeof(T), a.sp) ? to_f32(p[i]) : 0.f;
                q.set(v);
            }
        }
    }
    static __device__ __forceinline__ void take(Pair<VEC> (&o)[pairs<VEC>], uint32_t to, int t, int threads, const RowsAt& a, const Rows8&, uint32_t row,
                                                int c, uint32_t, const ResJob& j)
    {
        Raw<T, VEC> q;
        take(q, to, t, threads, a, row, c, j);
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) o[i] = pair_of<T, VEC>(q, i);
    }
};
// 8-bit copies.  Of rows on 16 bytes the codes alone come this way (`e`: the scale, fetched a row ahead).  Of the others the
// aligned words around the codes, shifted together afterwards, and the words of the two groups that they may lie in.  Words that reach outside the matrix are not
// copied; their bytes are read when they are wanted.
template <typename T, int VEC>
struct In<T, VEC, true, false> {
    static constexpr int BYTES = VEC;
    static __device__ __forceinline__ void take(Pair<VEC> (&o)[pairs<VEC>], uint32_t to, int t, int, const RowsAt&, const Rows8&, uint32_t,
                                                int c, uint32_t e, const ResJob& j)
    {
        Codes<VEC> k;
        k.zero();
        if (c < (int)j.cols) {
            if constexpr (VEC == 8)
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(k.w[0]), "=r"(k.w[1]) : "r"(to + t * 8) : "memory");
            else
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(k.w[0]) : "r"(to + t * 4) : "memory");
        }
        float v[VEC];
        values8<VEC>(k.w, unit8(e), v);
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) o[i] = pair_at<VEC>(v, i);
    }
};
template <typename T, int VEC>
struct In<T, VEC, true, true> {
    static constexpr int WORDS = VEC / 4 + 1, SCALES = 2, BYTES = 4 * (WORDS + SCALES);
    static __device__ __forceinline__ const uint8_t* scale_at(const Rows8& a, uint32_t row, int c, int which, const ResJob& j)
    {
        return scales_at(a, row, (which ? min(c + VEC - 1, (int)j.cols - 1) : max(c, 0)) / GROUP8);
    }
    // the words around a scale, up to three bytes to either side; and around the codes
    static __device__ __forceinline__ bool scale_inside(uint32_t row, int c, int which, const Rows8& a, const ResJob& j)
    {
        const int g = (which ? min(c + VEC - 1, (int)j.cols - 1) : max(c, 0)) / GROUP8;
        return (g >= 3 && (g + 3) * GROUP8 < (int)j.cols) || (amid(row, 3, j) && a.ssb >= 1);
    }
    static __device__ __forceinline__ bool inside(uint32_t row, int c, const Rows8& a, const ResJob& j)
    {
        return (c >= 3 && c + 4 * WORDS <= (int)j.cols) || (amid(row, 1, j) && a.sb >= 16);
    }
    static __device__ __forceinline__ void issue(uint32_t to, int t, int threads, const RowsAt&, const Rows8& a, uint32_t row, int c, const ResJob& j)
    {
        if (c >= (int)j.cols) return;
        const int8_t* p = codes_at(a, row, c);
        const int8_t* w = p - ((uintptr_t)p & 3);
        const bool in = inside(row, c, a, j) && TROP_IN(w, 4 * WORDS, a.sp_c);
#pragma unroll
        for (int i = 0; i < WORDS; ++i) copy_async(to + (i * threads + t) * 4, w + 4 * i, 4, in);
#pragma unroll
        for (int i = 0; i < SCALES; ++i) {
            const uint8_t* q = scale_at(a, row, c, i, j);
            const bool there = scale_inside(row, c, i, a, j);
            const uint8_t* word = q - ((uintptr_t)q & 3);
            const bool ok = there && TROP_IN(word, 4, a.sp_s);
            copy_async(to + ((WORDS + i) * threads + t) * 4, (const void*)((uintptr_t)word), 4, ok);
        }
    }
    static __device__ __forceinline__ void take(Pair<VEC> (&o)[pairs<VEC>], uint32_t to, int t, int threads, const RowsAt&, const Rows8& a, uint32_t row,
                                                int c, uint32_t, const ResJob& j)
    {
        const int cols = (int)j.cols;
        Codes<VEC> k;
        k.zero();
        uint32_t e[SCALES];
#pragma unroll
        for (int i = 0; i < SCALES; ++i) e[i] = LEAST8;
        if (c < cols) {
            const int8_t* p = codes_at(a, row, c);
            if (inside(row, c, a, j)) {
                uint32_t w[WORDS];
#pragma unroll
                for (int i = 0; i < WORDS; ++i)
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(to + (i * threads + t) * 4) : "memory");
#pragma unroll
                for (int i = 0; i + 1 < WORDS; ++i) k.w[i] = __funnelshift_r(w[i], w[i + 1], ((uint32_t)(uintptr_t)p & 3) * 8);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i >= 0 && c + i < cols && TROP_IN(p + i, 1, a.sp_c)) k.w[i / 4] |= (uint32_t)(uint8_t)p[i] << 8 * (i % 4);
            }
            if (!whole<VEC>(c, cols)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i < 0 || c + i >= cols) k.w[i / 4] &= ~(0xffu << 8 * (i % 4));
            }
#pragma unroll
            for (int i = 0; i < SCALES; ++i) {
                const uint8_t* q = scale_at(a, row, c, i, j);
                uint32_t w;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(to + ((WORDS + i) * threads + t) * 4) : "memory");
                e[i] = w >> ((uint32_t)(uintptr_t)q & 3) * 8 & 0xffu;
                if (!scale_inside(row, c, i, a, j)) e[i] = TROP_IN(q, 1, a.sp_s) ? *q : LEAST8;
            }
        }
        float v[VEC];
        const float unit = unit8(e[0]);
        const float other = unit8(e[SCALES - 1]);
        const int edge = max(c, 0) / GROUP8 * GROUP8 + GROUP8 - c;  // elements up to the first group's end
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = coded8(k.w[i / 4] ^ 0x80808080u, i % 4) * (i < edge ? unit : other);
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) o[i] = pair_at<VEC>(v, i);
    }
};

// A group's ring of bulk copies: part `i` of a stage begins at `at[i]`.  A copy that did not land in its bounded wait is
// reported, after which nothing more is fetched or waited for.
struct Ring {
    uint64_t* full;  // [4], the group's
    bool ok;
    __device__ __forceinline__ void init(uint64_t (*all)[4], int stages)
    {
        full = all[threadIdx.y];
        ok = true;
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i) mbar_init(full + i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncthreads();
    }
    __device__ __forceinline__ void wait(int slot, uint32_t phase, uint32_t* error)
    {
        if (ok && !mbar_wait(full + slot, phase)) {
            ok = false;
            *(volatile uint32_t*)error = 1;
            __threadfence_system();
        }
    }
    // after a failure: the copies still on their way get one more wait each before the block leaves
    __device__ __forceinline__ void leave(int stages)
    {
        if (ok || threadIdx.x != 0) return;
        for (int i = 0; i < 2 * stages; ++i) (void)mbar_wait(full + i % stages, i / stages);
    }
};
template <typename T>
__device__ __forceinline__ bool row_in(const RowsAt& a, uint32_t row, int c, int n)
{
    return TROP_IN(elem<T>(a, row, c), n * sizeof(T), a.sp);
}
__device__ __forceinline__ void bulk_to(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from), "r"(bytes),
                 "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ float row_gate(const ResJob& j, uint32_t row, bool is_f32, bool is_bf16)
{
    if (is_f32) {
        const float* p = (const float*)j.g.p + row * j.g.s;
        return TROP_IN(p, 4, j.g.sp) ? *p : 0.f;
    }
    const uint16_t* p = (const uint16_t*)j.g.p + row * j.g.s;
    const uint16_t h = TROP_IN(p, 2, j.g.sp) ? *p : (uint16_t)0;
    return is_bf16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}
template <typename U>
__device__ __forceinline__ float row_gate(const ResJob& j, uint32_t row)
{
    return row_gate(j, row, sizeof(U) == 4, std::is_same<U, bf16>::value);
}
template <typename U>
__device__ __forceinline__ void put_row_gate(const ResJob& j, uint32_t row, float v)
{
    U* p = (U*)j.dg.p + row * j.dg.s;
    if (TROP_IN(p, sizeof(U), j.dg.sp)) *p = from_f32<U>(v);
}
__device__ __forceinline__ float stat(const ResJob& j, int which, uint32_t row)
{
    const float* p = j.stats + which * j.rows + row;
    return TROP_IN(p, 4, j.sp_stats) ? *p : 0.f;
}
__device__ __forceinline__ void put_stat(const ResJob& j, int which, uint32_t row, float v)
{
    float* p = j.stats + which * j.rows + row;
    if (j.stats && TROP_IN(p, 4, j.sp_stats)) *p = v;
}

// The codes of a group's lanes (all of the warp take part; `live`: this one's vector is in the row).
template <typename T, int VEC>
__device__ __forceinline__ void keep(const Rows8& a, uint32_t row, int64_t c, bool live, const Raw<T, VEC>& q)
{
    const uint32_t e = scale8(group_top8<VEC>(live ? top8<T, VEC>(q) : 0u));
    if (!live) return;
    Codes<VEC> k;
    codes8<T, VEC>(q, e, k.w);
    int8_t* p = a.codes + row * a.sc + c;
    uint8_t* s = a.scales + row * a.ss + c / GROUP8;
    if (TROP_IN(p, VEC, a.sp_c)) k.write(p);
    if (c % GROUP8 == 0 && TROP_IN(s, 1, a.sp_s)) *s = (uint8_t)e;
}

// The sums over either half of a warp, for all of it.
__device__ __forceinline__ void halves(float v, float& a, float& b)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const float w = __shfl_xor_sync(0xffffffffu, v, 16);
    const bool up = threadIdx.x & 16;
    a = up ? w : v;
    b = up ? v : w;
}
// Two sums over a row's group (a warp, or the whole block): each half of a warp takes one of them, so that five shuffles
// serve both, of the warps' sums too.  Callers alternate between two of `sh`, [2][32] floats that
// start as zeros, which leaves one barrier a call.
__device__ __forceinline__ void row_sums(float& a, float& b, float (*sh)[32])
{
    const bool up = threadIdx.x & 16;
    float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (blockDim.x == 32) {
        const float w = __shfl_xor_sync(0xffffffffu, v, 16);
        a = up ? w : v;
        b = up ? v : w;
        return;
    }
    if ((threadIdx.x & 15) == 0) sh[up][threadIdx.x >> 5] = v;
    __syncthreads();
    const int l = threadIdx.x & 15;
    v = sh[up][l];
    if (blockDim.x > 512) v += sh[up][l + 16];
    halves(v, a, b);
}
// The same where `ctas` CTAs of a cluster share the row, up to eight of 16 warps: every warp hands its two sums to all of them by
// asynchronous stores, which each CTA's mbarrier counts.  (A barrier of the cluster's also waits for the row's stores to
// memory: 4096x8192 f16 from copies, 253 us.)  Callers alternate as above: whoever has a turn's sums knows that all warps have read
// those of the turn before.  A wait that runs out is reported.
struct WideSums {
    float2 (*sh)[128];
    uint64_t* bar;
    uint32_t rank, ctas, phases;
    __device__ __forceinline__ void init()
    {
        phases = 0;
        if (threadIdx.x == 0) {
            for (int i = 0; i < 3; ++i) mbar_init(bar + i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    __device__ __forceinline__ void operator()(float& a, float& b, int which, uint32_t* error)
    {
        const bool up = threadIdx.x & 16;
        float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
        halves(v, a, b);
        const uint32_t warps = blockDim.x >> 5, to = threadIdx.x & 31;
        if (threadIdx.x == 0) mbar_expect_tx(bar + which, ctas * warps * 8);
        if (to < ctas)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                             mapa(smem_u32(&sh[which][rank * 16 + (threadIdx.x >> 5)]), to)),
                         "f"(a), "f"(b), "r"(mapa(smem_u32(bar + which), to))
                         : "memory");
        if (!mbar_wait_cluster(bar + which, phases >> which & 1)) {
            *(volatile uint32_t*)error = 1;
            __threadfence_system();
        }
        phases ^= 1u << which;
        const float4 p = *reinterpret_cast<const float4*>(&sh[which][4 * to]), q = *reinterpret_cast<const float4*>(&sh[which][4 * to + 2]);
        a = (p.x + p.z) + (q.x + q.z);
        b = (p.y + p.w) + (q.y + q.w);
        v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
        halves(v, a, b);
    }
};
__device__ __forceinline__ void zero_sums(float* sh, int n)
{
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < n; i += blockDim.x * blockDim.y) sh[i] = 0.f;
    if (blockDim.x > 32) __syncthreads();
}

// ------------------------------------------------------------------ forward
// A group of threads, a warp or a block, has a row, which stays in registers between the norms: 16 elements a thread where
// there are many rows.  16384x4096 with a gate: f32 stream beside bf16 158 to 166 us, 5.7 to 6.0 TB/s, memory's rate; all bf16 162 us, 4.1 TB/s,
// and with 8-bit copies 233 us, both bound by instructions (72 % of the issue slots: unpacking, three passes over the
// row, codes).  Elements are worked on in packed pairs: one at a time, 81 instructions an element, it was 206 us.
template <int VEC, int NV>
using Pairs = Pair<VEC>[NV][pairs<VEC>];

// Mean and rstd of a row in a group's registers (zeros outside it).
template <int VEC, int NV, bool OFF>
__device__ __forceinline__ void row_stats(const ResJob& j, const Pairs<VEC, NV>& t, int off, float (*sh)[2][32], int& turn, float& mean,
                                          float& rstd)
{
    const int cols = (int)j.cols;
    float s0 = 0.f, s1 = 0.f;
    mean = 0.f;
    if (!j.rms) {
        Pair<VEC> a = p_of<Pair<VEC>>(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) a = p_add(a, t[k][i]);
        s0 = p_sum(a);
        row_sums(s0, s1, sh[turn]);
        turn ^= 1;
        mean = s0 * j.inv_cols;
    }
    Pair<VEC> a = p_of<Pair<VEC>>(0.f), b = a;
    float edge_a = 0.f, edge_b = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = column<VEC>(k, off);
        if (OFF ? whole<VEC>(c, cols) : c < cols) {
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) {
                const Pair<VEC> d = p_add(t[k][i], p_of<Pair<VEC>>(-mean));
                a = p_add(a, d);
                b = p_fma(d, d, b);
            }
        } else if (OFF && c < cols) {
            float v[VEC];
            apart<VEC>(t[k], v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = c + i >= 0 && c + i < cols ? v[i] - mean : 0.f;
                edge_a += d;
                edge_b = __fmaf_rn(d, d, edge_b);
            }
        }
    }
    s0 = j.rms ? 0.f : p_sum(a) + edge_a;
    s1 = p_sum(b) + edge_b;
    row_sums(s0, s1, sh[turn]);
    turn ^= 1;
    finish_stats(s0, s1, j, mean, rstd);
}

// t times the gate of a vector
template <typename U, int VEC>
__device__ __forceinline__ void gated(Pair<VEC> (&t)[pairs<VEC>], const Pair<VEC> (&g)[pairs<VEC>], int act)
{
    if (act == 0) {
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) t[i] = p_mul(t[i], g[i]);
    } else {
        float v[VEC];
        apart<VEC>(g, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = gate_value<U>(v[i], act);
#pragma unroll
        for (int i = 0; i < pairs<VEC>; ++i) t[i] = p_mul(t[i], pair_at<VEC>(v, i));
    }
}

// (f32 vectors beside f32 rows would leave no room for two stages)
template <typename U, typename Y, bool OFF>
constexpr bool shared_vectors = OFF || (sizeof(U) == 2 && sizeof(Y) == 2);

template <typename S, typename U, typename Y, int VEC, int NV, int MAXT, bool OFF, bool SHARED = OFF>
__global__ void __launch_bounds__(MAXT) k_residual(const ResJob j, int period, int stages, uint32_t* error)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) float sh[2][2][32];
    __shared__ __align__(8) uint64_t full[8][4];
    zero_sums(&sh[0][0][0], 128);
    const int cols = (int)j.cols;
    const Walk walk = walk_of<U, VEC, OFF>(j.u.p, j.u.s, period, blockIdx.x, gridDim.x);
    Vectors<Y, VEC, OFF, SHARED> vec;
    vec.template init<NV>(dyn, walk.off, j);
    const float scale = j.s.p ? 1.f : j.scale;
    using InU = In<U, VEC, false, OFF>;
    using InS = In<S, VEC, false, OFF>;
    const int wide = OFF ? blockDim.x * blockDim.y : blockDim.x;  // threads whose vectors lie together
    const int t0 = OFF ? threadIdx.y * blockDim.x + threadIdx.x : threadIdx.x;
    const int at_x = NV * InU::BYTES * wide, at_g = at_x + NV * InS::BYTES * wide;
    const int size = at_g + (j.gate == GATE_FULL ? NV * InU::BYTES * wide : 0), stage = OFF ? size : size * blockDim.y;
    const uint32_t base = smem_u32(dyn) + (SHARED ? 5 * vec.span : 0) + (OFF ? 0 : threadIdx.y * size);
    Ring ring;
    if (!OFF) ring.init(full, stages);
    auto issue = [&](uint32_t row, int slot) {
        const uint32_t to = base + slot * stage;
        if constexpr (OFF) {
            if (row < (uint32_t)j.rows) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = column<VEC>(k, walk.off);
                    InU::issue(to + k * InU::BYTES * wide, t0, wide, j.u, j.ku, row, c, j);
                    InS::issue(to + at_x + k * InS::BYTES * wide, t0, wide, j.x, j.kr, row, c, j);
                    if (j.gate == GATE_FULL) InU::issue(to + at_g + k * InU::BYTES * wide, t0, wide, j.g, j.kg, row, c, j);
                }
            }
            copies_commit();
        } else if (threadIdx.x == 0 && row < (uint32_t)j.rows && ring.ok) {
            const bool g = j.gate == GATE_FULL;
            if (row_in<U>(j.u, row, 0, cols) && row_in<S>(j.x, row, 0, cols) && (!g || row_in<U>(j.g, row, 0, cols))) {
                const uint32_t bu = cols * sizeof(U), bx = cols * sizeof(S);
                uint64_t* const bar = ring.full + slot;
                mbar_expect_tx(bar, bx + (g ? 2 : 1) * bu);
                bulk_to(to, elem<U>(j.u, row, 0), bu, bar);
                bulk_to(to + at_x, elem<S>(j.x, row, 0), bx, bar);
                if (g) bulk_to(to + at_g, elem<U>(j.g, row, 0), bu, bar);
            } else {
                mbar_expect_tx(ring.full + slot, 0);
            }
        }
    };
    for (int i = 0; i < stages; ++i) issue(walk.first + i * walk.step, i);
    int turn = 0, slot = 0;
    uint32_t phase = 0;
    float gate = 0.f;
    if (j.gate == GATE_ROW && walk.first < (uint32_t)j.rows) gate = row_gate<U>(j, walk.first);
    for (uint32_t row = walk.first; row < (uint32_t)j.rows; row += walk.step) {
        const float ga = scale * (j.gate == GATE_ROW ? gate_value<U>(gate, j.act) : 1.f);
        if (j.gate == GATE_ROW && row + walk.step < (uint32_t)j.rows) gate = row_gate<U>(j, row + walk.step);
        if (OFF) copies_wait(stages);
        else ring.wait(slot, phase, error);
        const uint32_t from = base + slot * stage;
        Pairs<VEC, NV> t;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column<VEC>(k, walk.off);
            Raw<U, VEC> q;
            InU::take(q, from + k * InU::BYTES * wide, t0, wide, j.u, row, c, j);
            if (!OFF && j.ku.codes) keep<U, VEC>(j.ku, row, c, c < cols, q);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) t[k][i] = pair_of<U, VEC>(q, i);
        }
        float um = 0.f, ur = 1.f, mean, rstd;
        if (j.post) row_stats<VEC, NV, OFF>(j, t, walk.off, sh, turn, um, ur);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column<VEC>(k, walk.off);
            Pair<VEC> f[pairs<VEC>], o[pairs<VEC>];
            if (j.post) {
                vec.get(2, j.pw, k, c, j, 1.f, f);
                vec.get(3, j.pb, k, c, j, 0.f, o);
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i)
                    t[k][i] = p_fma(p_mul(p_add(t[k][i], p_of<Pair<VEC>>(-um)), p_of<Pair<VEC>>(ur)), f[i], o[i]);
            }
            if (j.s.p) {
                vec.get(4, j.s, k, c, j, 1.f, f);
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) t[k][i] = p_mul(t[k][i], f[i]);
            }
            if (j.gate == GATE_FULL) {
                Raw<U, VEC> g;
                InU::take(g, from + at_g + k * InU::BYTES * wide, t0, wide, j.g, row, c, j);
                if (!OFF && j.kg.codes) keep<U, VEC>(j.kg, row, c, c < cols, g);
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) o[i] = pair_of<U, VEC>(g, i);
                gated<U, VEC>(t[k], o, j.act);
            }
            Raw<S, VEC> q;
            InS::take(q, from + at_x + k * InS::BYTES * wide, t0, wide, j.x, row, c, j);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i)
                t[k][i] = p_fma(p_of<Pair<VEC>>(j.alpha), pair_of<S, VEC>(q, i), p_mul(t[k][i], p_of<Pair<VEC>>(ga)));
            float v[VEC];
            apart<VEC>(t[k], v);
            q.set(v);
            put<S, VEC, OFF>(j.r, row, c, q, cols);
            if (!OFF && j.kr.codes) keep<S, VEC>(j.kr, row, c, c < cols, q);
        }
        row_stats<VEC, NV, OFF>(j, t, walk.off, sh, turn, mean, rstd);
        if (!OFF && blockDim.x == 32) __syncwarp();
        issue(row + stages * walk.step, slot);  // (all of the group have passed a sum since they read the stage)
        if (++slot == stages) slot = 0, phase ^= 1;
        if (threadIdx.x == 0) put_stat(j, 0, row, um), put_stat(j, 1, row, ur), put_stat(j, 2, row, mean), put_stat(j, 3, row, rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column<VEC>(k, walk.off);
            if (c >= cols) continue;
            Pair<VEC> f[pairs<VEC>], o[pairs<VEC>];
            vec.get(0, j.w, k, c, j, 1.f, f);
            vec.get(1, j.b, k, c, j, 0.f, o);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i)
                f[i] = p_fma(p_mul(p_add(t[k][i], p_of<Pair<VEC>>(-mean)), p_of<Pair<VEC>>(rstd)), f[i], o[i]);
            put<Y, VEC, OFF>(j.y, row, c, f, cols);
        }
    }
    if (!OFF) ring.leave(stages);
}

// The scalar forms that the long rows' kernels use.
template <typename T>
__device__ __forceinline__ float one_of(const VecAt& a, int64_t c, const ResJob& j, float none)
{
    if (!a.p) return none;
    if (j.wide_w) return TROP_IN((const float*)a.p + c, 4, a.sp) ? ((const float*)a.p)[c] : 0.f;
    return TROP_IN((const T*)a.p + c, sizeof(T), a.sp) ? to_f32(((const T*)a.p)[c]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void put_one(const RowsAt& a, int64_t row, int64_t c, float v)
{
    T* p = (T*)a.p + row * a.s + c;
    if (TROP_IN(p, sizeof(T), a.sp)) *p = from_f32<T>(v);
}

// Rows longer than a block's registers, or whose tensors do not lie alike: a block per row walks over it once for every sum; r
// is formed again each time.
template <typename S, typename U, typename Y>
__global__ void __launch_bounds__(1024) k_residual_long(const ResJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[2][32][1];
    const int64_t row = blockIdx.x;
    const float ga = j.gate == GATE_ROW ? gate_value<U>(row_gate<U>(j, row), j.act) : 1.f;
    int turn = 0;
    auto of = [&](const RowsAt& a, int64_t c, auto type) {
        using T = decltype(type);
        const T* p = (const T*)a.p + row * a.s + c;
        return c < j.cols && TROP_IN(p, sizeof(T), a.sp) ? to_f32(*p) : 0.f;
    };
    // sum over the row of f(column)
    auto sum = [&](auto f) {
        float s[1] = {0.f};
        for (int64_t c = threadIdx.x; c < j.cols; c += blockDim.x) s[0] += f(c);
        group_sum_turn<1>(s, sh[turn]);
        turn ^= 1;
        return s[0];
    };
    auto stats = [&](auto f, float& mean, float& rstd) {
        mean = j.rms ? 0.f : sum(f) * j.inv_cols;
        const float m = mean, off = j.rms ? 0.f : sum([&](int64_t c) { return f(c) - m; });
        finish_stats(off, sum([&](int64_t c) { return (f(c) - m) * (f(c) - m); }), j, mean, rstd);
    };
    float um = 0.f, ur = 1.f, mean, rstd;
    auto u_at = [&](int64_t c) { return of(j.u, c, U()); };
    if (j.post) stats(u_at, um, ur);
    auto r_at = [&](int64_t c) {
        float t = u_at(c);
        if (j.post) t = __fmaf_rn((t - um) * ur, one_of<Y>(j.pw, c, j, 1.f), one_of<Y>(j.pb, c, j, 0.f));
        return __fmaf_rn(j.alpha, of(j.x, c, S()), t * one_of<Y>(j.s, c, j, j.scale) * (j.gate == GATE_FULL ? gate_value<U>(of(j.g, c, U()), j.act) : ga));
    };
    stats(r_at, mean, rstd);
    if (threadIdx.x == 0) put_stat(j, 0, row, um), put_stat(j, 1, row, ur), put_stat(j, 2, row, mean), put_stat(j, 3, row, rstd);
    for (int64_t c0 = 0; c0 < j.cols; c0 += blockDim.x) {
        const int64_t c = c0 + threadIdx.x;
        const bool live = c < j.cols;
        const float t = live ? r_at(c) : 0.f;
        const float one[1] = {t};
        Raw<S, 1> q;
        q.set(one);
        if (live) {
            S* r = (S*)j.r.p + row * j.r.s + c;
            if (TROP_IN(r, sizeof(S), j.r.sp)) q.write(r);
            put_one<Y>(j.y, row, c, __fmaf_rn((t - mean) * rstd, one_of<Y>(j.w, c, j, 1.f), one_of<Y>(j.b, c, j, 0.f)));
        }
        if (j.kr.codes) keep<S, 1>(j.kr, row, c, live, q);
        if (j.ku.codes) {
            Raw<U, 1> v;
            const float uv[1] = {live ? u_at(c) : 0.f};
            v.set(uv);
            keep<U, 1>(j.ku, row, c, live, v);
            if (j.gate == GATE_FULL) {
                const float gv[1] = {live ? of(j.g, c, U()) : 0.f};
                v.set(gv);
                keep<U, 1>(j.kg, row, c, live, v);
            }
        }
    }
}

// ------------------------------------------------------------------ backward
// d, the whole gradient of r, from dr, e = dy w and h.
__device__ __forceinline__ float grad_r(float dr, float e, float h, float rstd, float flat, float along)
{
    return __fmaf_rn(rstd, e - flat - h * along, dr);
}

// A block's column sums into its rows of the partial sums; blocks of several warps that each took rows of their own add
// theirs in warp order, through `across` [warps][cols].
template <int VEC, int NV>
__device__ __forceinline__ void put_partials(const ResJob& j, const Pair<VEC> (&acc)[4][NV][pairs<VEC>], float* across, int off, int block)
{
    const int cols = (int)j.cols;
#pragma unroll
    for (int which = 0; which < 4; ++which) {
        if (!(j.want >> which & 1)) continue;
        float* part = j.part + ((int64_t)block * 4 + which) * cols;
        if (blockDim.y > 1) __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column<VEC>(k, off);
            float v[VEC];
            apart<VEC>(acc[which][k], v);
            if (blockDim.y == 1 && VEC % 4 == 0 && cols % VEC == 0 && off % VEC == 0) {
                if (c < cols) store<float, VEC>(part + c, v, j.sp_part);
                continue;
            }
            float* to = blockDim.y > 1 ? across + threadIdx.y * cols : part;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (c + i >= 0 && c + i < cols && (blockDim.y > 1 || TROP_IN(part + c + i, 4, j.sp_part))) to[c + i] = v[i];
        }
        if (blockDim.y > 1) {
            __syncthreads();
            for (int c = threadIdx.y * 32 + threadIdx.x; c < cols; c += 32 * blockDim.y) {
                float a = 0.f;
                for (int r = 0; r < (int)blockDim.y; ++r) a += across[r * cols + c];
                if (TROP_IN(part + c, 4, j.sp_part)) part[c] = a;
            }
        }
    }
}

// A thread has eight columns at most, whose four sums it keeps in registers over all of its block's rows: 128 registers, so that
// an SM has one block of 512 threads (4096 columns).  Longer rows are shared by the CTAs of a cluster (WIDE).  What bounds it is a
// row's two rounds of sums, which nothing else on the SM covers, and instructions (83 an element, half of the issue slots):
// 16384x4096 bf16 246 us, 4.4 TB/s, from copies 270 us; 4096x8192 f16 from copies 176 us; f32 335 us, 4.8 TB/s.  (Two blocks of
// 256 threads an SM, as clusters of twice as many: 16384x4096 bf16 292 us, 4096x8192 294 us.)
template <typename S, typename U, typename Y, int VEC, int NV, bool CODED, bool OFF, bool WIDE>
__global__ void __launch_bounds__(512) k_residual_back(const ResJob j, int period, int stages, uint32_t* error)
{
    pdl_wait();
    pdl_signal();
    constexpr bool SHARED = shared_vectors<U, Y, OFF>;
    extern __shared__ __align__(16) uint8_t dyn[];
    constexpr int SUMS = WIDE ? 128 : 32;
    __shared__ __align__(16) float sh[3][2][SUMS];
    __shared__ __align__(8) uint64_t arrived[3];
    __shared__ __align__(8) uint64_t full[8][4];
    zero_sums(&sh[0][0][0], 6 * SUMS);
    const int cols = (int)j.cols;
    const uint32_t rank = WIDE ? cluster_ctarank() : 0, ctas = WIDE ? cluster_ctas() : 1;
    const int block = blockIdx.x / ctas;
    Walk walk = walk_of<Y, VEC, OFF>(j.dy.p, j.dy.s, period, block, gridDim.x / ctas);
    WideSums others = {reinterpret_cast<float2(*)[128]>(&sh[0][0][0]), arrived, rank, ctas, 0};
    if (WIDE) {
        walk.off -= rank * NV * blockDim.x * VEC;
        others.init();
        __syncthreads();
        cluster_sync_all();  // the others' sums are zeros, and their mbarriers ready
    }
    auto sums = [&](float& a, float& b, int which) {
        if constexpr (WIDE) others(a, b, which, error);
        else row_sums(a, b, sh[which]);
    };
    Vectors<Y, VEC, OFF, SHARED> vec;
    vec.template init<NV>(dyn, walk.off, j);
    const float scale = j.s.p ? 1.f : j.scale;
    Pair<VEC> acc[4][NV][pairs<VEC>];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) acc[a][k][i] = p_of<Pair<VEC>>(0.f);
    using P = Pair<VEC>;
    using InY = In<Y, VEC, false, OFF>;
    using InD = In<S, VEC, false, OFF>;
    using InR = In<S, VEC, CODED, OFF>;
    using InU = In<U, VEC, CODED, OFF>;
    const int wide = OFF ? blockDim.x * blockDim.y : blockDim.x;  // threads whose vectors lie together
    const int t0 = OFF ? threadIdx.y * blockDim.x + threadIdx.x : threadIdx.x;
    const int at_r = NV * InY::BYTES * wide, at_u = at_r + NV * InR::BYTES * wide, at_d = at_u + NV * InU::BYTES * wide;
    const int at_g = at_d + (j.dr.p ? NV * InD::BYTES * wide : 0);
    const int size = at_g + (j.gate == GATE_FULL ? NV * InU::BYTES * wide : 0), stage = OFF ? size : size * blockDim.y;
    const uint32_t base = smem_u32(dyn) + (SHARED ? 5 * vec.span : 0) + (OFF ? 0 : threadIdx.y * size);
    Ring ring;
    if (!OFF) ring.init(full, stages);
    auto issue = [&](uint32_t row, int slot) {
        const uint32_t to = base + slot * stage;
        if constexpr (OFF) {
            if (row < (uint32_t)j.rows) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int c = column<VEC>(k, walk.off);
                    InY::issue(to + k * InY::BYTES * wide, t0, wide, j.dy, j.kr, row, c, j);
                    InR::issue(to + at_r + k * InR::BYTES * wide, t0, wide, j.r, j.kr, row, c, j);
                    InU::issue(to + at_u + k * InU::BYTES * wide, t0, wide, j.u, j.ku, row, c, j);
                    if (j.dr.p) InD::issue(to + at_d + k * InD::BYTES * wide, t0, wide, j.dr, j.kr, row, c, j);
                    if (j.gate == GATE_FULL) InU::issue(to + at_g + k * InU::BYTES * wide, t0, wide, j.g, j.kg, row, c, j);
                }
            }
            copies_commit();
        } else if (threadIdx.x == 0 && row < (uint32_t)j.rows && ring.ok) {
            const int c = -walk.off, n = max(0, min(cols - c, (int)(NV * blockDim.x) * VEC));
            const bool g = j.gate == GATE_FULL, d = j.dr.p;
            bool in = row_in<Y>(j.dy, row, c, n) && (!d || row_in<S>(j.dr, row, c, n));
            if constexpr (CODED) {
                in = in && TROP_IN(codes_at(j.kr, row, c), n, j.kr.sp_c) && TROP_IN(codes_at(j.ku, row, c), n, j.ku.sp_c) &&
                     (!g || TROP_IN(codes_at(j.kg, row, c), n, j.kg.sp_c));
            } else {
                in = in && row_in<S>(j.r, row, c, n) && row_in<U>(j.u, row, c, n) && (!g || row_in<U>(j.g, row, c, n));
            }
            uint64_t* const bar = ring.full + slot;
            if (in && n > 0) {
                const uint32_t br = n * (CODED ? 1 : sizeof(S)), bu = n * (CODED ? 1 : sizeof(U)), by = n * sizeof(Y), bd = n * sizeof(S);
                mbar_expect_tx(bar, by + br + (g ? 2 : 1) * bu + (d ? bd : 0));
                bulk_to(to, elem<Y>(j.dy, row, c), by, bar);
                bulk_to(to + at_r, CODED ? (void*)codes_at(j.kr, row, c) : (void*)elem<S>(j.r, row, c), br, bar);
                if (d) bulk_to(to + at_d, elem<S>(j.dr, row, c), bd, bar);
                bulk_to(to + at_u, CODED ? (void*)codes_at(j.ku, row, c) : (void*)elem<U>(j.u, row, c), bu, bar);
                if (g) bulk_to(to + at_g, CODED ? (void*)codes_at(j.kg, row, c) : (void*)elem<U>(j.g, row, c), bu, bar);
            } else {
                mbar_expect_tx(bar, 0);
            }
        }
    };
    // a row's statistics, gate and scales, fetched a row ahead
    constexpr bool SCALED = CODED && !OFF;
    float um, ur, mean, rstd, gate;
    uint32_t sr[NV], su[NV], sg[NV];
    auto scale_of = [&](const Rows8& a, uint32_t row, int c) -> uint32_t {
        const uint8_t* p = scales_at(a, row, c / GROUP8);
        return c < cols && TROP_IN(p, 1, a.sp_s) ? *p : LEAST8;
    };
    auto ahead = [&](uint32_t row) {
        um = ur = mean = rstd = gate = 0.f;
        if (row >= (uint32_t)j.rows) return;
        um = stat(j, 0, row), ur = stat(j, 1, row), mean = stat(j, 2, row), rstd = stat(j, 3, row);
        if (j.gate == GATE_ROW) gate = row_gate<U>(j, row);
        if constexpr (SCALED) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = column<VEC>(k, walk.off);
                sr[k] = scale_of(j.kr, row, c);
                su[k] = scale_of(j.ku, row, c);
                if (j.gate == GATE_FULL) sg[k] = scale_of(j.kg, row, c);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) sr[k] = su[k] = sg[k] = LEAST8;
    for (int i = 0; i < stages; ++i) issue(walk.first + i * walk.step, i);
    int turn = 0, slot = 0;
    uint32_t phase = 0;
    ahead(walk.first);
    for (uint32_t row = walk.first; row < (uint32_t)j.rows; row += walk.step) {
        const uint32_t from = base + slot * stage;
        const float um0 = um, ur0 = ur, mean0 = mean, rstd0 = rstd;
        uint32_t er[NV], eu[NV], eg[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) er[k] = sr[k], eu[k] = su[k], eg[k] = sg[k];
        float ga = 1.f, gs = 1.f;
        if (j.gate == GATE_ROW) gate_both<U>(gate, j.act, ga, gs);
        ahead(row + walk.step);
        if (OFF) copies_wait(stages);
        else ring.wait(slot, phase, error);
        P h[NV][pairs<VEC>], e[NV][pairs<VEC>];
        P sum0 = p_of<P>(0.f), sum1 = sum0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column<VEC>(k, walk.off);
            P w[pairs<VEC>];
            vec.get(0, j.w, k, c, j, 1.f, w);
            InY::take(e[k], from + k * InY::BYTES * wide, t0, wide, j.dy, j.kr, row, c, 0, j);
            InR::take(h[k], from + at_r + k * InR::BYTES * wide, t0, wide, j.r, j.kr, row, c, er[k], j);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) {
                h[k][i] = p_mul(p_add(h[k][i], p_of<P>(-mean0)), p_of<P>(rstd0));
                acc[0][k][i] = p_fma(e[k][i], h[k][i], acc[0][k][i]);
                acc[1][k][i] = p_add(acc[1][k][i], e[k][i]);
                e[k][i] = p_mul(e[k][i], w[i]);
                sum0 = p_add(sum0, e[k][i]);
                sum1 = p_fma(e[k][i], h[k][i], sum1);
            }
        }
        float s0 = p_sum(sum0), s1 = p_sum(sum1);
        sums(s0, s1, turn);
        // (bulk copies: all of the group have read the stage before this one)
        if (!OFF && row != walk.first) {
            if (blockDim.x == 32) __syncwarp();
            issue(row + (stages - 1) * walk.step, slot == 0 ? stages - 1 : slot - 1);
        }
        const P flat = p_of<P>(j.rms ? 0.f : -s0 * j.inv_cols), along = p_of<P>(-s1 * j.inv_cols);
        P sum2 = sum0 = sum1 = p_of<P>(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = column<VEC>(k, walk.off);
            P o[pairs<VEC>], d[pairs<VEC>], f[pairs<VEC>], a[pairs<VEC>];
            if (j.dr.p) {
                InD::take(d, from + at_d + k * InD::BYTES * wide, t0, wide, j.dr, j.kr, row, c, 0, j);
            } else {
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) d[i] = p_of<P>(0.f);
            }
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) {
                d[i] = p_fma(p_of<P>(rstd0), p_fma(h[k][i], along, p_add(e[k][i], flat)), d[i]);
                o[i] = p_mul(p_of<P>(j.alpha), d[i]);
            }
            if (j.dx.p && c < cols) put<S, VEC, OFF>(j.dx, row, c, o, cols);
            InU::take(h[k], from + at_u + k * InU::BYTES * wide, t0, wide, j.u, j.ku, row, c, eu[k], j);  // from here on h is u's
            if (j.post)
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) h[k][i] = p_mul(p_add(h[k][i], p_of<P>(-um0)), p_of<P>(ur0));
            // o: d times the scale and, once v and the gate's slope are in, the gate's gradient; a: the gate
            vec.get(4, j.s, k, c, j, 1.f, f);
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) o[i] = p_mul(p_mul(d[i], f[i]), p_of<P>(scale));
            if (j.gate == GATE_FULL) {
                InU::take(a, from + at_g + k * InU::BYTES * wide, t0, wide, j.g, j.kg, row, c, eg[k], j);
                if (j.act != 0) {
                    float g[VEC], slope[VEC];
                    apart<VEC>(a, g);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) gate_both<U>(g[i], j.act, g[i], slope[i]);
#pragma unroll
                    for (int i = 0; i < pairs<VEC>; ++i) a[i] = pair_at<VEC>(g, i), f[i] = pair_at<VEC>(slope, i);
                }
            } else {
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) a[i] = p_of<P>(ga);
            }
            P slope[pairs<VEC>];
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) {
                slope[i] = f[i];
                const P da = p_mul(d[i], a[i]);
                acc[2][k][i] = p_fma(da, h[k][i], acc[2][k][i]);
                acc[3][k][i] = p_add(acc[3][k][i], da);
                e[k][i] = p_mul(o[i], a[i]);
                d[i] = h[k][i];  // v
            }
            if (j.post) {
                P pb[pairs<VEC>];
                vec.get(2, j.pw, k, c, j, 1.f, f);
                vec.get(3, j.pb, k, c, j, 0.f, pb);
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) {
                    d[i] = p_fma(h[k][i], f[i], pb[i]);
                    e[k][i] = p_mul(e[k][i], f[i]);
                    sum0 = p_add(sum0, e[k][i]);
                    sum1 = p_fma(e[k][i], h[k][i], sum1);
                }
            }
            if (j.gate == GATE_FULL && j.dg.p) {
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) {
                    o[i] = p_mul(o[i], d[i]);
                    if (j.act != 0) o[i] = p_mul(o[i], slope[i]);
                }
                if (c < cols) put<U, VEC, OFF>(j.dg, row, c, o, cols);
            } else if (j.gate == GATE_ROW) {
#pragma unroll
                for (int i = 0; i < pairs<VEC>; ++i) sum2 = p_fma(o[i], d[i], sum2);
            }
        }
        if (OFF) issue(row + stages * walk.step, slot);
        s0 = p_sum(sum0), s1 = p_sum(sum1);
        if (j.post) sums(s0, s1, turn ^ 1);
        else turn ^= 1;  // (the next row's first sums take the other of the two)
        if (j.gate == GATE_ROW) {
            float s2 = p_sum(sum2), none = 0.f;
            sums(s2, none, 2);
            if (j.dg.p && threadIdx.x == 0 && rank == 0) put_row_gate<U>(j, row, s2 * gs);
        }
        if (j.du.p) {
            const P flat2 = p_of<P>(j.rms ? 0.f : -s0 * j.inv_cols), along2 = p_of<P>(-s1 * j.inv_cols);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = column<VEC>(k, walk.off);
                if (j.post)
#pragma unroll
                    for (int i = 0; i < pairs<VEC>; ++i)
                        e[k][i] = p_mul(p_of<P>(ur0), p_fma(h[k][i], along2, p_add(e[k][i], flat2)));
                if (c < cols) put<U, VEC, OFF>(j.du, row, c, e[k], cols);
            }
        }
        if (++slot == stages) slot = 0, phase ^= 1;
    }
    if (!OFF) ring.leave(stages);
    if (j.want && blockDim.y > 1) __syncthreads();  // (the warps' sums go where the ring was)
    if (j.want) put_partials<VEC, NV>(j, acc, reinterpret_cast<float*>(dyn), walk.off, block);
    if (WIDE) cluster_sync_all();  // no CTA leaves before the others have written its sums
}

// Rows longer than that: a block per row, three walks; the row's two sums of the norm of r are left for the columns.
template <typename S, typename U, typename Y, bool CODED>
struct LongRow {
    const ResJob& j;
    int64_t row;
    float um, ur, mean, rstd, ga, gs;
    __device__ LongRow(const ResJob& j_, int64_t row_) : j(j_), row(row_), ga(1.f), gs(1.f)
    {
        um = stat(j, 0, row), ur = stat(j, 1, row), mean = stat(j, 2, row), rstd = stat(j, 3, row);
        if (j.gate == GATE_ROW) gate_both<U>(row_gate<U>(j, row), j.act, ga, gs);
    }
    template <typename T, bool C>
    __device__ float of(const RowsAt& a, const Rows8& k, int64_t c) const
    {
        if (C) {
            const int8_t* p = k.codes + row * k.sc + c;
            const uint8_t* s = k.scales + row * k.ss + c / GROUP8;
            return TROP_IN(p, 1, k.sp_c) && TROP_IN(s, 1, k.sp_s) ? (float)*p * unit8(*s) : 0.f;
        }
        const T* p = (const T*)a.p + row * a.s + c;
        return TROP_IN(p, sizeof(T), a.sp) ? to_f32(*p) : 0.f;
    }
    __device__ float vec(const VecAt& a, int64_t c, float none) const { return one_of<Y>(a, c, j, none); }
    __device__ void first(int64_t c, float& dy, float& h) const
    {
        dy = of<Y, false>(j.dy, j.kr, c);
        h = (of<S, CODED>(j.r, j.kr, c) - mean) * rstd;
    }
    // d; and da, uh and what the gate's gradient is (dg), dv pw
    __device__ float second(int64_t c, float flat, float along, float& da, float& uh, float& dg, float& q) const
    {
        float dy, h, a = ga, slope = 1.f;
        first(c, dy, h);
        const float dr = j.dr.p ? of<S, false>(j.dr, j.kr, c) : 0.f;
        const float d = grad_r(dr, dy * vec(j.w, c, 1.f), h, rstd, flat, along);
        const float u = of<U, CODED>(j.u, j.ku, c), pw = vec(j.pw, c, 1.f);
        uh = j.post ? (u - um) * ur : u;
        if (j.gate == GATE_FULL) gate_both<U>(of<U, CODED>(j.g, j.kg, c), j.act, a, slope);
        const float ds = d * vec(j.s, c, j.scale);
        da = d * a;
        dg = ds * (j.post ? __fmaf_rn(uh, pw, vec(j.pb, c, 0.f)) : u) * slope;
        q = j.post ? ds * a * pw : ds * a;
        return d;
    }
};
template <typename S, typename U, typename Y, bool CODED>
__global__ void __launch_bounds__(1024) k_residual_back_long(const ResJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[2][32][3];
    const LongRow<S, U, Y, CODED> at(j, blockIdx.x);
    float s[3] = {0.f, 0.f, 0.f}, dy, h, da, uh, dg, q;
    for (int64_t c = threadIdx.x; c < j.cols; c += blockDim.x) {
        at.first(c, dy, h);
        const float e = dy * at.vec(j.w, c, 1.f);
        s[0] += e;
        s[1] = __fmaf_rn(e, h, s[1]);
    }
    group_sum_turn<3>(s, sh[0]);
    const float flat = j.rms ? 0.f : s[0] * j.inv_cols, along = s[1] * j.inv_cols;
    if (j.sums && threadIdx.x == 0 && TROP_IN(j.sums + 2 * at.row, 8, j.sp_sums)) j.sums[2 * at.row] = flat, j.sums[2 * at.row + 1] = along;
    s[0] = s[1] = s[2] = 0.f;
    for (int64_t c = threadIdx.x; c < j.cols; c += blockDim.x) {
        at.second(c, flat, along, da, uh, dg, q);
        s[0] += q;
        s[1] = __fmaf_rn(q, uh, s[1]);
        s[2] += dg;
    }
    group_sum_turn<3>(s, sh[1]);
    const float flat2 = j.rms ? 0.f : s[0] * j.inv_cols, along2 = s[1] * j.inv_cols;
    for (int64_t c = threadIdx.x; c < j.cols; c += blockDim.x) {
        const float d = at.second(c, flat, along, da, uh, dg, q);
        if (j.dx.p) put_one<S>(j.dx, at.row, c, j.alpha * d);
        if (j.dg.p && j.gate == GATE_FULL) put_one<U>(j.dg, at.row, c, dg);
        if (j.du.p) put_one<U>(j.du, at.row, c, j.post ? at.ur * (q - flat2 - uh * along2) : q);
    }
    if (j.dg.p && j.gate == GATE_ROW && threadIdx.x == 0) put_row_gate<U>(j, at.row, s[2] * at.gs);
}
// The columns' sums over rows blockIdx.y, + gridDim.y, ...: a thread per column.
template <typename S, typename U, typename Y, bool CODED>
__global__ void __launch_bounds__(256) k_residual_columns(const ResJob j)
{
    pdl_wait();
    pdl_signal();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= j.cols) return;
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, dy, h, da, uh, dg, q;
    for (int64_t row = blockIdx.y; row < j.rows; row += gridDim.y) {
        const LongRow<S, U, Y, CODED> at(j, row);
        at.first(c, dy, h);
        acc[0] = __fmaf_rn(dy, h, acc[0]);
        acc[1] += dy;
        if (!(j.want & (SUM_1 | SUM_2))) continue;
        const bool in = TROP_IN(j.sums + 2 * row, 8, j.sp_sums);
        at.second(c, in ? j.sums[2 * row] : 0.f, in ? j.sums[2 * row + 1] : 0.f, da, uh, dg, q);
        acc[2] = __fmaf_rn(da, uh, acc[2]);
        acc[3] += da;
    }
#pragma unroll
    for (int which = 0; which < 4; ++which) {
        float* part = j.part + ((int64_t)blockIdx.y * 4 + which) * j.cols + c;
        if ((j.want >> which & 1) && TROP_IN(part, 4, j.sp_part)) *part = acc[which];
    }
}

// The blocks' column sums, in block order: 32 columns per block of threads, whose warps take every WARPS'th block's
// sums.  blockIdx.y: dw, db, or what comes of A1 and A2, whose loads are on their way together.  It is bound by the latency of those
// loads: 32 warps where every SM has one block of them at most (608 blocks' sums of 1001 columns 9 us, with 16 warps 15), else 16,
// of which an SM takes three (76 blocks' sums of 8192 columns 7 us, with 32 warps 13).
template <int N, int WARPS>
__device__ __forceinline__ void column_sums(const JoinJob& j, int which, const bool (&wanted)[N], float (*sh)[WARPS][32], float (&a)[N])
{
    constexpr int AHEAD = 8 / N;  // blocks whose loads are on their way
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
#pragma unroll
    for (int n = 0; n < N; ++n) a[n] = 0.f;
    if (c < j.cols)
        for (int b = threadIdx.y; b < j.blocks; b += WARPS * AHEAD) {
            float v[N][AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const float* p = j.part + ((int64_t)(b + WARPS * k) * 4 + which + n) * j.cols + c;
                    v[n][k] = wanted[n] && b + WARPS * k < j.blocks && TROP_IN(p, 4, j.sp_part) ? *p : 0.f;
                }
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int k = 0; k < AHEAD; k += 2) a[n] += v[n][k] + v[n][k + 1];
        }
#pragma unroll
    for (int n = 0; n < N; ++n) sh[n][threadIdx.y][threadIdx.x] = a[n];
    __syncthreads();
    if (threadIdx.y != 0) return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        a[n] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; w += 2) a[n] += sh[n][w][threadIdx.x] + sh[n][w + 1][threadIdx.x];
    }
}
template <typename Y, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 16 ? 3 : 1) k_residual_join(const JoinJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[2][WARPS][32];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const bool mine = threadIdx.y == 0 && c < j.cols;
    auto at = [&](const VecAt& a, float none) {
        if (!a.p) return none;
        if (j.wide_w) return TROP_IN((const float*)a.p + c, 4, a.sp) ? ((const float*)a.p)[c] : 0.f;
        return TROP_IN((const Y*)a.p + c, sizeof(Y), a.sp) ? to_f32(((const Y*)a.p)[c]) : 0.f;
    };
    auto put = [&](void* to, float v, const Span& sp) {
        (void)sp;
        if (!to) return;
        if (j.wide_w) {
            if (TROP_IN((float*)to + c, 4, sp)) ((float*)to)[c] = v;
        } else if (TROP_IN((Y*)to + c, sizeof(Y), sp)) {
            ((Y*)to)[c] = from_f32<Y>(v);
        }
    };
    if (blockIdx.y < 2) {
        void* to = blockIdx.y ? j.db : j.dw;
        if (!to) return;
        float a[1];
        column_sums<1, WARPS>(j, blockIdx.y, {true}, sh, a);
        if (mine) put(to, a[0], blockIdx.y ? j.sp_db : j.sp_dw);
        return;
    }
    const bool first = j.dpw || j.ds, second = j.dpb || (j.ds && j.post && j.pb.p);
    if (!first && !second) return;
    const float s = mine ? at(j.s, j.scale) : 0.f, pw = mine ? at(j.pw, 1.f) : 0.f, pb = mine ? at(j.pb, 0.f) : 0.f;
    float a[2];
    column_sums<2, WARPS>(j, 2, {first, second}, sh, a);
    if (!mine) return;
    put(j.dpw, s * a[0], j.sp_dpw);
    put(j.dpb, s * a[1], j.sp_dpb);
    if (j.ds) put(j.ds, j.post ? __fmaf_rn(pw, a[0], second ? pb * a[1] : 0.f) : a[0], j.sp_ds);
}

// ------------------------------------------------------------------ host
// A row's group: threads and vectors per thread.  Many rows: as many elements per thread as there may be, down to a warp a
// row; few rows: spread over more threads.
bool shape_of(int64_t units, int vec, int most_elems, int most_threads, int64_t rows, int sm, int warps, int* nv, dim3* block)
{
    *nv = 0;
    for (int n = std::max(1, most_elems / vec); n >= 1; n /= 2) {
        const int64_t g = ((units + n - 1) / n + 31) / 32 * 32;
        if (g > most_threads) break;
        *nv = n;
        *block = g == 32 ? dim3(32, (unsigned)warps) : dim3((unsigned)g, 1);
        if (rows * (g / 32) >= (int64_t)sm * 8) return true;
    }
    return *nv > 0;
}

template <typename S, typename U, typename Y>
struct Types {
    static constexpr int VEC = sizeof(U) == 2 ? 8 : 4;  // elements of the narrower rows' 16 bytes
};
// The rows' places in granules of VEC elements: after how many rows they repeat, the same for all the matrices (1: every row
// starts on one); 0 where they differ, or too many rows share none.
struct Places {
    int vec;
    int64_t rows, cols;
    int64_t base = -1, stride = 0;
    bool same = true, bulk = true;  // bulk: whole rows in units of 16 bytes
    void add(RowsAt& a, size_t elem)
    {
        if (!a.p) return;
        const int64_t step = rows > 1 ? a.s : 0, b = (uintptr_t)a.p / elem % vec, s = step % vec;
        if (base < 0) base = b, stride = s;
        else if (b != base || s != stride) same = false;
        if (step < 0 || step * elem >> 32) same = false;
        a.sb = (uint32_t)(step * elem);
        if ((uintptr_t)a.p % 16 || step * elem % 16 || cols * elem % 16) bulk = false;
    }
    void add(Rows8& k)
    {
        if (!k.codes) return;
        const int64_t step = rows > 1 ? k.sc : 0, ss = rows > 1 ? k.ss : 0;
        if (step < 0 || step >> 32 || ss < 0 || ss >> 32) same = false;
        k.sb = (uint32_t)step, k.ssb = (uint32_t)ss;
        if ((uintptr_t)k.codes % 16 || step % 16 || cols % 16) bulk = false;
    }
    int period() const
    {
        if (!same) return 0;
        int p = 1;
        while (p * stride % vec) p *= 2;
        return p;
    }
    bool on() const { return same && base <= 0 && stride == 0 && bulk; }
};

int launch_pack(const RowsAt& a, int dtype, const Rows8& k, int64_t rows, int64_t cols, cudaStream_t s)
{
    return launch_activation_pack(rows, cols, {a.p, a.s, dtype}, {k.codes, k.sc, k.scales, k.ss}, s);
}
template <typename T>
constexpr int dtype_of() { return sizeof(T) == 4 ? (int)TROP_F32 : std::is_same<T, bf16>::value ? (int)TROP_BF16 : (int)TROP_F16; }

// Stages of a ring: up to four rows, in what a block's share of the SM's shared memory leaves.
constexpr size_t SM_SMEM = 227 * 1024;
int stages_of(size_t stage, size_t beside, int per_sm)
{
    const size_t share = SM_SMEM / per_sm - 1024 - 4096;  // (a block's own kilobyte, and the static arrays)
    const size_t n = share > beside ? (share - beside) / stage : 0;
    return (int)std::min<size_t>(4, n);
}

dim3 long_block(int64_t cols) { return dim3((unsigned)std::min<int64_t>(1024, (cols + 31) / 32 * 32)); }

}  // namespace

template <typename S, typename U, typename Y>
int residual_forward(ResJob j, int sm, cudaStream_t s)
{
    constexpr int V = Types<S, U, Y>::VEC;
    const size_t we = j.wide_w ? 4 : sizeof(Y);
    Places at = {V, j.rows, j.cols};
    at.add(j.x, sizeof(S)), at.add(j.r, sizeof(S)), at.add(j.u, sizeof(U)), at.add(j.y, sizeof(Y));
    if (j.gate == GATE_FULL) at.add(j.g, sizeof(U));
    at.add(j.ku), at.add(j.kg), at.add(j.kr);
    bool vec = j.cols % V == 0 && at.on();
    for (const VecAt* a : {&j.w, &j.b, &j.pw, &j.pb, &j.s}) vec = vec && aligned(a->p, 0, we, V, 1);
    const int period = at.period();
    const bool off = !vec && period > 0 && j.cols >= 2 * V;
    const int64_t units = off ? (j.cols + V - 1) / V + 1 : j.cols / V;
    int nv = 0, stages = 0;
    dim3 block;
    size_t smem = 0;
    if ((vec || off) && shape_of(units, V, 16, 1024, j.rows, sm, 8, &nv, &block)) {
        const int threads = block.x * block.y;
        const bool shared = shared_vectors<U, Y, false> && block.y > 1;
        const size_t beside = off || shared ? (size_t)5 * nv * block.x * V * we : 0;
        const size_t stage = (size_t)nv * threads * V * (sizeof(S) + sizeof(U) * (j.gate == GATE_FULL ? 2 : 1));
        // Of bulk copies one stage a block, more blocks: with two the ring takes the L1 cache that keeps the vectors
        // (16384x4096, f32 stream beside bf16: 158 us against 186; all f32: 230 against 285).
        stages = std::min(off ? 2 : 1, stages_of(stage, beside, std::max(1, (off ? 768 : 1024) / threads)));
        if (stages == 0) stages = std::min(1, stages_of(stage, beside, 1));
        smem = beside + stages * stage;
    }
    if (stages == 0) {
        TROP_LAUNCH((k_residual_long<S, U, Y>), dim3((unsigned)j.rows), long_block(j.cols), 0, j);
        return TROP_OK;
    }
    ResJob k = j;
    if (off) k.ku.codes = k.kg.codes = k.kr.codes = nullptr;  // (whose groups lie across these vectors: a pass of their own)
    auto kernel = off ? (nv == 1          ? k_residual<S, U, Y, V, 1, 1024, true>
                         : nv * V < 16    ? k_residual<S, U, Y, V, 2, 1024, true>
                         : block.x <= 512 ? k_residual<S, U, Y, V, 16 / V, 512, true>
                                          : k_residual<S, U, Y, V, 16 / V, 1024, true>)
                      : (nv == 1          ? k_residual<S, U, Y, V, 1, 1024, false>
                         : nv * V < 16    ? k_residual<S, U, Y, V, 2, 1024, false>
                         : block.x <= 512 ? k_residual<S, U, Y, V, 16 / V, 512, false>
                                          : k_residual<S, U, Y, V, 16 / V, 1024, false>);
    if constexpr (shared_vectors<U, Y, false>)
        if (!off && block.y > 1) kernel = nv == 1 ? k_residual<S, U, Y, V, 1, 512, false, true> : k_residual<S, U, Y, V, 16 / V, 512, false, true>;
    if (smem > PLAIN_SMEM) TROP_TRY(allow_dynamic((const void*)kernel));
    int64_t blocks = (j.rows + block.y - 1) / block.y;
    if (blocks > sm) {  // as many as run at once
        int per_sm = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, (int)(block.x * block.y), smem);
        if (e != cudaSuccess) return cuda_error(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor(k_residual)");
        blocks = std::min<int64_t>(blocks, (int64_t)sm * std::max(1, per_sm));
    }
    if (off) blocks = std::max<int64_t>(1, blocks / period) * period;
    uint32_t* error;
    TROP_TRY(device_error_word(&error));
    TROP_LAUNCH(kernel, dim3((unsigned)blocks), block, smem, k, period, stages, error);
    if (off) {
        if (j.ku.codes) TROP_TRY(launch_pack(j.u, dtype_of<U>(), j.ku, j.rows, j.cols, s));
        if (j.kg.codes) TROP_TRY(launch_pack(j.g, dtype_of<U>(), j.kg, j.rows, j.cols, s));
        if (j.kr.codes) TROP_TRY(launch_pack(j.r, dtype_of<S>(), j.kr, j.rows, j.cols, s));
    }
    return TROP_OK;
}

template <typename S, typename U, typename Y, bool CODED>
int residual_backward(ResJob j, JoinJob t, int sm, cudaStream_t s)
{
    constexpr int V = Types<S, U, Y>::VEC;
    const size_t we = j.wide_w ? 4 : sizeof(Y);
    Places at = {V, j.rows, j.cols};
    at.add(j.dy, sizeof(Y)), at.add(j.dr, sizeof(S)), at.add(j.dx, sizeof(S)), at.add(j.du, sizeof(U));
    if (j.gate == GATE_FULL) at.add(j.dg, sizeof(U));
    if (!CODED) {
        at.add(j.r, sizeof(S)), at.add(j.u, sizeof(U));
        if (j.gate == GATE_FULL) at.add(j.g, sizeof(U));
    } else {
        at.add(j.ku), at.add(j.kg), at.add(j.kr);
    }
    bool vec = j.cols % V == 0 && at.on();
    for (const VecAt* a : {&j.w, &j.pw, &j.pb, &j.s}) vec = vec && aligned(a->p, 0, we, V, 1);
    const int period = at.period();
    // eight elements a thread, up to 512 threads; more columns: up to eight CTAs of them
    const bool off = !vec && period > 0 && j.cols >= 2 * V;
    const int64_t units = off ? (j.cols + V - 1) / V + 1 : j.cols / V;
    const int64_t ctas = (units * V + 4095) / 4096;
    int nv = 0;
    dim3 block;
    bool fits = (vec || off) && ctas <= 8;
    if (fits && ctas == 1) shape_of(units, V, 8, 512, j.rows, sm, 4, &nv, &block);
    else if (fits) nv = 8 / V, block = dim3((unsigned)(((units + ctas * nv - 1) / (ctas * nv) + 31) / 32 * 32), 1);
    const size_t vectors = off || shared_vectors<U, Y, false> ? (size_t)5 * nv * block.x * V * we : 0, across = block.y > 1 && j.want ? block.y * (size_t)j.cols * 4 : 0;
    int stages = 0;
    size_t smem = 0;
    const int threads = block.x * block.y;
    int per_sm = fits ? std::max(1, 512 / threads) : 1;
    if (fits) {
        const size_t copy = CODED ? (off ? V + 12 : V) : 0, pr = CODED ? copy : V * sizeof(S), pu = CODED ? copy : V * sizeof(U);
        const size_t stage = (size_t)nv * threads * (V * sizeof(Y) + pr + pu * (j.gate == GATE_FULL ? 2 : 1) + (j.dr.p ? V * sizeof(S) : 0));
        // (bulk copies: two, for the vectors' sake as above; 16384x4096 f32 337 us against 433 of three)
        // Where eight blocks of 64 threads leave no room for two beside 32-bit vectors, a gate and dr, seven do (65536x512, f32 stream
        // beside bf16: 152 us, 1590 us by the long rows' kernels).
        const int least = off ? 1 : 2;  // (a bulk ring is filled a row late)
        stages = std::min(off ? 4 : 2, stages_of(stage, vectors, per_sm));
        while (stages < least && per_sm > 1) stages = std::min(off ? 4 : 2, stages_of(stage, vectors, --per_sm));
        smem = std::max(vectors + stages * stage, across);
        fits = stages >= least;
    }
    int64_t most = std::max<int64_t>(1, (int64_t)sm * per_sm / ctas);
    const auto wide = off ? k_residual_back<S, U, Y, V, 8 / V, CODED, true, true> : k_residual_back<S, U, Y, V, 8 / V, CODED, false, true>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    if (fits && ctas > 1) {
        if (smem > PLAIN_SMEM) TROP_TRY(allow_dynamic((const void*)wide));
        cfg.gridDim = dim3((unsigned)(most * ctas));
        cfg.blockDim = block;
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)ctas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        // As many as run at once: a cluster's CTAs lie in one part of the chip, where some SMs may be left over.  (4096x16384 bf16,
        // 36 clusters of four instead of 38: 341 us against 611, of which the last two clusters ran alone for half.)
        if (j.rows > 1) {
            int clusters = 0;
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters, wide, &cfg);
            if (e != cudaSuccess) return cuda_error(e, "cudaOccupancyMaxActiveClusters(k_residual_back)");
            most = std::min<int64_t>(most, std::max(1, clusters));
        }
    }
    int64_t blocks = fits ? std::min<int64_t>((j.rows + block.y - 1) / block.y, most)
                          : std::min({j.rows, (int64_t)65535, std::max<int64_t>(1, (int64_t)sm * 8 * 256 / j.cols)});  // (a grid's y)
    if (fits && off) blocks = std::max<int64_t>(1, blocks / period) * period;
    if (j.rows == 0) blocks = 0;  // sums over no rows
    const size_t part = j.want && j.rows ? (size_t)blocks * 4 * j.cols * 4 : 0, sums = !fits && (j.want & (SUM_1 | SUM_2)) ? (size_t)j.rows * 8 : 0;
    Workspace ws(s);
    const size_t at_part = ws.add(part), at_sums = ws.add(sums);
    if (ws.bytes) {
        TROP_TRY(ws.take());
        j.part = part ? (float*)(ws.base + at_part) : nullptr;
        j.sums = sums ? (float*)(ws.base + at_sums) : nullptr;
        j.sp_part = span_bytes(j.part, part);
        j.sp_sums = span_bytes(j.sums, sums);
    }
    uint32_t* error = nullptr;
    if (fits) TROP_TRY(device_error_word(&error));
    if (j.rows == 0) {
    } else if (!fits) {
        if (j.dx.p || j.du.p || j.dg.p || j.sums)
            TROP_LAUNCH((k_residual_back_long<S, U, Y, CODED>), dim3((unsigned)j.rows), long_block(j.cols), 0, j);
        if (j.want)
            TROP_LAUNCH((k_residual_columns<S, U, Y, CODED>), dim3((unsigned)((j.cols + 255) / 256), (unsigned)blocks), dim3(256), 0, j);
    } else if (ctas == 1) {
        const auto kernel = off ? (nv == 1 ? k_residual_back<S, U, Y, V, 1, CODED, true, false> : k_residual_back<S, U, Y, V, 8 / V, CODED, true, false>)
                                : (nv == 1 ? k_residual_back<S, U, Y, V, 1, CODED, false, false> : k_residual_back<S, U, Y, V, 8 / V, CODED, false, false>);
        if (smem > PLAIN_SMEM) TROP_TRY(allow_dynamic((const void*)kernel));
        TROP_LAUNCH(kernel, dim3((unsigned)blocks), block, smem, j, period, stages, error);
    } else {
        cfg.gridDim = dim3((unsigned)(blocks * ctas));
        const cudaError_t e = cudaLaunchKernelEx(&cfg, wide, j, period, stages, error);
        if (e != cudaSuccess) return cuda_error(e, "k_residual_back launch");
        count_launches(1);
    }
    if (j.want) {
        t.part = j.part;
        t.blocks = (int)blocks;
        t.sp_part = j.sp_part;
        const dim3 grid((unsigned)((j.cols + 31) / 32), 3);
        if ((int64_t)grid.x * 3 <= sm) TROP_LAUNCH((k_residual_join<Y, 32>), grid, dim3(32, 32), 0, t);
        else TROP_LAUNCH((k_residual_join<Y, 16>), grid, dim3(32, 16), 0, t);
    }
    return TROP_OK;
}

}  // namespace trop
