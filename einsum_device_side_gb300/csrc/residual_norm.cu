// residual_norm.cu -- the norms after and before a block, fused with its gate, its residual scale and the addition to the
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
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#define TROP_TU 12  // this file's id in a bounds-violation record
#include "block.h"
#include "pack8.h"
#include "rows.h"
#include "tcgen05.h"

namespace trop {
namespace {

using bf16 = __nv_bfloat16;
enum { GATE_NONE = 0, GATE_ROW = 1, GATE_FULL = 2 };
enum { SUM_W = 1, SUM_B = 2, SUM_1 = 4, SUM_2 = 8 };  // column sums that are wanted

struct Rows8 {  // 8-bit copies, null: absent
    int8_t* codes;
    int64_t sc;
    uint8_t* scales;
    int64_t ss;
    Span sp_c, sp_s;
};
struct RowsAt {
    void* p;
    int64_t s;
    Span sp;
};
struct VecAt {
    const void* p;
    Span sp;
};
struct ResJob {
    int64_t rows, cols;
    float inv_cols, eps, alpha, scale;
    int rms, post, act, gate, wide_w;  // wide_w: the vectors are f32
    RowsAt x, u, g, y, r, dy, dr, dx, du, dg;
    VecAt w, b, pw, pb, s;
    Rows8 ku, kg, kr;
    float* stats;  // [4][rows]: mean and rstd of u, of r
    float* part;   // [blocks][4][cols]
    float* sums;   // long rows, backward: [rows][2]
    int want;
    Span sp_stats, sp_part, sp_sums;
};

// A row's statistics from two passes over registers: a first mean, then the sums of the deviations from it and of their
// squares, which correct each other (Chan, Golub and LeVeque, "Algorithms for computing the sample variance", 1983): the
// first mean's error, some last places, is what the deviations' mean says, so that a constant row's mean is its value and
// its norm zero, whatever the deviation is divided by.
__device__ __forceinline__ void finish_stats(float sum, float squares, const ResJob& j, float& mean, float& rstd)
{
    const float off = sum * j.inv_cols, var = fmaxf(__fmaf_rn(-off, sum, squares), 0.f) + (squares - squares);  // (NaN stays)
    mean += off;
    rstd = __fdiv_rn(1.f, __fsqrt_rn(__fmaf_rn(var, j.inv_cols, j.eps)));
}

// The gate's value and slope.  The exponential's and the reciprocal's hardware approximations are good to 2^-22, and the
// values are rounded with the products that follow.
__device__ __forceinline__ float sigmoid(float g)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(g * -1.4426950408889634f)));
    return r;
}
__device__ __forceinline__ float gate_value(float g, int act)
{
    if (act == 0) return g;
    const float s = sigmoid(g);
    return act == 1 ? s : g * s;
}
__device__ __forceinline__ void gate_both(float g, int act, float& value, float& slope)
{
    value = g, slope = 1.f;
    if (act == 0) return;
    const float s = sigmoid(g), t = s * (1.f - s);
    value = act == 1 ? s : g * s;
    slope = act == 1 ? t : __fmaf_rn(g, t, s);
}

// VEC elements of a vector over the columns: f32, or of type T.  `none` where it is absent, zero past the row.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const VecAt& a, int64_t c, const ResJob& j, float none, float (&v)[VEC])
{
    if (!a.p || c >= j.cols) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = c < j.cols ? none : 0.f;
    } else if (j.wide_w) {
        load<float, VEC>((const float*)a.p + c, v, a.sp);
    } else {
        load<T, VEC>((const T*)a.p + c, v, a.sp);
    }
}
// VEC elements of a row, or their 8-bit copy
template <typename T, int VEC, bool CODED>
struct Held {
    Raw<T, VEC> q;
    __device__ __forceinline__ void zero() { q.zero(); }
    __device__ __forceinline__ void read(const RowsAt& a, const Rows8&, int64_t row, int64_t c)
    {
        const T* p = (const T*)a.p + row * a.s + c;
        if (TROP_IN(p, VEC * sizeof(T), a.sp)) q.read(p);
        else q.zero();
    }
    __device__ __forceinline__ void again() { q.again(); }
    __device__ __forceinline__ void get(float (&v)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = q.get(i);
    }
};
template <typename T, int VEC>
struct Held<T, VEC, true> {
    Codes<VEC> k;
    uint32_t e;
    __device__ __forceinline__ void zero() { k.zero(), e = LEAST8; }
    __device__ __forceinline__ void read(const RowsAt&, const Rows8& a, int64_t row, int64_t c)
    {
        const int8_t* p = a.codes + row * a.sc + c;
        const uint8_t* s = a.scales + row * a.ss + c / GROUP8;
        zero();
        if (TROP_IN(p, VEC, a.sp_c) && TROP_IN(s, 1, a.sp_s)) k.read(p), e = *s;
    }
    __device__ __forceinline__ void again() {}
    __device__ __forceinline__ void get(float (&v)[VEC]) const { values8<VEC>(k.w, unit8(e), v); }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_row(const RowsAt& a, int64_t row, int64_t c, const float (&v)[VEC])
{
    store<T, VEC>((T*)a.p + row * a.s + c, v, a.sp);
}
__device__ __forceinline__ float row_gate(const ResJob& j, int64_t row, bool is_f32, bool is_bf16)
{
    (void)row;
    if (is_f32) {
        const float* p = (const float*)j.g.p + row * j.g.s;
        return TROP_IN(p, 4, j.g.sp) ? *p : 0.f;
    }
    const uint16_t* p = (const uint16_t*)j.g.p + row * j.g.s;
    const uint16_t h = TROP_IN(p, 2, j.g.sp) ? *p : (uint16_t)0;
    return is_bf16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}
template <typename U>
__device__ __forceinline__ float row_gate(const ResJob& j, int64_t row)
{
    return row_gate(j, row, sizeof(U) == 4, std::is_same<U, bf16>::value);
}
__device__ __forceinline__ float stat(const ResJob& j, int which, int64_t row)
{
    const float* p = j.stats + which * j.rows + row;
    return TROP_IN(p, 4, j.sp_stats) ? *p : 0.f;
}
__device__ __forceinline__ void put_stat(const ResJob& j, int which, int64_t row, float v)
{
    float* p = j.stats + which * j.rows + row;
    if (j.stats && TROP_IN(p, 4, j.sp_stats)) *p = v;
}

// The codes of a group's lanes (all of the warp take part; `live`: this one's vector is in the row).
template <typename T, int VEC>
__device__ __forceinline__ void keep(const Rows8& a, int64_t row, int64_t c, bool live, const Raw<T, VEC>& q)
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

// ------------------------------------------------------------------ forward
// Mean and rstd of a row in a group's registers.
template <int VEC, int NV>
__device__ __forceinline__ void row_stats(const ResJob& j, const float (&t)[NV][VEC], float (*sh)[32][2], int& turn, float& mean,
                                          float& rstd)
{
    float s[2] = {0.f, 0.f};
    mean = 0.f;
    if (!j.rms) {
        Pair<VEC> a = p_of<Pair<VEC>>(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) a = p_add(a, pair_at<VEC>(t[k], i));
        s[0] = p_sum(a);
        group_sum_turn<2>(s, sh[turn]);
        turn ^= 1;
        mean = s[0] * j.inv_cols;
    }
    Pair<VEC> a = p_of<Pair<VEC>>(0.f), b = a;
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if ((int64_t)(k * blockDim.x + threadIdx.x) * VEC < j.cols)
#pragma unroll
            for (int i = 0; i < pairs<VEC>; ++i) {
                const Pair<VEC> d = p_add(pair_at<VEC>(t[k], i), p_of<Pair<VEC>>(-mean));
                a = p_add(a, d);
                b = p_fma(d, d, b);
            }
    s[0] = j.rms ? 0.f : p_sum(a);
    s[1] = p_sum(b);
    group_sum_turn<2>(s, sh[turn]);
    turn ^= 1;
    finish_stats(s[0], s[1], j, mean, rstd);
}

template <typename S, typename U, typename Y, int VEC, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) k_residual(const ResJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[2][32][2];
    int turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < j.rows; row += step) {
        Raw<U, VEC> qu[NV], qg[NV];
        Raw<S, VEC> qx[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            qu[k].zero(), qg[k].zero(), qx[k].zero();
            if (c >= j.cols) continue;
            const U* u = (const U*)j.u.p + row * j.u.s + c;
            const S* x = (const S*)j.x.p + row * j.x.s + c;
            if (TROP_IN(u, VEC * sizeof(U), j.u.sp)) qu[k].read(u);
            if (TROP_IN(x, VEC * sizeof(S), j.x.sp)) qx[k].read(x);
            if (j.gate == GATE_FULL) {
                const U* g = (const U*)j.g.p + row * j.g.s + c;
                if (TROP_IN(g, VEC * sizeof(U), j.g.sp)) qg[k].read(g);
            }
        }
        const float ga = j.gate == GATE_ROW ? gate_value(row_gate<U>(j, row), j.act) : 1.f;
        if (j.ku.codes)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
                keep<U, VEC>(j.ku, row, c, c < j.cols, qu[k]);
                if (j.gate == GATE_FULL) keep<U, VEC>(j.kg, row, c, c < j.cols, qg[k]);
            }
        float t[NV][VEC];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) t[k][i] = qu[k].get(i);
        float um = 0.f, ur = 1.f, mean, rstd;
        if (j.post) row_stats<VEC, NV>(j, t, sh, turn, um, ur);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            float f[VEC], o[VEC];
            if (j.post) {
                load_vec<Y, VEC>(j.pw, c, j, 1.f, f);
                load_vec<Y, VEC>(j.pb, c, j, 0.f, o);
#pragma unroll
                for (int i = 0; i < VEC; ++i) t[k][i] = __fmaf_rn((t[k][i] - um) * ur, f[i], o[i]);
            }
            load_vec<Y, VEC>(j.s, c, j, j.scale, f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float a = j.gate == GATE_FULL ? gate_value(qg[k].get(i), j.act) : ga;
                t[k][i] = __fmaf_rn(j.alpha, qx[k].get(i), t[k][i] * f[i] * a);
            }
            Raw<S, VEC> q;
            q.set(t[k]);
            S* r = (S*)j.r.p + row * j.r.s + c;
            if (c < j.cols && TROP_IN(r, VEC * sizeof(S), j.r.sp)) q.write(r);
            if (j.kr.codes) keep<S, VEC>(j.kr, row, c, c < j.cols, q);
        }
        row_stats<VEC, NV>(j, t, sh, turn, mean, rstd);
        if (threadIdx.x == 0) put_stat(j, 0, row, um), put_stat(j, 1, row, ur), put_stat(j, 2, row, mean), put_stat(j, 3, row, rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            if (c >= j.cols) continue;
            float f[VEC], o[VEC];
            load_vec<Y, VEC>(j.w, c, j, 1.f, f);
            load_vec<Y, VEC>(j.b, c, j, 0.f, o);
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = __fmaf_rn((t[k][i] - mean) * rstd, f[i], o[i]);
            store_row<Y, VEC>(j.y, row, c, f);
        }
    }
}

// Rows longer than a block's registers: a block per row walks over it once for every sum; r is formed again each time.
template <typename S, typename U, typename Y>
__global__ void __launch_bounds__(1024) k_residual_long(const ResJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[2][32][1];
    const int64_t row = blockIdx.x;
    const float ga = j.gate == GATE_ROW ? gate_value(row_gate<U>(j, row), j.act) : 1.f;
    int turn = 0;
    auto of = [&](const RowsAt& a, int64_t c, auto type) {
        using T = decltype(type);
        const T* p = (const T*)a.p + row * a.s + c;
        return c < j.cols && TROP_IN(p, sizeof(T), a.sp) ? to_f32(*p) : 0.f;
    };
    // sum over the row of f(column)
    auto sum = [&](auto f) {
        float s[1] = {0.f};
        for (int64_t c = threadIdx.x; c < j.cols; c += 1024) s[0] += f(c);
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
        float f[1], o[1], t = u_at(c);
        if (j.post) {
            load_vec<Y, 1>(j.pw, c, j, 1.f, f);
            load_vec<Y, 1>(j.pb, c, j, 0.f, o);
            t = __fmaf_rn((t - um) * ur, f[0], o[0]);
        }
        load_vec<Y, 1>(j.s, c, j, j.scale, f);
        return __fmaf_rn(j.alpha, of(j.x, c, S()), t * f[0] * (j.gate == GATE_FULL ? gate_value(of(j.g, c, U()), j.act) : ga));
    };
    stats(r_at, mean, rstd);
    if (threadIdx.x == 0) put_stat(j, 0, row, um), put_stat(j, 1, row, ur), put_stat(j, 2, row, mean), put_stat(j, 3, row, rstd);
    for (int64_t c0 = 0; c0 < j.cols; c0 += 1024) {
        const int64_t c = c0 + threadIdx.x;
        const bool live = c < j.cols;
        const float t = live ? r_at(c) : 0.f;
        const float one[1] = {t};
        Raw<S, 1> q;
        q.set(one);
        if (live) {
            S* r = (S*)j.r.p + row * j.r.s + c;
            if (TROP_IN(r, sizeof(S), j.r.sp)) q.write(r);
            float f[1], o[1];
            load_vec<Y, 1>(j.w, c, j, 1.f, f);
            load_vec<Y, 1>(j.b, c, j, 0.f, o);
            f[0] = __fmaf_rn((t - mean) * rstd, f[0], o[0]);
            store_row<Y, 1>(j.y, row, c, f);
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
__device__ __forceinline__ void put_partials(const ResJob& j, const float (&acc)[4][NV][VEC], float* across)
{
#pragma unroll
    for (int which = 0; which < 4; ++which) {
        if (!(j.want >> which & 1)) continue;
        float* part = j.part + ((int64_t)blockIdx.x * 4 + which) * j.cols;
        if (blockDim.y > 1) __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            if (c >= j.cols) continue;
            if (blockDim.y > 1) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) across[threadIdx.y * j.cols + c + i] = acc[which][k][i];
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (TROP_IN(part + c + i, 4, j.sp_part)) part[c + i] = acc[which][k][i];
            }
        }
        if (blockDim.y > 1) {
            __syncthreads();
            for (int64_t c = threadIdx.y * 32 + threadIdx.x; c < j.cols; c += 32 * blockDim.y) {
                float a = 0.f;
                for (int r = 0; r < (int)blockDim.y; ++r) a += across[r * j.cols + c];
                if (TROP_IN(part + c, 4, j.sp_part)) part[c] = a;
            }
        }
    }
}

template <typename S, typename U, typename Y, int VEC, int NV, bool CODED>
__global__ void __launch_bounds__(512) k_residual_back(const ResJob j)
{
    pdl_wait();
    pdl_signal();
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float sh[2][32][3];
    float acc[4][NV][VEC];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[a][k][i] = 0.f;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < j.rows; row += step) {
        Held<Y, VEC, false> qy[NV];
        Held<S, VEC, false> qd[NV];
        Held<S, VEC, CODED> qr[NV];
        Held<U, VEC, CODED> qu[NV], qg[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            qy[k].zero(), qd[k].zero(), qr[k].zero(), qu[k].zero(), qg[k].zero();
            if (c >= j.cols) continue;
            qy[k].read(j.dy, j.kr, row, c);
            if (j.dr.p) qd[k].read(j.dr, j.kr, row, c);
            qr[k].read(j.r, j.kr, row, c);
            qu[k].read(j.u, j.ku, row, c);
            if (j.gate == GATE_FULL) qg[k].read(j.g, j.kg, row, c);
        }
        const float um = stat(j, 0, row), ur = stat(j, 1, row), mean = stat(j, 2, row), rstd = stat(j, 3, row);
        float ga = 1.f, gs = 1.f;
        if (j.gate == GATE_ROW) gate_both(row_gate<U>(j, row), j.act, ga, gs);
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            float w[VEC], dy[VEC], r[VEC];
            load_vec<Y, VEC>(j.w, c, j, 1.f, w);
            qy[k].get(dy);
            qr[k].get(r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float h = (r[i] - mean) * rstd, e = dy[i] * w[i];
                acc[0][k][i] = __fmaf_rn(dy[i], h, acc[0][k][i]);
                acc[1][k][i] += dy[i];
                s[0] += e;
                s[1] = __fmaf_rn(e, h, s[1]);
            }
        }
        group_sum_turn<3>(s, sh[0]);
        const float flat = j.rms ? 0.f : s[0] * j.inv_cols, along = s[1] * j.inv_cols;
        s[0] = s[1] = s[2] = 0.f;
        float d[NV][VEC];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
            qy[k].again(), qr[k].again();
            float w[VEC], dy[VEC], r[VEC], dr[VEC], o[VEC], u[VEC], g[VEC], pb[VEC], sc[VEC];
            load_vec<Y, VEC>(j.w, c, j, 1.f, w);
            qy[k].get(dy);
            qr[k].get(r);
            qd[k].get(dr);
            qu[k].get(u);
            qg[k].get(g);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                d[k][i] = grad_r(dr[i], dy[i] * w[i], (r[i] - mean) * rstd, rstd, flat, along);
                o[i] = j.alpha * d[k][i];
            }
            if (j.dx.p && c < j.cols) store_row<S, VEC>(j.dx, row, c, o);
            load_vec<Y, VEC>(j.pw, c, j, 1.f, w);
            load_vec<Y, VEC>(j.pb, c, j, 0.f, pb);
            load_vec<Y, VEC>(j.s, c, j, j.scale, sc);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float uh = j.post ? (u[i] - um) * ur : u[i], v = j.post ? __fmaf_rn(uh, w[i], pb[i]) : u[i];
                float a = ga, slope = 1.f;
                if (j.gate == GATE_FULL) gate_both(g[i], j.act, a, slope);
                const float da = d[k][i] * a, ds = d[k][i] * sc[i];
                acc[2][k][i] = __fmaf_rn(da, uh, acc[2][k][i]);
                acc[3][k][i] += da;
                o[i] = ds * v * slope;
                const float dv = ds * a;
                d[k][i] = j.post ? dv * w[i] : dv;
                s[0] += d[k][i];
                s[1] = __fmaf_rn(d[k][i], uh, s[1]);
                s[2] += o[i];
            }
            if (j.dg.p && j.gate == GATE_FULL && c < j.cols) store_row<U, VEC>(j.dg, row, c, o);
        }
        if (j.post || j.gate == GATE_ROW) group_sum_turn<3>(s, sh[1]);
        else if (blockDim.x > 32) __syncthreads();  // sh[0] is written again
        const float flat2 = j.rms ? 0.f : s[0] * j.inv_cols, along2 = s[1] * j.inv_cols;
        if (j.du.p)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int64_t c = (int64_t)(k * blockDim.x + threadIdx.x) * VEC;
                if (c >= j.cols) continue;
                qu[k].again();
                float u[VEC];
                qu[k].get(u);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (j.post) d[k][i] = ur * (d[k][i] - flat2 - (u[i] - um) * ur * along2);
                store_row<U, VEC>(j.du, row, c, d[k]);
            }
        if (j.dg.p && j.gate == GATE_ROW && threadIdx.x == 0) {
            const float o[1] = {s[2] * gs};
            store_row<U, 1>(j.dg, row, 0, o);
        }
    }
    if (j.want) put_partials<VEC, NV>(j, acc, reinterpret_cast<float*>(dyn));
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
        if (j.gate == GATE_ROW) gate_both(row_gate<U>(j, row), j.act, ga, gs);
    }
    template <typename T, bool C>
    __device__ float of(const RowsAt& a, const Rows8& k, int64_t c) const
    {
        Held<T, 1, C> q;
        float v[1];
        q.read(a, k, row, c);
        q.get(v);
        return v[0];
    }
    __device__ float vec(const VecAt& a, int64_t c, float none) const
    {
        float v[1];
        load_vec<Y, 1>(a, c, j, none, v);
        return v[0];
    }
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
        if (j.gate == GATE_FULL) gate_both(of<U, CODED>(j.g, j.kg, c), j.act, a, slope);
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
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        at.first(c, dy, h);
        const float e = dy * at.vec(j.w, c, 1.f);
        s[0] += e;
        s[1] = __fmaf_rn(e, h, s[1]);
    }
    group_sum_turn<3>(s, sh[0]);
    const float flat = j.rms ? 0.f : s[0] * j.inv_cols, along = s[1] * j.inv_cols;
    if (j.sums && threadIdx.x == 0 && TROP_IN(j.sums + 2 * at.row, 8, j.sp_sums)) j.sums[2 * at.row] = flat, j.sums[2 * at.row + 1] = along;
    s[0] = s[1] = s[2] = 0.f;
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        at.second(c, flat, along, da, uh, dg, q);
        s[0] += q;
        s[1] = __fmaf_rn(q, uh, s[1]);
        s[2] += dg;
    }
    group_sum_turn<3>(s, sh[1]);
    const float flat2 = j.rms ? 0.f : s[0] * j.inv_cols, along2 = s[1] * j.inv_cols;
    for (int64_t c = threadIdx.x; c < j.cols; c += 1024) {
        float o[1] = {j.alpha * at.second(c, flat, along, da, uh, dg, q)};
        if (j.dx.p) store_row<S, 1>(j.dx, at.row, c, o);
        o[0] = dg;
        if (j.dg.p && j.gate == GATE_FULL) store_row<U, 1>(j.dg, at.row, c, o);
        o[0] = j.post ? at.ur * (q - flat2 - uh * along2) : q;
        if (j.du.p) store_row<U, 1>(j.du, at.row, c, o);
    }
    if (j.dg.p && j.gate == GATE_ROW && threadIdx.x == 0) {
        const float o[1] = {s[2] * at.gs};
        store_row<U, 1>(j.dg, at.row, 0, o);
    }
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

// The blocks' column sums, in block order: 32 columns per block of threads, 32 warps taking every 32nd block's sums.
// blockIdx.y: dw, db, or what comes of A1 and A2.
struct JoinJob {
    const float* part;
    int blocks;
    int64_t cols;
    void *dw, *db, *dpw, *dpb, *ds;
    VecAt pw, pb, s;
    float scale;
    int post, wide_w;
    Span sp_part, sp_dw, sp_db, sp_dpw, sp_dpb, sp_ds;
};
__device__ __forceinline__ float column_sum(const JoinJob& j, int which, float (*sh)[33])
{
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (c < j.cols) {
        float v[4];
        int b = threadIdx.y;
        for (; b + 96 < j.blocks; b += 128) {  // four loads on their way
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float* p = j.part + ((int64_t)(b + 32 * k) * 4 + which) * j.cols + c;
                v[k] = TROP_IN(p, 4, j.sp_part) ? *p : 0.f;
            }
            a += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; b < j.blocks; b += 32) {
            const float* p = j.part + ((int64_t)b * 4 + which) * j.cols + c;
            if (TROP_IN(p, 4, j.sp_part)) a += *p;
        }
    }
    __syncthreads();
    sh[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    a = sh[threadIdx.x][threadIdx.y];  // warp y sums column y's 32 values
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
}
template <typename Y>
__global__ void __launch_bounds__(1024) k_residual_join(const JoinJob j)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.y;
    const bool mine = threadIdx.x == 0 && c < j.cols;
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
        const float a = column_sum(j, blockIdx.y, sh);
        if (mine) put(to, a, blockIdx.y ? j.sp_db : j.sp_dw);
        return;
    }
    const bool first = j.dpw || j.ds, second = j.dpb || (j.ds && j.post && j.pb.p);
    const float a1 = first ? column_sum(j, 2, sh) : 0.f, a2 = second ? column_sum(j, 3, sh) : 0.f;
    if (!mine) return;
    const float s = at(j.s, j.scale);
    put(j.dpw, s * a1, j.sp_dpw);
    put(j.dpb, s * a2, j.sp_dpb);
    if (j.ds) put(j.ds, j.post ? __fmaf_rn(at(j.pw, 1.f), a1, second ? at(j.pb, 0.f) * a2 : 0.f) : a1, j.sp_ds);
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
    static constexpr int SMALL = std::min({sizeof(S), sizeof(U), sizeof(Y)}) == 2 && sizeof(U) == 2 ? 2 : 4;
    static constexpr int VEC = 16 / SMALL;
};
bool on16(const RowsAt& a, size_t elem, int vec, int64_t rows) { return aligned(a.p, a.s, elem, vec, rows); }
bool on8(const Rows8& k, int vec, int64_t rows) { return aligned(k.codes, k.sc, 1, vec, rows); }

template <typename S, typename U, typename Y>
int forward(const ResJob& j, int sm, cudaStream_t s)
{
    constexpr int V = Types<S, U, Y>::VEC;
    const size_t we = j.wide_w ? 4 : sizeof(Y);
    bool vec = j.cols % V == 0 && on16(j.x, sizeof(S), V, j.rows) && on16(j.r, sizeof(S), V, j.rows) && on16(j.u, sizeof(U), V, j.rows) &&
               on16(j.y, sizeof(Y), V, j.rows) && (j.gate != GATE_FULL || on16(j.g, sizeof(U), V, j.rows)) &&
               on8(j.ku, V, j.rows) && on8(j.kg, V, j.rows) && on8(j.kr, V, j.rows);
    for (const VecAt* a : {&j.w, &j.b, &j.pw, &j.pb, &j.s}) vec = vec && aligned(a->p, 0, we, V, 1);
    int nv = 0;
    dim3 block;
    if (!shape_of(vec ? j.cols / V : j.cols, vec ? V : 1, 16, 1024, j.rows, sm, 8, &nv, &block)) {
        TROP_LAUNCH((k_residual_long<S, U, Y>), dim3((unsigned)j.rows), dim3(1024), 0, j);
        return TROP_OK;
    }
    const dim3 grid((unsigned)((j.rows + block.y - 1) / block.y));
    if (vec) {
        const auto kernel = nv == 1             ? k_residual<S, U, Y, V, 1, 1024>
                            : nv * V < 16       ? k_residual<S, U, Y, V, 2, 1024>
                            : block.x <= 512    ? k_residual<S, U, Y, V, 16 / V, 512>
                                                : k_residual<S, U, Y, V, 16 / V, 1024>;
        TROP_LAUNCH(kernel, grid, block, 0, j);
    } else {
        const auto kernel = nv <= 2          ? k_residual<S, U, Y, 1, 2, 1024>
                            : nv <= 4        ? k_residual<S, U, Y, 1, 4, 1024>
                            : block.x <= 512 ? k_residual<S, U, Y, 1, 16, 512>
                                             : k_residual<S, U, Y, 1, 16, 1024>;
        TROP_LAUNCH(kernel, grid, block, 0, j);
    }
    return TROP_OK;
}

template <typename S, typename U, typename Y, bool CODED>
int backward(ResJob j, JoinJob t, int sm, cudaStream_t s)
{
    constexpr int V = Types<S, U, Y>::VEC;
    const size_t we = j.wide_w ? 4 : sizeof(Y);
    bool vec = j.cols % V == 0 && on16(j.dy, sizeof(Y), V, j.rows) && on16(j.dr, sizeof(S), V, j.rows) && on16(j.dx, sizeof(S), V, j.rows) &&
               on16(j.du, sizeof(U), V, j.rows) && (j.gate != GATE_FULL || on16(j.dg, sizeof(U), V, j.rows));
    if (CODED) vec = vec && on8(j.ku, V, j.rows) && on8(j.kg, V, j.rows) && on8(j.kr, V, j.rows);
    else vec = vec && on16(j.r, sizeof(S), V, j.rows) && on16(j.u, sizeof(U), V, j.rows) && (j.gate != GATE_FULL || on16(j.g, sizeof(U), V, j.rows));
    for (const VecAt* a : {&j.w, &j.pw, &j.pb, &j.s}) vec = vec && aligned(a->p, 0, we, V, 1);
    int nv = 0;
    dim3 block;
    const bool fits = shape_of(vec ? j.cols / V : j.cols, vec ? V : 1, j.cols <= 4096 ? 8 : 16, 512, j.rows, sm, 4, &nv, &block);
    int64_t blocks = fits ? std::min<int64_t>((j.rows + block.y - 1) / block.y, (int64_t)sm * std::max<int>(1, 512 / (int)(block.x * block.y)))
                          : std::min<int64_t>(j.rows, std::max<int64_t>(1, (int64_t)sm * 8 * 256 / j.cols));
    const size_t part = j.want && j.rows ? (size_t)blocks * 4 * j.cols * 4 : 0, sums = !fits && (j.want & (SUM_1 | SUM_2)) ? (size_t)j.rows * 8 : 0;
    if (j.rows == 0) blocks = 0;  // sums over no rows
    Workspace ws(s);
    const size_t at_part = ws.add(part), at_sums = ws.add(sums);
    if (ws.bytes) {
        TROP_TRY(ws.take());
        j.part = part ? (float*)(ws.base + at_part) : nullptr;
        j.sums = sums ? (float*)(ws.base + at_sums) : nullptr;
        j.sp_part = span_bytes(j.part, part);
        j.sp_sums = span_bytes(j.sums, sums);
    }
    if (j.rows == 0) {
    } else if (!fits) {
        if (j.dx.p || j.du.p || j.dg.p || j.sums)
            TROP_LAUNCH((k_residual_back_long<S, U, Y, CODED>), dim3((unsigned)j.rows), dim3(1024), 0, j);
        if (j.want)
            TROP_LAUNCH((k_residual_columns<S, U, Y, CODED>), dim3((unsigned)((j.cols + 255) / 256), (unsigned)blocks), dim3(256), 0, j);
    } else {
        const dim3 grid((unsigned)blocks);
        const size_t smem = block.y > 1 && j.want ? block.y * (size_t)j.cols * 4 : 0;  // (a warp's row: 16 KB at most)
        if (vec) {
            const auto kernel = nv == 1   ? k_residual_back<S, U, Y, V, 1, CODED>
                                : nv == 2 ? k_residual_back<S, U, Y, V, 2, CODED>
                                          : k_residual_back<S, U, Y, V, 16 / V, CODED>;
            TROP_LAUNCH(kernel, grid, block, smem, j);
        } else {
            const auto kernel = nv <= 2   ? k_residual_back<S, U, Y, 1, 2, CODED>
                                : nv <= 8 ? k_residual_back<S, U, Y, 1, 8, CODED>
                                          : k_residual_back<S, U, Y, 1, 16, CODED>;
            TROP_LAUNCH(kernel, grid, block, smem, j);
        }
    }
    if (j.want) {
        t.part = j.part;
        t.blocks = (int)blocks;
        t.sp_part = j.sp_part;
        TROP_LAUNCH((k_residual_join<Y>), dim3((unsigned)((j.cols + 31) / 32), 3), dim3(32, 32), 0, t);
    }
    return TROP_OK;
}

RowsAt rows_at(const NormMat& m, int64_t rows, int64_t cols)
{
    const int64_t size[2] = {rows, cols}, stride[2] = {m.sr, 1};
    return {m.p, m.sr, m.p ? span_of(m.p, model_bytes(m.dtype), 2, size, stride) : Span{}};
}
VecAt vec_at(const void* p, int64_t cols, int dtype) { return {p, span_bytes(p, cols * model_bytes(dtype))}; }
Rows8 rows8(const Kept8& k, int64_t rows, int64_t cols)
{
    const int64_t groups = (cols + GROUP8 - 1) / GROUP8;
    const int64_t size[2] = {rows, cols}, stride[2] = {k.sc, 1}, gsize[2] = {rows, groups}, gstride[2] = {k.ss, 1};
    Rows8 r = {k.codes, k.sc, k.scales, k.ss, Span{}, Span{}};
    if (k.codes) r.sp_c = span_of(k.codes, 1, 2, size, stride), r.sp_s = span_of(k.scales, 1, 2, gsize, gstride);
    return r;
}

ResJob job_of(const Residual& q)
{
    ResJob j = {};
    j.rows = q.rows;
    j.cols = q.cols;
    j.inv_cols = (float)(1.0 / (double)q.cols);
    j.eps = (float)q.eps;
    j.alpha = (float)q.alpha;
    j.scale = (float)q.scale;
    j.rms = q.rms;
    j.post = q.post;
    j.act = q.act;
    j.gate = !q.has_gate ? GATE_NONE : q.gate_cols == q.cols && (!q.kr.codes || q.kg.codes) ? GATE_FULL : GATE_ROW;
    j.wide_w = q.wdtype == TROP_F32;
    j.u = rows_at(q.u, q.rows, q.cols);
    j.r = rows_at(q.r, q.rows, q.cols);
    j.g = rows_at(q.gate, q.rows, q.gate_cols);
    j.w = vec_at(q.weight, q.cols, q.wdtype);
    j.b = vec_at(q.bias, q.cols, q.wdtype);
    j.pw = vec_at(q.post_weight, q.cols, q.wdtype);
    j.pb = vec_at(q.post_bias, q.cols, q.wdtype);
    j.s = vec_at(q.scale_vector, q.cols, q.wdtype);
    j.ku = rows8(q.ku, q.rows, q.cols);
    j.kg = rows8(q.kg, q.rows, q.cols);
    j.kr = rows8(q.kr, q.rows, q.cols);
    j.stats = q.stats;
    j.sp_stats = span_bytes(q.stats, (size_t)q.rows * 16);
    return j;
}

// f(S, U, Y) of the types that go together (block.cpp has checked that they are one of these)
template <typename T>
struct Tag {
    using type = T;
};
template <typename F>
int by_types(int s, int u, int y, F f)
{
    const Tag<float> f32;
    const Tag<bf16> b;
    const Tag<__half> h;
    if (s == TROP_F32) {
        if (u == TROP_F32) return y == TROP_F32 ? f(f32, f32, f32) : y == TROP_BF16 ? f(f32, f32, b) : f(f32, f32, h);
        return u == TROP_BF16 ? f(f32, b, b) : f(f32, h, h);
    }
    return s == TROP_BF16 ? f(b, b, b) : f(h, h, h);
}

}  // namespace

int launch_residual_norm(const Residual& q, const NormMat& x, const NormMat& y, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    ResJob j = job_of(q);
    j.x = rows_at(x, q.rows, q.cols);
    j.y = rows_at(y, q.rows, q.cols);
    return by_types(x.dtype, q.u.dtype, y.dtype, [&](auto S, auto U, auto Y) {
        return forward<typename decltype(S)::type, typename decltype(U)::type, typename decltype(Y)::type>(j, dev->sm_count, s);
    });
}

int launch_residual_norm_backward(const Residual& q, const NormMat& dy, const NormMat& dr, const ResidualGrads& g, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    ResJob j = job_of(q);
    j.dy = rows_at(dy, q.rows, q.cols);
    j.dr = rows_at(dr, q.rows, q.cols);
    j.dx = rows_at(g.dx, q.rows, q.cols);
    j.du = rows_at(g.du, q.rows, q.cols);
    j.dg = rows_at(g.dgate, q.rows, q.gate_cols);
    JoinJob t = {};
    t.cols = q.cols;
    t.dw = g.dweight, t.db = g.dbias, t.dpw = g.dpost_weight, t.dpb = g.dpost_bias, t.ds = g.dscale;
    t.pw = j.pw, t.pb = j.pb, t.s = j.s;
    t.scale = j.scale;
    t.post = j.post;
    t.wide_w = j.wide_w;
    const size_t bytes = q.cols * model_bytes(q.wdtype);
    t.sp_dw = span_bytes(t.dw, bytes), t.sp_db = span_bytes(t.db, bytes), t.sp_dpw = span_bytes(t.dpw, bytes);
    t.sp_dpb = span_bytes(t.dpb, bytes), t.sp_ds = span_bytes(t.ds, bytes);
    j.want = (t.dw ? SUM_W : 0) | (t.db ? SUM_B : 0) | (t.dpw || t.ds ? SUM_1 : 0) |
             (t.dpb || (t.ds && j.post && j.pb.p) ? SUM_2 : 0);
    return by_types(q.r.dtype, q.u.dtype, dy.dtype, [&](auto S, auto U, auto Y) {
        using TS = typename decltype(S)::type;
        using TU = typename decltype(U)::type;
        using TY = typename decltype(Y)::type;
        return j.kr.codes ? backward<TS, TU, TY, true>(j, t, dev->sm_count, s) : backward<TS, TU, TY, false>(j, t, dev->sm_count, s);
    });
}

}  // namespace trop
