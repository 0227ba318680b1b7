// residual_norm.cu -- the jobs of the norms around a block (residual_norm.cuh), by their types.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pack8.h"
#include "residual_job.h"

namespace trop {
namespace {

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
        return residual_forward<typename decltype(S)::type, typename decltype(U)::type, typename decltype(Y)::type>(j, dev->sm_count, s);
    });
}

int launch_residual_norm_backward(const Residual& q, const NormMat& dy, const NormMat& dr, const ResidualGrads& g, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    ResJob j = job_of(q);
    // No gradient depends on y's bias, so that its address is not among those that the route asks after: it is left out, or the
    // blocks' copies of the vectors would read it in whole vectors wherever it starts.
    j.b = {};
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
        return j.kr.codes ? residual_backward<TS, TU, TY, true>(j, t, dev->sm_count, s) : residual_backward<TS, TU, TY, false>(j, t, dev->sm_count, s);
    });
}

}  // namespace trop
