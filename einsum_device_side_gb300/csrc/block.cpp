// block.cpp -- entry points of a residual block's operators: argument checks, then activation.cu, residual_norm.cu and
// weight_grad.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "block.h"
#include "checks.h"
#include "internal.h"
#include "pack8.h"

using namespace trop;

namespace {

// rows of floating elements: type, layout, extents, and that elements do not straddle addresses of theirs
int float_rows(const trop_tensor* t, const char* name, bool written)
{
    if (!is_model_float(t->dtype)) return set_error(TROP_ERR_DTYPE, "%s has dtype %d: f32, bf16 or f16 is wanted", name, t->dtype);
    TROP_TRY(row_layout(t, name, written));
    if ((uintptr_t)t->data % model_bytes(t->dtype))
        return set_error(TROP_ERR_INVALID_ARG, "%s does not start on an element of its type", name);
    return TROP_OK;
}

// codes and scales of a matrix of rows x cols
int kept8(const trop_tensor* codes, const trop_tensor* scales, const char* name, int64_t rows, int64_t cols, bool written, Kept8* k)
{
    TROP_TRY(same_shape(codes, name, rows, cols));
    if (!scales) return set_error(TROP_ERR_INVALID_ARG, "%s has no scales", name);
    TROP_TRY(same_shape(scales, "scales", rows, (cols + GROUP8 - 1) / GROUP8));
    if (codes->dtype != TROP_I8 || scales->dtype != TROP_U8)
        return set_error(TROP_ERR_DTYPE, "%s has dtype %d, its scales %d: i8 and u8 are wanted", name, codes->dtype, scales->dtype);
    TROP_TRY(row_layout(codes, name, written));
    TROP_TRY(row_layout(scales, "scales", written));
    *k = {(int8_t*)codes->data, codes->stride[0], (uint8_t*)scales->data, scales->stride[0]};
    return TROP_OK;
}

// a vector of elements of that many bytes, or none
int element_start(const void* p, const char* name, size_t bytes)
{
    if ((uintptr_t)p % bytes) return set_error(TROP_ERR_INVALID_ARG, "%s does not start on an element of its type", name);
    return TROP_OK;
}

int extents(int64_t rows, int64_t cols)
{
    if (rows > MOST || cols > MOST) return set_error(TROP_ERR_UNSUPPORTED, "extents above %lld", (long long)MOST);
    return TROP_OK;
}

int activation(const trop_tensor* x, const trop_tensor* codes, const trop_tensor* scales, bool pack, void* stream)
{
    clear_error();
    int64_t rows, cols;
    Kept8 k;
    TROP_TRY(matrix(x, "x", &rows, &cols));
    TROP_TRY(float_rows(x, "x", !pack));
    TROP_TRY(extents(rows, cols));
    TROP_TRY(kept8(codes, scales, "codes", rows, cols, pack, &k));
    TROP_TRY(ensure_device(nullptr));
    if (rows == 0 || cols == 0) return TROP_OK;
    PointerCheck check;
    TROP_TRY(check(x->data, "x"));
    TROP_TRY(check(codes->data, "codes"));
    TROP_TRY(check(scales->data, "scales"));
    const NormMat m = {x->data, x->stride[0], x->dtype};
    return pack ? launch_activation_pack(rows, cols, m, k, (cudaStream_t)stream)
                : launch_activation_values(rows, cols, k, m, (cudaStream_t)stream);
}

}  // namespace

extern "C" int tropical_activation_pack(const trop_tensor* x, const trop_tensor* codes, const trop_tensor* scales, void* stream)
{
    return activation(x, codes, scales, true, stream);
}

extern "C" int tropical_activation_values(const trop_tensor* codes, const trop_tensor* scales, const trop_tensor* x, void* stream)
{
    return activation(x, codes, scales, false, stream);
}

namespace {

bool narrow(int dtype) { return dtype == TROP_BF16 || dtype == TROP_F16; }

// the types that go together: x and r; u and gate; y
int residual_types(int x, int u, int y)
{
    if (!is_model_float(x) || !is_model_float(u) || !is_model_float(y))
        return set_error(TROP_ERR_DTYPE, "x has dtype %d, u %d, y %d: f32, bf16 or f16 is wanted", x, u, y);
    if (u != x && !(x == TROP_F32 && narrow(u)))
        return set_error(TROP_ERR_DTYPE, "u has dtype %d beside x's %d: x's own, or bf16 or f16 beside f32", u, x);
    if (y != u && !(u == TROP_F32 && narrow(y)))
        return set_error(TROP_ERR_DTYPE, "y has dtype %d beside u's %d: u's own, or bf16 or f16 beside f32", y, u);
    return TROP_OK;
}

int residual_options(const trop_residual_options* o, int ydtype, Residual* q)
{
    if (!o) return set_error(TROP_ERR_INVALID_ARG, "options is NULL");
    if ((o->norm != 0 && o->norm != 1) || o->gate_act < 0 || o->gate_act > 2)
        return set_error(TROP_ERR_INVALID_ARG, "norm %d, gate function %d", o->norm, o->gate_act);
    if (!(o->eps >= 0) || !std::isfinite(o->eps) || !std::isfinite(o->alpha) || !std::isfinite(o->scale))
        return set_error(TROP_ERR_INVALID_ARG, "eps %g, alpha %g, scale %g", o->eps, o->alpha, o->scale);
    const bool vectors = o->weight || o->bias || o->post_weight || o->post_bias || o->scale_vector;
    if (vectors && o->wdtype != ydtype && o->wdtype != TROP_F32)
        return set_error(TROP_ERR_DTYPE, "the vectors have dtype %d: y's (%d) or f32 is wanted", o->wdtype, ydtype);
    if (!o->post_norm && (o->post_weight || o->post_bias))
        return set_error(TROP_ERR_INVALID_ARG, "a weight or bias of a norm that is left out");
    q->rms = o->norm;
    q->post = o->post_norm != 0;
    q->act = o->gate_act;
    q->eps = o->eps;
    q->alpha = o->alpha;
    q->scale = o->scale;
    q->wdtype = o->wdtype == TROP_F32 ? TROP_F32 : ydtype;
    q->weight = o->weight;
    q->bias = o->bias;
    q->post_weight = o->post_weight;
    q->post_bias = o->post_bias;
    q->scale_vector = o->scale_vector;
    return TROP_OK;
}

int residual_vectors(PointerCheck& check, const Residual& q)
{
    const struct {
        const void* p;
        const char* name;
    } all[] = {{q.weight, "weight"}, {q.bias, "bias"}, {q.post_weight, "post_weight"}, {q.post_bias, "post_bias"}, {q.scale_vector, "scale"}};
    for (const auto& a : all) {
        if (!a.p) continue;
        TROP_TRY(element_start(a.p, a.name, model_bytes(q.wdtype)));
        TROP_TRY(check(a.p, a.name));
    }
    return TROP_OK;
}

NormMat mat(const trop_tensor* t) { return t ? NormMat{t->data, t->stride[0], t->dtype} : NormMat{nullptr, 0, TROP_F32}; }

// A gate [rows, cols] or [rows, 1] of u's type, or none.
int residual_gate(const trop_tensor* gate, const char* name, int64_t rows, int64_t cols, int dtype, bool written, int64_t* gate_cols)
{
    int64_t r;
    TROP_TRY(matrix(gate, name, &r, gate_cols));
    if (r != rows || (*gate_cols != cols && *gate_cols != 1))
        return set_error(TROP_ERR_SHAPE, "%s is %lld x %lld: %lld x %lld or x 1 is wanted", name, (long long)r, (long long)*gate_cols,
                         (long long)rows, (long long)cols);
    TROP_TRY(float_rows(gate, name, written));
    if (gate->dtype != dtype) return set_error(TROP_ERR_DTYPE, "%s has dtype %d, u %d", name, gate->dtype, dtype);
    return TROP_OK;
}

int check_kept(PointerCheck& check, const Kept8& k, const char* name)
{
    if (!k.codes && !k.scales) return TROP_OK;
    TROP_TRY(check(k.codes, name));
    return check(k.scales, name);
}

}  // namespace

extern "C" int tropical_residual_norm(const trop_residual_options* options, const trop_tensor* x, const trop_tensor* u,
                                      const trop_tensor* gate, const trop_tensor* y, const trop_tensor* r, float* stats,
                                      const trop_kept* kept, void* stream)
{
    clear_error();
    Residual q = {};
    TROP_TRY(matrix(x, "x", &q.rows, &q.cols));
    TROP_TRY(same_shape(u, "u", q.rows, q.cols));
    TROP_TRY(same_shape(y, "y", q.rows, q.cols));
    TROP_TRY(same_shape(r, "r", q.rows, q.cols));
    TROP_TRY(residual_types(x->dtype, u->dtype, y->dtype));
    if (r->dtype != x->dtype) return set_error(TROP_ERR_DTYPE, "r has dtype %d, x %d", r->dtype, x->dtype);
    TROP_TRY(residual_options(options, y->dtype, &q));
    if (q.cols == 0) return set_error(TROP_ERR_SHAPE, "a norm over no elements");
    TROP_TRY(extents(q.rows, q.cols));
    TROP_TRY(float_rows(x, "x", false));
    TROP_TRY(float_rows(u, "u", false));
    TROP_TRY(float_rows(y, "y", true));
    TROP_TRY(float_rows(r, "r", true));
    TROP_TRY(element_start(stats, "stats", 4));
    q.has_gate = gate != nullptr;
    q.gate_cols = 1;
    if (gate) TROP_TRY(residual_gate(gate, "gate", q.rows, q.cols, u->dtype, false, &q.gate_cols));
    q.u = mat(u);
    q.gate = mat(gate);
    q.r = mat(r);
    q.stats = stats;
    if (kept) {
        TROP_TRY(kept8(kept[0].codes, kept[0].scales, "u's copy", q.rows, q.cols, true, &q.ku));
        TROP_TRY(kept8(kept[2].codes, kept[2].scales, "r's copy", q.rows, q.cols, true, &q.kr));
        const bool full = gate && q.gate_cols == q.cols;
        if (!full && (kept[1].codes || kept[1].scales)) return set_error(TROP_ERR_INVALID_ARG, "a copy of a gate that is not [rows, cols]");
        if (full) TROP_TRY(kept8(kept[1].codes, kept[1].scales, "gate's copy", q.rows, q.cols, true, &q.kg));
    }
    TROP_TRY(ensure_device(nullptr));
    if (q.rows == 0) return TROP_OK;
    PointerCheck check;
    TROP_TRY(check(x->data, "x"));
    TROP_TRY(check(u->data, "u"));
    if (gate) TROP_TRY(check(gate->data, "gate"));
    TROP_TRY(check(y->data, "y"));
    TROP_TRY(check(r->data, "r"));
    if (stats) TROP_TRY(check(stats, "stats"));
    TROP_TRY(residual_vectors(check, q));
    if (kept) {
        TROP_TRY(check(q.ku.codes, "u's copy"));
        TROP_TRY(check(q.ku.scales, "u's copy"));
        TROP_TRY(check(q.kr.codes, "r's copy"));
        TROP_TRY(check(q.kr.scales, "r's copy"));
        TROP_TRY(check_kept(check, q.kg, "gate's copy"));
    }
    return launch_residual_norm(q, mat(x), mat(y), (cudaStream_t)stream);
}

extern "C" int tropical_residual_norm_backward(const trop_residual_options* options, const trop_tensor* dy, const trop_tensor* dr,
                                               const trop_tensor* r, const trop_tensor* u, const trop_tensor* gate,
                                               const float* stats, const trop_kept* kept, int x_dtype, int u_dtype,
                                               const trop_residual_grads* grads, void* stream)
{
    clear_error();
    Residual q = {};
    if (!grads) return set_error(TROP_ERR_INVALID_ARG, "grads is NULL");
    TROP_TRY(matrix(dy, "dy", &q.rows, &q.cols));
    if (!kept) {
        TROP_TRY(same_shape(r, "r", q.rows, q.cols));
        TROP_TRY(same_shape(u, "u", q.rows, q.cols));
        x_dtype = r->dtype;
        u_dtype = u->dtype;
    } else if (r || u) {
        return set_error(TROP_ERR_INVALID_ARG, "r or u beside their 8-bit copies");
    }
    TROP_TRY(residual_types(x_dtype, u_dtype, dy->dtype));
    TROP_TRY(residual_options(options, dy->dtype, &q));
    if (q.cols == 0) return set_error(TROP_ERR_SHAPE, "a norm over no elements");
    TROP_TRY(extents(q.rows, q.cols));
    TROP_TRY(float_rows(dy, "dy", false));
    TROP_TRY(element_start(stats, "stats", 4));
    if (dr) {
        TROP_TRY(same_shape(dr, "dr", q.rows, q.cols));
        if (dr->dtype != x_dtype) return set_error(TROP_ERR_DTYPE, "dr has dtype %d, x %d", dr->dtype, x_dtype);
        TROP_TRY(float_rows(dr, "dr", false));
    }
    q.gate_cols = 1;
    q.r.dtype = x_dtype;
    q.u.dtype = u_dtype;
    if (kept) {
        TROP_TRY(kept8(kept[0].codes, kept[0].scales, "u's copy", q.rows, q.cols, false, &q.ku));
        TROP_TRY(kept8(kept[2].codes, kept[2].scales, "r's copy", q.rows, q.cols, false, &q.kr));
        q.has_gate = kept[1].codes || kept[1].scales;
        if (q.has_gate) {
            if (gate) return set_error(TROP_ERR_INVALID_ARG, "a gate beside its 8-bit copy");
            TROP_TRY(kept8(kept[1].codes, kept[1].scales, "gate's copy", q.rows, q.cols, false, &q.kg));
            q.gate_cols = q.cols;
        }
    } else {
        TROP_TRY(float_rows(r, "r", false));
        TROP_TRY(float_rows(u, "u", false));
        q.r = mat(r);
        q.u = mat(u);
    }
    if (gate) {
        TROP_TRY(residual_gate(gate, "gate", q.rows, q.cols, u_dtype, false, &q.gate_cols));
        if (kept && q.gate_cols == q.cols && q.cols > 1) return set_error(TROP_ERR_INVALID_ARG, "the gate's 8-bit copy is wanted beside r's and u's");
        q.has_gate = 1;
        q.gate = mat(gate);
        if (kept) q.gate_cols = 1;
    }
    ResidualGrads g = {};
    const struct {
        const trop_tensor* t;
        const char* name;
        int dtype;
        NormMat* to;
    } outs[] = {{grads->dx, "dx", x_dtype, &g.dx}, {grads->du, "du", u_dtype, &g.du}};
    for (const auto& o : outs) {
        if (!o.t) continue;
        TROP_TRY(same_shape(o.t, o.name, q.rows, q.cols));
        if (o.t->dtype != o.dtype) return set_error(TROP_ERR_DTYPE, "%s has dtype %d, not %d", o.name, o.t->dtype, o.dtype);
        TROP_TRY(float_rows(o.t, o.name, true));
        *o.to = mat(o.t);
    }
    if (grads->dgate) {
        int64_t cols;
        if (!q.has_gate) return set_error(TROP_ERR_INVALID_ARG, "the gradient of no gate");
        TROP_TRY(residual_gate(grads->dgate, "dgate", q.rows, q.gate_cols, u_dtype, true, &cols));
        if (cols != q.gate_cols) return set_error(TROP_ERR_SHAPE, "dgate has %lld columns, gate %lld", (long long)cols, (long long)q.gate_cols);
        g.dgate = mat(grads->dgate);
    }
    if (grads->dscale && !q.scale_vector) return set_error(TROP_ERR_INVALID_ARG, "the gradient of a scale that is no vector");
    if ((grads->dpost_weight || grads->dpost_bias) && !q.post)
        return set_error(TROP_ERR_INVALID_ARG, "the gradient of a norm that is left out");
    g.dscale = grads->dscale;
    g.dweight = grads->dweight;
    g.dbias = grads->dbias;
    g.dpost_weight = grads->dpost_weight;
    g.dpost_bias = grads->dpost_bias;
    const bool vectors = g.dscale || g.dweight || g.dbias || g.dpost_weight || g.dpost_bias;
    if (vectors && options->wdtype != dy->dtype && options->wdtype != TROP_F32)
        return set_error(TROP_ERR_DTYPE, "the vectors' gradients have dtype %d: dy's (%d) or f32 is wanted", options->wdtype, dy->dtype);
    const struct {
        void* p;
        const char* name;
    } vecs[] = {{g.dscale, "dscale"}, {g.dweight, "dweight"}, {g.dbias, "dbias"}, {g.dpost_weight, "dpost_weight"}, {g.dpost_bias, "dpost_bias"}};
    for (const auto& v : vecs)
        if (v.p) TROP_TRY(element_start(v.p, v.name, model_bytes(q.wdtype)));
    TROP_TRY(ensure_device(nullptr));
    if (!vectors && (q.rows == 0 || (!g.dx.p && !g.du.p && !g.dgate.p))) return TROP_OK;
    PointerCheck check;
    if (q.rows > 0) {
        TROP_TRY(check(dy->data, "dy"));
        if (dr) TROP_TRY(check(dr->data, "dr"));
        TROP_TRY(check(stats, "stats"));
        if (kept) {
            TROP_TRY(check(q.ku.codes, "u's copy"));
            TROP_TRY(check(q.ku.scales, "u's copy"));
            TROP_TRY(check(q.kr.codes, "r's copy"));
            TROP_TRY(check(q.kr.scales, "r's copy"));
            TROP_TRY(check_kept(check, q.kg, "gate's copy"));
        } else {
            TROP_TRY(check(r->data, "r"));
            TROP_TRY(check(u->data, "u"));
        }
        if (gate) TROP_TRY(check(gate->data, "gate"));
        if (grads->dx) TROP_TRY(check(g.dx.p, "dx"));
        if (grads->du) TROP_TRY(check(g.du.p, "du"));
        if (grads->dgate) TROP_TRY(check(g.dgate.p, "dgate"));
    }
    TROP_TRY(residual_vectors(check, q));  // (sums over no rows read them too)
    for (const auto& v : vecs)
        if (v.p) TROP_TRY(check(v.p, v.name));
    q.stats = const_cast<float*>(stats);
    return launch_residual_norm_backward(q, mat(dy), mat(dr), g, (cudaStream_t)stream);
}

extern "C" int tropical_activation_weight_grad(const trop_tensor* dy, const trop_tensor* codes, const trop_tensor* scales,
                                               const trop_tensor* dw, void* db, void* stream)
{
    clear_error();
    WeightGrad q = {};
    int64_t t, o, tc;
    TROP_TRY(matrix(dy, "dy", &t, &o));
    TROP_TRY(matrix(codes, "codes", &tc, &q.cols));
    if (!narrow(dy->dtype)) return set_error(TROP_ERR_DTYPE, "dy has dtype %d: bf16 or f16 is wanted", dy->dtype);
    if (tc != t) return set_error(TROP_ERR_SHAPE, "dy has %lld rows, codes %lld", (long long)t, (long long)tc);
    TROP_TRY(kept8(codes, scales, "codes", t, q.cols, false, &q.x));
    TROP_TRY(same_shape(dw, "dw", o, q.cols));
    if (dw->dtype != dy->dtype && dw->dtype != TROP_F32)
        return set_error(TROP_ERR_DTYPE, "dw has dtype %d: dy's (%d) or f32 is wanted", dw->dtype, dy->dtype);
    TROP_TRY(float_rows(dw, "dw", true));
    if ((uintptr_t)dy->data % 2) return set_error(TROP_ERR_INVALID_ARG, "dy does not start on an element of its type");
    if ((uintptr_t)db % model_bytes(dw->dtype)) return set_error(TROP_ERR_INVALID_ARG, "db does not start on an element of its type");
    TROP_TRY(extents(t, std::max(o, q.cols)));
    if ((o / 256 + 1) * (q.cols / 256 + 1) > INT32_MAX / 64) return set_error(TROP_ERR_UNSUPPORTED, "too many tiles for one call");
    TROP_TRY(ensure_device(nullptr));
    PointerCheck check;
    const bool some = o > 0 && q.cols > 0;
    if (some) TROP_TRY(check(dw->data, "dw"));
    if (db && o > 0) TROP_TRY(check(db, "db"));
    const int64_t words = dw->dtype == TROP_F32 ? 2 : 1;  // 16-bit words of an element
    if (t == 0) {  // sums over no tokens
        if (some) TROP_TRY(launch_zero16({dw->data, o, q.cols * words, dw->stride[0] * words, 1}, (cudaStream_t)stream));
        if (db && o > 0) TROP_TRY(launch_zero16({db, 1, o * words, o * words, 1}, (cudaStream_t)stream));
        return TROP_OK;
    }
    if (o == 0 || (!some && !db)) return TROP_OK;
    TROP_TRY(check(dy->data, "dy"));
    if (some) {
        TROP_TRY(check(codes->data, "codes"));
        TROP_TRY(check(scales->data, "scales"));
    }
    q.bf16 = dy->dtype == TROP_BF16;
    q.dy = {dy->data, t, o, dy->stride[0], dy->stride[1]};
    q.wide = dw->dtype == TROP_F32;
    q.dw = dw->data;
    q.ldw = dw->stride[0];
    q.db = db;
    return launch_weight_grad(q, (cudaStream_t)stream);
}
