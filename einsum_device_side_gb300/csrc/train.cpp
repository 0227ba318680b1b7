// train.cpp -- entry points of the training operators: argument checks, then layer_norm.cu,
// linear_ce.cu and adamw.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "train.h"

using namespace trop;

namespace {

constexpr int64_t MOST = INT32_MAX - 1024;  // rows and columns the kernels index in 32 bits

// Device-pointer checks of a call's tensors: one driver query each (a third of the runtime's), and none for
// a pointer inside an allocation already checked in this call (torch's allocator hands out pieces of a
// few large ones).  Whatever is not plain memory of the current device goes the long way.
struct PointerCheck {
    uintptr_t lo[16], hi[16];
    int n = 0, at = 0, device = -1;
    PointerCheck() { cudaGetDevice(&device); }
    int operator()(const void* p, const char* name)
    {
        const uintptr_t a = (uintptr_t)p;
        for (int i = 0; i < n; ++i)
            if (a >= lo[i] && a < hi[i]) return TROP_OK;
        using Fn = CUresult (*)(unsigned int, CUpointer_attribute*, void**, CUdeviceptr);
        static const Fn query = [] {
            void* f = nullptr;
            cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
            if (cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
                q != cudaDriverEntryPointSuccess) {
                cudaGetLastError();
                f = nullptr;
            }
            return (Fn)f;
        }();
        unsigned int type = 0;
        int ordinal = -1;
        CUdeviceptr base = 0;
        size_t size = 0;
        CUpointer_attribute what[4] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL,
                                       CU_POINTER_ATTRIBUTE_RANGE_START_ADDR, CU_POINTER_ATTRIBUTE_RANGE_SIZE};
        void* to[4] = {&type, &ordinal, &base, &size};
        if (!p || !query || query(4, what, to, (CUdeviceptr)a) != CUDA_SUCCESS || type != CU_MEMORYTYPE_DEVICE || ordinal != device)
            return check_device_pointer(p, name);
        if (size) {
            lo[at] = base;
            hi[at] = base + size;
            at = (at + 1) % 16;
            if (n < 16) ++n;
        }
        return TROP_OK;
    }
};

int matrix(const trop_tensor* t, const char* name, int64_t* rows, int64_t* cols)
{
    if (!t) return set_error(TROP_ERR_INVALID_ARG, "%s is NULL", name);
    if (t->rank != 2) return set_error(TROP_ERR_INVALID_ARG, "%s has rank %d, not 2", name, t->rank);
    if (t->shape[0] < 0 || t->shape[1] < 0) return set_error(TROP_ERR_INVALID_ARG, "%s has a negative extent", name);
    *rows = t->shape[0];
    *cols = t->shape[1];
    return TROP_OK;
}
int same_shape(const trop_tensor* t, const char* name, int64_t rows, int64_t cols)
{
    int64_t r, c;
    TROP_TRY(matrix(t, name, &r, &c));
    if (r != rows || c != cols)
        return set_error(TROP_ERR_SHAPE, "%s is %lld x %lld, not %lld x %lld", name, (long long)r, (long long)c,
                         (long long)rows, (long long)cols);
    return TROP_OK;
}
// rows of contiguous elements that do not overlap one another when written
int row_layout(const trop_tensor* t, const char* name, bool written)
{
    if (t->shape[1] > 1 && t->stride[1] != 1)
        return set_error(TROP_ERR_UNSUPPORTED, "%s: the last axis must be contiguous (stride %lld)", name,
                         (long long)t->stride[1]);
    if (t->shape[0] > 1 && (t->stride[0] < 0 || (written && t->stride[0] < t->shape[1])))
        return set_error(TROP_ERR_INVALID_ARG, "%s: row stride %lld", name, (long long)t->stride[0]);
    return TROP_OK;
}

int norm_types(const trop_tensor* x, const char* other, int other_dtype, int wdtype, bool has_w)
{
    if (!is_model_float(x->dtype)) return set_error(TROP_ERR_DTYPE, "x has dtype %d: f32, bf16 or f16 is wanted", x->dtype);
    if (other_dtype != x->dtype && !(x->dtype == TROP_F32 && (other_dtype == TROP_BF16 || other_dtype == TROP_F16)))
        return set_error(TROP_ERR_DTYPE, "%s has dtype %d beside x's %d: x's own, or bf16 or f16 beside f32", other,
                         other_dtype, x->dtype);
    if (has_w && wdtype != x->dtype && wdtype != TROP_F32)
        return set_error(TROP_ERR_DTYPE, "weight and bias have dtype %d: x's (%d) or f32 is wanted", wdtype, x->dtype);
    return TROP_OK;
}

}  // namespace

extern "C" int tropical_layer_norm(const trop_tensor* x, const void* weight, const void* bias, int wdtype, double eps,
                                   const trop_tensor* y, float* mean, float* rstd, void* stream)
{
    clear_error();
    int64_t rows, cols;
    TROP_TRY(matrix(x, "x", &rows, &cols));
    TROP_TRY(same_shape(y, "y", rows, cols));
    TROP_TRY(norm_types(x, "y", y->dtype, wdtype, weight || bias));
    if (!(eps >= 0)) return set_error(TROP_ERR_INVALID_ARG, "eps = %g", eps);
    if (cols == 0) return set_error(TROP_ERR_SHAPE, "a norm over no elements");
    if (rows > MOST || cols > MOST) return set_error(TROP_ERR_UNSUPPORTED, "extents above %lld", (long long)MOST);
    TROP_TRY(row_layout(x, "x", false));
    TROP_TRY(row_layout(y, "y", true));
    TROP_TRY(ensure_device(nullptr));
    if (rows == 0) return TROP_OK;
    PointerCheck check;
    TROP_TRY(check(x->data, "x"));
    TROP_TRY(check(y->data, "y"));
    if (weight) TROP_TRY(check(weight, "weight"));
    if (bias) TROP_TRY(check(bias, "bias"));
    if (mean) TROP_TRY(check(mean, "mean"));
    if (rstd) TROP_TRY(check(rstd, "rstd"));
    return launch_layer_norm(rows, cols, {x->data, x->stride[0], x->dtype}, {(void*)weight, wdtype},
                             {(void*)bias, wdtype}, eps, {y->data, y->stride[0], y->dtype}, mean, rstd,
                             (cudaStream_t)stream);
}

extern "C" int tropical_layer_norm_backward(const trop_tensor* dy, const trop_tensor* x, const float* mean,
                                            const float* rstd, const void* weight, int wdtype, const trop_tensor* dx,
                                            void* dweight, void* dbias, void* stream)
{
    clear_error();
    int64_t rows, cols;
    TROP_TRY(matrix(x, "x", &rows, &cols));
    TROP_TRY(same_shape(dy, "dy", rows, cols));
    TROP_TRY(norm_types(x, "dy", dy->dtype, wdtype, weight || dweight || dbias));
    if (dx) {
        TROP_TRY(same_shape(dx, "dx", rows, cols));
        if (dx->dtype != x->dtype) return set_error(TROP_ERR_DTYPE, "dx has dtype %d, x %d", dx->dtype, x->dtype);
        TROP_TRY(row_layout(dx, "dx", true));
    }
    if (cols == 0) return set_error(TROP_ERR_SHAPE, "a norm over no elements");
    if (rows > MOST || cols > MOST) return set_error(TROP_ERR_UNSUPPORTED, "extents above %lld", (long long)MOST);
    TROP_TRY(row_layout(x, "x", false));
    TROP_TRY(row_layout(dy, "dy", false));
    TROP_TRY(ensure_device(nullptr));
    PointerCheck check;
    if (rows > 0) {
        TROP_TRY(check(x->data, "x"));
        TROP_TRY(check(dy->data, "dy"));
        TROP_TRY(check(mean, "mean"));
        TROP_TRY(check(rstd, "rstd"));
        if (weight) TROP_TRY(check(weight, "weight"));
        if (dx) TROP_TRY(check(dx->data, "dx"));
    }
    if (dweight) TROP_TRY(check(dweight, "dweight"));
    if (dbias) TROP_TRY(check(dbias, "dbias"));
    if (!dx && !dweight && !dbias) return TROP_OK;
    NormMat out = {nullptr, 0, x->dtype};
    if (dx) out = {dx->data, dx->stride[0], dx->dtype};
    return launch_layer_norm_backward(rows, cols, {dy->data, dy->stride[0], dy->dtype},
                                      {x->data, x->stride[0], x->dtype}, mean, rstd, {(void*)weight, wdtype}, out,
                                      {dweight, wdtype}, {dbias, wdtype}, (cudaStream_t)stream);
}

namespace {

// The operands both directions share.
int ce_operands(const trop_tensor* x, const trop_tensor* w, const trop_tensor* target, int64_t ignore_index, LinearCe* q)
{
    int64_t n, d, v, dw;
    TROP_TRY(matrix(x, "x", &n, &d));
    TROP_TRY(matrix(w, "w", &v, &dw));
    if (x->dtype != TROP_BF16 && x->dtype != TROP_F16)
        return set_error(TROP_ERR_DTYPE, "x has dtype %d: bf16 or f16 is wanted", x->dtype);
    if (w->dtype != x->dtype) return set_error(TROP_ERR_DTYPE, "w has dtype %d, x %d", w->dtype, x->dtype);
    if (!target || target->rank != 1) return set_error(TROP_ERR_INVALID_ARG, "target must have rank 1");
    if (target->dtype != TROP_I32 && target->dtype != TROP_I64)
        return set_error(TROP_ERR_DTYPE, "target has dtype %d: i32 or i64 is wanted", target->dtype);
    if (dw != d) return set_error(TROP_ERR_SHAPE, "x has %lld columns, w %lld", (long long)d, (long long)dw);
    if (target->shape[0] != n)
        return set_error(TROP_ERR_SHAPE, "%lld targets for %lld tokens", (long long)target->shape[0], (long long)n);
    if (d == 0 || v == 0) return set_error(TROP_ERR_SHAPE, "an empty vocabulary or empty vectors");
    if (n > MOST || d > MOST || v > MOST) return set_error(TROP_ERR_UNSUPPORTED, "extents above %lld", (long long)MOST);
    // tiles are counted in 32 bits
    if ((n / 128 + 1) * (v / 256 + 1) > INT32_MAX || (n / 128 + 1) * (d / 256 + 1) > INT32_MAX / 64 ||
        (v / 128 + 1) * (d / 256 + 1) > INT32_MAX)
        return set_error(TROP_ERR_UNSUPPORTED, "too many tiles for one call");
    *q = {x->dtype == TROP_BF16,
          {x->data, n, d, x->stride[0], x->stride[1]},
          {w->data, v, d, w->stride[0], w->stride[1]},
          target->data,
          target->stride[0],
          ignore_index,
          target->dtype == TROP_I64};
    return TROP_OK;
}

}  // namespace

extern "C" int tropical_linear_cross_entropy(const trop_tensor* x, const trop_tensor* w, const trop_tensor* target,
                                             int64_t ignore_index, int mean, float* loss, float* lse, float* total,
                                             float* kept, void* stream)
{
    clear_error();
    LinearCe q;
    TROP_TRY(ce_operands(x, w, target, ignore_index, &q));
    if (!lse && q.x.rows > 0) return set_error(TROP_ERR_INVALID_ARG, "lse is NULL");
    TROP_TRY(ensure_device(nullptr));
    PointerCheck check;
    if (q.x.rows > 0) {
        TROP_TRY(check(x->data, "x"));
        TROP_TRY(check(w->data, "w"));
        TROP_TRY(check(target->data, "target"));
        TROP_TRY(check(lse, "lse"));
        if (loss) TROP_TRY(check(loss, "loss"));
    } else if (!total && !kept) {
        return TROP_OK;
    }
    if (total) TROP_TRY(check(total, "total"));
    if (kept) TROP_TRY(check(kept, "kept"));
    return launch_linear_ce(q, loss, lse, total, kept, mean, (cudaStream_t)stream);
}

extern "C" int tropical_linear_cross_entropy_backward(const float* dloss, int64_t dloss_stride, const trop_tensor* x,
                                                      const trop_tensor* w, const trop_tensor* target,
                                                      int64_t ignore_index, const float* lse, const float* kept,
                                                      const trop_tensor* dx, const trop_tensor* dw, void* stream)
{
    clear_error();
    LinearCe q;
    TROP_TRY(ce_operands(x, w, target, ignore_index, &q));
    Mat16 out[2];
    const Mat16* want[2] = {nullptr, nullptr};
    const trop_tensor* grads[2] = {dx, dw};
    for (int i = 0; i < 2; ++i) {
        const trop_tensor* t = grads[i];
        if (!t) continue;
        const char* name = i ? "dw" : "dx";
        TROP_TRY(same_shape(t, name, i ? q.w.rows : q.x.rows, q.x.cols));
        if (t->dtype != x->dtype) return set_error(TROP_ERR_DTYPE, "%s has dtype %d, x %d", name, t->dtype, x->dtype);
        TROP_TRY(row_layout(t, name, true));
        out[i] = {t->data, t->shape[0], t->shape[1], t->stride[0], 1};
        if (t->shape[0] > 0) want[i] = &out[i];
    }
    if (!want[0] && !want[1]) return TROP_OK;
    TROP_TRY(ensure_device(nullptr));
    PointerCheck check;
    for (int i = 0; i < 2; ++i)
        if (want[i]) TROP_TRY(check(out[i].p, i ? "dw" : "dx"));
    if (q.x.rows == 0) return want[1] ? launch_zero16(out[1], (cudaStream_t)stream) : TROP_OK;
    TROP_TRY(check(x->data, "x"));
    TROP_TRY(check(w->data, "w"));
    TROP_TRY(check(target->data, "target"));
    TROP_TRY(check(lse, "lse"));
    TROP_TRY(check(dloss, "dloss"));
    if (kept) TROP_TRY(check(kept, "kept"));
    return launch_linear_ce_backward(q, dloss, dloss_stride, lse, kept, want[0], want[1], (cudaStream_t)stream);
}

namespace {

int adamw_tensors(int64_t n, const trop_adamw_tensor* tensors, int param_dtype, int grad_dtype, int state_bits,
                  int copy_dtype)
{
    if (n < 0 || (n > 0 && !tensors)) return set_error(TROP_ERR_INVALID_ARG, "n = %lld or a NULL argument", (long long)n);
    if (!is_model_float(param_dtype) || !is_model_float(grad_dtype))
        return set_error(TROP_ERR_DTYPE, "parameters of dtype %d, gradients of %d: f32, bf16 or f16 is wanted",
                         param_dtype, grad_dtype);
    if (param_dtype != TROP_F32 && grad_dtype != param_dtype && grad_dtype != TROP_F32)
        return set_error(TROP_ERR_DTYPE, "gradients of dtype %d beside parameters of %d", grad_dtype, param_dtype);
    if (state_bits != 8 && state_bits != 32) return set_error(TROP_ERR_INVALID_ARG, "states of %d bits", state_bits);
    TROP_TRY(ensure_device(nullptr));
    PointerCheck check;
    for (int64_t i = 0; i < n; ++i) {
        const trop_adamw_tensor& t = tensors[i];
        if (t.numel < 0) return set_error(TROP_ERR_INVALID_ARG, "tensor %lld has %lld elements", (long long)i, (long long)t.numel);
        if (t.numel == 0) continue;
        TROP_TRY(check(t.param, "param"));
        TROP_TRY(check(t.grad, "grad"));
        TROP_TRY(check(t.exp_avg, "exp_avg"));
        TROP_TRY(check(t.exp_avg_sq, "exp_avg_sq"));
        if (state_bits == 8) {
            TROP_TRY(check(t.exp_avg_scale, "exp_avg_scale"));
            TROP_TRY(check(t.exp_avg_sq_scale, "exp_avg_sq_scale"));
        }
        if (t.copy) {
            if (param_dtype != TROP_F32 || (copy_dtype != TROP_BF16 && copy_dtype != TROP_F16))
                return set_error(TROP_ERR_DTYPE, "a copy of dtype %d of parameters of dtype %d: bf16 or f16 of f32",
                                 copy_dtype, param_dtype);
            TROP_TRY(check(t.copy, "copy"));
        }
    }
    return TROP_OK;
}

int adamw_states(int64_t n, const trop_adamw_state* states)
{
    if (n < 0 || (n > 0 && !states)) return set_error(TROP_ERR_INVALID_ARG, "n = %lld or a NULL argument", (long long)n);
    TROP_TRY(ensure_device(nullptr));
    PointerCheck check;
    for (int64_t i = 0; i < n; ++i) {
        const trop_adamw_state& t = states[i];
        if (t.numel < 0) return set_error(TROP_ERR_INVALID_ARG, "tensor %lld has %lld elements", (long long)i, (long long)t.numel);
        if (t.numel == 0) continue;
        TROP_TRY(check(t.exp_avg, "exp_avg"));
        TROP_TRY(check(t.exp_avg_sq, "exp_avg_sq"));
        TROP_TRY(check(t.exp_avg_scale, "exp_avg_scale"));
        TROP_TRY(check(t.exp_avg_sq_scale, "exp_avg_sq_scale"));
        TROP_TRY(check(t.exp_avg_value, "exp_avg_value"));
        TROP_TRY(check(t.exp_avg_sq_value, "exp_avg_sq_value"));
    }
    return TROP_OK;
}

int adamw_scalars(const trop_adamw_options* o, AdamwScalars* k)
{
    if (!o) return set_error(TROP_ERR_INVALID_ARG, "options is NULL");
    if (o->step < 1) return set_error(TROP_ERR_INVALID_ARG, "step %lld: the first is 1", (long long)o->step);
    if (!(o->beta1 >= 0 && o->beta1 < 1 && o->beta2 >= 0 && o->beta2 < 1 && o->eps >= 0) || !std::isfinite(o->lr) ||
        !std::isfinite(o->weight_decay) || !std::isfinite(o->eps) || !std::isfinite(o->grad_scale))
        return set_error(TROP_ERR_INVALID_ARG, "lr %g, betas %g %g, eps %g, weight decay %g, gradient scale %g", o->lr,
                         o->beta1, o->beta2, o->eps, o->weight_decay, o->grad_scale);
    const double first = 1.0 - std::pow(o->beta1, (double)o->step), second = 1.0 - std::pow(o->beta2, (double)o->step);
    *k = {(float)o->beta1,
          (float)(1.0 - o->beta1),
          (float)o->beta2,
          (float)(1.0 - o->beta2),
          (float)(1.0 / std::sqrt(second)),
          (float)o->eps,
          (float)(1.0 - o->lr * o->weight_decay),
          (float)(o->lr / first),
          (float)o->grad_scale};
    return TROP_OK;
}

// No C++ exception leaves an entry point: the tables' memory is the only thing here that can throw.
template <typename F>
int guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return set_error(TROP_ERR_OOM, "host memory for the tensor table");
    }
}

struct TablesOwner {
    AdamwTables* t = adamw_tables();
    ~TablesOwner() { adamw_tables_free(t); }
};

}  // namespace

struct trop_adamw_plan_s {
    TablesOwner tables;
    int device = 0;
    bool values = false;
};

extern "C" int tropical_adamw_step(int64_t n, const trop_adamw_tensor* tensors, int param_dtype, int grad_dtype,
                                   int state_bits, int copy_dtype, const trop_adamw_options* options, void* stream)
{
    clear_error();
    AdamwScalars k;
    TROP_TRY(adamw_scalars(options, &k));
    TROP_TRY(adamw_tensors(n, tensors, param_dtype, grad_dtype, state_bits, copy_dtype));
    return launch_adamw(n, tensors, param_dtype, grad_dtype, state_bits == 8, copy_dtype, k, (cudaStream_t)stream);
}

extern "C" int tropical_adamw_state_values(int64_t n, const trop_adamw_state* states, void* stream)
{
    clear_error();
    TROP_TRY(adamw_states(n, states));
    return launch_adamw_values(n, states, (cudaStream_t)stream);
}

extern "C" int tropical_adamw_plan_create(int64_t n, const trop_adamw_tensor* tensors, int param_dtype, int grad_dtype,
                                          int state_bits, int copy_dtype, const trop_adamw_state* states,
                                          trop_adamw_plan* plan)
{
    clear_error();
    if (!plan) return set_error(TROP_ERR_INVALID_ARG, "plan is NULL");
    *plan = nullptr;
    TROP_TRY(adamw_tensors(n, tensors, param_dtype, grad_dtype, state_bits, copy_dtype));
    if (states) {
        if (state_bits != 8) return set_error(TROP_ERR_INVALID_ARG, "values of states that are not in 8 bits");
        TROP_TRY(adamw_states(n, states));
    }
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    return guarded([&] {
        struct Held {
            trop_adamw_plan p;
            ~Held() { delete p; }
        } held{new trop_adamw_plan_s()};
        held.p->device = dev->device;
        TROP_TRY(adamw_tables_fill(held.p->tables.t, n, tensors, param_dtype, grad_dtype, state_bits == 8, copy_dtype));
        if (states) {
            TROP_TRY(adamw_states_fill(held.p->tables.t, n, states));
            held.p->values = true;
        }
        *plan = held.p;
        held.p = nullptr;
        return (int)TROP_OK;
    });
}

namespace {
int plan_ready(trop_adamw_plan plan)
{
    if (!plan) return set_error(TROP_ERR_INVALID_ARG, "plan is NULL");
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    if (dev->device != plan->device)
        return set_error(TROP_ERR_DEVICE_MISMATCH, "the plan is for device %d, current device is %d", plan->device, dev->device);
    return TROP_OK;
}
}  // namespace

extern "C" int tropical_adamw_plan_step(trop_adamw_plan plan, const trop_adamw_options* options, void* stream)
{
    clear_error();
    AdamwScalars k;
    TROP_TRY(adamw_scalars(options, &k));
    TROP_TRY(plan_ready(plan));
    return launch_adamw_plan(*plan->tables.t, k, (cudaStream_t)stream);
}

extern "C" int tropical_adamw_plan_values(trop_adamw_plan plan, void* stream)
{
    clear_error();
    TROP_TRY(plan_ready(plan));
    if (!plan->values) return set_error(TROP_ERR_INVALID_ARG, "the plan was made without buffers for the states' values");
    return launch_adamw_plan_values(*plan->tables.t, (cudaStream_t)stream);
}

extern "C" int tropical_adamw_plan_destroy(trop_adamw_plan plan)
{
    clear_error();
    delete plan;
    return TROP_OK;
}
