// train.h -- what the training operators' entry points (train.cpp) hand to their kernels
// (layer_norm.cu, linear_ce.cu, adamw.cu).  All extents and strides are in elements; everything
// here has been validated.
#pragma once

#include <stdint.h>

#include "internal.h"

namespace trop {

// element types of these operators, by their trop_dtype codes
inline bool is_model_float(int dtype) { return dtype == TROP_F32 || dtype == TROP_BF16 || dtype == TROP_F16; }
inline size_t model_bytes(int dtype) { return dtype == TROP_F32 ? 4 : is_model_float(dtype) ? 2 : 0; }

// ---------------------------------------------------------------- layer norm
struct NormMat {  // [rows, cols], columns contiguous
    void* p;
    int64_t sr;
    int dtype;
};
struct NormVec {  // [cols], contiguous; p null: absent
    void* p;
    int dtype;
};
int launch_layer_norm(int64_t rows, int64_t cols, const NormMat& x, const NormVec& w, const NormVec& b, double eps,
                      const NormMat& y, float* mean, float* rstd, cudaStream_t s);
int launch_layer_norm_backward(int64_t rows, int64_t cols, const NormMat& dy, const NormMat& x, const float* mean,
                               const float* rstd, const NormVec& w, const NormMat& dx, const NormVec& dw,
                               const NormVec& db, cudaStream_t s);

// ---------------------------------------------------------------- cross entropy of a linear head
struct Mat16 {  // 16-bit matrix
    void* p;
    int64_t rows, cols, sr, sc;
};
struct LinearCe {
    int bf16;      // else f16
    Mat16 x, w;    // tokens [N, D], weights [V, D]; N, D, V > 0
    const void* target;
    int64_t starget, ignore;
    int target_wide;  // int64, else int32
};
int launch_linear_ce(const LinearCe& q, float* loss, float* lse, float* total, float* kept, int mean, cudaStream_t s);
// dx, dw: null or with contiguous columns
int launch_linear_ce_backward(const LinearCe& q, const float* g, int64_t sg, const float* lse, const float* kept,
                              const Mat16* dx, const Mat16* dw, cudaStream_t s);
int launch_zero16(const Mat16& m, cudaStream_t s);

// ---------------------------------------------------------------- AdamW
// The step's scalars, rounded to f32 from the caller's doubles.
struct AdamwScalars {
    float b1, c1, b2, c2;     // beta and 1 - beta
    float k2, eps;            // 1 / sqrt(1 - beta2^step)
    float decay, lr;          // 1 - lr weight_decay; lr / (1 - beta1^step)
    float gscale;             // the gradient's factor
};
// A plan's tensors (and the states whose values are wanted), laid out in device memory.
struct AdamwTables;
AdamwTables* adamw_tables();
void adamw_tables_free(AdamwTables* t);
int adamw_tables_fill(AdamwTables* a, int64_t n, const trop_adamw_tensor* t, int pdtype, int gdtype, int state8,
                      int copy_dtype);
int adamw_states_fill(AdamwTables* a, int64_t n, const trop_adamw_state* t);
int launch_adamw_plan(const AdamwTables& a, const AdamwScalars& k, cudaStream_t s);
int launch_adamw_plan_values(const AdamwTables& a, cudaStream_t s);
// One call's tensors, in the launches' parameters.
int launch_adamw(int64_t n, const trop_adamw_tensor* t, int pdtype, int gdtype, int state8, int copy_dtype,
                 const AdamwScalars& k, cudaStream_t s);
int launch_adamw_values(int64_t n, const trop_adamw_state* t, cudaStream_t s);

}  // namespace trop
