// block.h -- what the entry points of a residual block's operators (block.cpp) hand to their kernels
// (activation.cu, residual_norm.cu, weight_grad.cu).  Everything here has been validated; strides are in elements.
#pragma once

#include <stdint.h>

#include "train.h"

namespace trop {

// ---------------------------------------------------------------- activations in 8 bits (pack8.h)
struct Kept8 {  // codes [rows, cols] and scales [rows, groups], columns contiguous; codes null: absent
    int8_t* codes;
    int64_t sc;
    uint8_t* scales;
    int64_t ss;
};
int launch_activation_pack(int64_t rows, int64_t cols, const NormMat& x, const Kept8& k, cudaStream_t s);
int launch_activation_values(int64_t rows, int64_t cols, const Kept8& k, const NormMat& x, cudaStream_t s);

// ---------------------------------------------------------------- norms around a block
struct Residual {
    int64_t rows, cols, gate_cols;  // gate_cols: cols, or 1
    int rms, post, act, has_gate;
    double eps, alpha, scale;
    int wdtype;  // of the vectors below, [cols], null: absent
    const void *weight, *bias, *post_weight, *post_bias, *scale_vector;
    NormMat u, gate, r;  // backward from 8-bit copies: only their types (r, u; a row's gate as it is)
    Kept8 ku, kg, kr;    // forward: where the copies go; backward: what is read
    float* stats;        // [4][rows]
};
struct ResidualGrads {  // null: not wanted
    NormMat dx, du, dgate;
    void *dscale, *dweight, *dbias, *dpost_weight, *dpost_bias;
};
int launch_residual_norm(const Residual& q, const NormMat& x, const NormMat& y, cudaStream_t s);  // writes q.r
int launch_residual_norm_backward(const Residual& q, const NormMat& dy, const NormMat& dr, const ResidualGrads& g, cudaStream_t s);

// ---------------------------------------------------------------- the weight gradient from an 8-bit copy
struct WeightGrad {
    int bf16;      // dy's type, else f16
    Mat16 dy;      // [T, O]; T, O, cols > 0
    int64_t cols;  // C
    Kept8 x;       // [T, C]
    int wide;      // results in f32, else in dy's type
    void* dw;      // [O, C], rows of ldw
    int64_t ldw;
    void* db;      // [O], null: not wanted
};
int launch_weight_grad(const WeightGrad& q, cudaStream_t s);

}  // namespace trop
