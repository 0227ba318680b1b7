// residual_job.h -- what residual_norm.cu hands to the kernels of residual_norm.cuh.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "block.h"

namespace trop {

using bf16 = __nv_bfloat16;
enum { GATE_NONE = 0, GATE_ROW = 1, GATE_FULL = 2 };
enum { SUM_W = 1, SUM_B = 2, SUM_1 = 4, SUM_2 = 8 };  // column sums that are wanted

struct Rows8 {  // 8-bit copies, null: absent
    int8_t* codes;
    int64_t sc;
    uint8_t* scales;
    int64_t ss;
    Span sp_c, sp_s;
    uint32_t sb = 0, ssb = 0;  // the strides, where 32 bits hold them
};
struct RowsAt {
    void* p;
    int64_t s;
    Span sp;
    uint32_t sb = 0;  // the stride in bytes, where 32 bits hold it
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

// by the types of x and r, of u and gate, of y
template <typename S, typename U, typename Y>
int residual_forward(ResJob j, int sm, cudaStream_t s);
template <typename S, typename U, typename Y, bool CODED>
int residual_backward(ResJob j, JoinJob t, int sm, cudaStream_t s);

}  // namespace trop
