// operands.h -- 16-bit operands of the tensor-core kernels (linear_ce.cu, weight_grad.cu) as TMA reads them: tensor
// maps, and packed copies of matrices whose rows do not lie on 16 bytes.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "train.h"

namespace trop {

// a row-major matrix of bf16, f16 or f32, its rows 16-byte aligned, in boxes of `box_rows` x 128 bytes
int make_map(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows);

struct Matrix16 {
    const uint16_t* p;
    int64_t rows, cols, ld;
};

// One operand's copy by k_pack.
struct Pack {
    const uint16_t* in;
    int64_t sr, sc, rows, cols;
    uint16_t* out;
    int64_t ld;
    Span sp;
};

// The operands as TMA can read them: themselves, or packed copies, both made by one launch.
struct Operand {
    Matrix16 m;
    const Mat16& a;
    size_t at = 0;
    bool packed = false;
    Operand(const Mat16& a_, Workspace& ws) : m{(const uint16_t*)a_.p, a_.rows, a_.cols, a_.sr}, a(a_)
    {
        if (a.rows == 1) m.ld = (a.cols + 7) / 8 * 8;  // no second row: any pitch
        packed = !((a.sc == 1 || a.cols == 1) && m.ld % 8 == 0 && m.ld >= a.cols && m.ld < (int64_t)1 << 38 &&
                   ((uintptr_t)a.p & 15) == 0);
        if (!packed) return;
        m.ld = (a.cols + 7) / 8 * 8;
        at = ws.add((size_t)a.rows * m.ld * 2);
    }
    Pack job() const
    {
        const int64_t size[2] = {a.rows, a.cols}, stride[2] = {a.sr, a.sc};
        const Span sp = span_of(a.p, 2, 2, size, stride);
        return {(const uint16_t*)a.p, a.sr, a.sc, a.rows, a.cols, const_cast<uint16_t*>(m.p), m.ld, sp};
    }
};
int pack(Operand& x, Operand& w, const Workspace& ws, int sm);  // the copies of those that need one
int pack(Operand& x, const Workspace& ws, int sm);

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
// Splits of a product's depth of kt stages: the fewest rounds of stages, each split costing about the time of
// 8 stages more for its partial sums of `bytes` (1 GiB of them at most).  dw of 8192x128x256, one tile of 128
// stages, takes 64 splits: the whole backward pass 30 us, without splits 55 us.
int splits(int tiles, int kt, int teams, int64_t bytes);

}  // namespace trop
