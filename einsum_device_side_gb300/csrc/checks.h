// checks.h -- argument checks that the training operators' entry points share (train.cpp, block.cpp).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace trop {

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

inline int matrix(const trop_tensor* t, const char* name, int64_t* rows, int64_t* cols)
{
    if (!t) return set_error(TROP_ERR_INVALID_ARG, "%s is NULL", name);
    if (t->rank != 2) return set_error(TROP_ERR_INVALID_ARG, "%s has rank %d, not 2", name, t->rank);
    if (t->shape[0] < 0 || t->shape[1] < 0) return set_error(TROP_ERR_INVALID_ARG, "%s has a negative extent", name);
    *rows = t->shape[0];
    *cols = t->shape[1];
    return TROP_OK;
}
inline int same_shape(const trop_tensor* t, const char* name, int64_t rows, int64_t cols)
{
    int64_t r, c;
    TROP_TRY(matrix(t, name, &r, &c));
    if (r != rows || c != cols)
        return set_error(TROP_ERR_SHAPE, "%s is %lld x %lld, not %lld x %lld", name, (long long)r, (long long)c,
                         (long long)rows, (long long)cols);
    return TROP_OK;
}
// rows of contiguous elements that do not overlap one another when written
inline int row_layout(const trop_tensor* t, const char* name, bool written)
{
    if (t->shape[1] > 1 && t->stride[1] != 1)
        return set_error(TROP_ERR_UNSUPPORTED, "%s: the last axis must be contiguous (stride %lld)", name,
                         (long long)t->stride[1]);
    if (t->shape[0] > 1 && (t->stride[0] < 0 || (written && t->stride[0] < t->shape[1])))
        return set_error(TROP_ERR_INVALID_ARG, "%s: row stride %lld", name, (long long)t->stride[0]);
    return TROP_OK;
}

}  // namespace trop
