// operands.cu -- see operands.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#define TROP_TU 10  // this file's id in a bounds-violation record
#include "operands.h"

namespace trop {
namespace {

// The copy of one operand, or of both: rows of consecutive elements by a warp each, in 4-byte words (a row
// that starts inside a word shifts two of them together; a word that reaches outside the matrix is read by
// halves), any other strides an element at a time.  60000x2049: 92 us, 5.3 TB/s; by elements 285 us.
constexpr int PACK_WORDS = 8;  // of a thread at once: 64 warps then have 64 KB of an SM on their way
__global__ void __launch_bounds__(256) k_pack(const Pack first, const Pack second)
{
    pdl_wait();
    pdl_signal();
    const Pack& a = blockIdx.y ? second : first;
    const uint16_t* const in = a.in;
    uint16_t* const out = a.out;
    const int64_t sr = a.sr, rows = a.rows, cols = a.cols, ld = a.ld;
    const Span& sp_in = a.sp;
    (void)sp_in;
    if (a.sc != 1 || sr < 0) {
        const int64_t n = rows * cols, sc = a.sc;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.y * 32 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
            const int64_t r = i / cols, c = i % cols;
            const uint16_t* p = in + r * sr + c * sc;
            out[r * ld + c] = TROP_IN(p, 2, sp_in) ? *p : (uint16_t)0;
        }
        return;
    }
    const uint16_t* const end = in + (rows - 1) * sr + cols;
    const int64_t words = (cols + 1) / 2;
    for (int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.y; r < rows; r += (int64_t)gridDim.x * 8) {
        const uint16_t* const row = in + r * sr;
        uint32_t* const to = reinterpret_cast<uint32_t*>(out + r * ld);
        const int odd = ((uintptr_t)row & 2) != 0;
        for (int64_t at = threadIdx.x; at < words; at += 32 * PACK_WORDS) {
            uint32_t lo[PACK_WORDS], hi[PACK_WORDS];
            const int64_t begin = at - threadIdx.x;
            if (begin + 32 * PACK_WORDS < words && (row > in || begin > 0)) {  // nothing reaches outside
                const uint32_t* const src = reinterpret_cast<const uint32_t*>(row - odd) + at;
#pragma unroll
                for (int u = 0; u < PACK_WORDS; ++u) {
                    lo[u] = TROP_IN(src + 32 * u, 4, sp_in) ? src[32 * u] : 0;
                    hi[u] = odd && TROP_IN(src + 32 * u + 1, 4, sp_in) ? src[32 * u + 1] : 0;
                }
#pragma unroll
                for (int u = 0; u < PACK_WORDS; ++u) to[at + 32 * u] = odd ? __funnelshift_r(lo[u], hi[u], 16) : lo[u];
                continue;
            }
#pragma unroll
            for (int u = 0; u < PACK_WORDS; ++u) {
                lo[u] = hi[u] = 0;
                if (at + 32 * u >= words) continue;
                const uint16_t* const p = row + 2 * (at + 32 * u);
                if (p - odd >= in && p - odd + 2 <= end) {
                    if (TROP_IN(p - odd, 4, sp_in)) lo[u] = *reinterpret_cast<const uint32_t*>(p - odd);
                } else if (TROP_IN(p, 2, sp_in)) {
                    lo[u] = (uint32_t)*p << 16 * odd;
                }
                if (!odd) continue;
                if (p + 3 <= end) {
                    if (TROP_IN(p + 1, 4, sp_in)) hi[u] = *reinterpret_cast<const uint32_t*>(p + 1);
                } else if (p + 1 < end && TROP_IN(p + 1, 2, sp_in)) {
                    hi[u] = p[1];
                }
            }
#pragma unroll
            for (int u = 0; u < PACK_WORDS; ++u) {
                const int64_t w = at + 32 * u;
                if (w >= words) break;
                const uint32_t v = odd ? __funnelshift_r(lo[u], hi[u], 16) : lo[u];
                to[w] = 2 * w + 1 < cols ? v : v & 0xffffu;
            }
        }
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// from the driver, looked up once (the library does not link against libcuda); nullptr if it is not there
EncodeTiledFn encode_tiled()
{
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return (EncodeTiledFn)p;
    }();
    return fn;
}

template <typename F>
int encode_checked(F encode)
{
    CUresult r = encode();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {  // a host thread (autograd's, say) that has not touched the device yet
        int dev = 0;
        cudaGetDevice(&dev);
        cudaSetDevice(dev);
        r = encode();
    }
    if (r != CUDA_SUCCESS) return set_error(TROP_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return TROP_OK;
}

}  // namespace

int make_map(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_rows)
{
    const bool wide = type == TROP_F32;
    const EncodeTiledFn enc = encode_tiled();
    if (!enc) return set_error(TROP_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * (wide ? 4 : 2)};
    const cuuint32_t box[2] = {wide ? 32u : 64u, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode_checked([&] {
        return enc(map,
                   wide                ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                   : type == TROP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
}
int pack(Operand& x, Operand& w, const Workspace& ws, int sm)
{
    int64_t blocks = 0;
    for (Operand* o : {&x, &w})
        if (o->packed) {
            o->m.p = (const uint16_t*)(ws.base + o->at);
            blocks = std::max(blocks, (o->a.rows + 7) / 8);
        }
    if (blocks == 0) return TROP_OK;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)sm * 8), x.packed && w.packed ? 2 : 1);
    const cudaError_t e = launch_pdl(k_pack, grid, dim3(32, 8), 0, ws.s, (x.packed ? x : w).job(), w.job());
    if (e != cudaSuccess) return cuda_error(e, "k_pack launch");
    count_launches(1);
    return TROP_OK;
}

int pack(Operand& x, const Workspace& ws, int sm)
{
    if (!x.packed) return TROP_OK;
    x.m.p = (const uint16_t*)(ws.base + x.at);
    const dim3 grid((unsigned)std::min<int64_t>((x.a.rows + 7) / 8, (int64_t)sm * 8));
    const cudaError_t e = launch_pdl(k_pack, grid, dim3(32, 8), 0, ws.s, x.job(), x.job());
    if (e != cudaSuccess) return cuda_error(e, "k_pack launch");
    count_launches(1);
    return TROP_OK;
}

int splits(int tiles, int kt, int teams, int64_t bytes)
{
    int ks = 1;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= std::min(kt, 64); ++c) {
        const int per = cdiv(kt, c);
        if (cdiv(kt, per) != c) continue;
        if (c > 1 && c * bytes > (int64_t)1 << 30) break;
        const int64_t cost = (int64_t)cdiv((int64_t)tiles * c, teams) * (per + (c > 1 ? 8 : 0));
        if (cost < best) best = cost, ks = c;
    }
    return ks;
}

}  // namespace trop
