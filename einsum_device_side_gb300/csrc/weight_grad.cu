// weight_grad.cu -- the weight gradient of a linear layer whose input was kept in 8 bits (pack8.h).
//
//   dw[o, c] = sum_t dy[t, o] x[t, c],   x[t, c] = code[t, c] 2^(scale[t, c / 32] - 133) in dy's type,
//   db[o]    = sum_t dy[t, o]
// dy bf16 or f16, sums in f32, results in dy's type or f32, rounded once.  A code has seven bits and its scale is a power
// of two, so bf16 operands hold the values exactly (f16 where they lie in its range).
//
// The codes become operands in workspace, a piece of x's columns at a time (64 MiB, which is still in the L2 when the products
// read it; of more than 32768 tokens 1024 columns, 2048 bytes a token), by the kernel of activation.cu; the products are tiles of
// 256 x 256 of dw by pairs of CTAs, both operands token-major as they lie:
//   warp 0       loads: boxes of 64 tokens x 64 columns of dy and of x, by TMA into a ring of six stages
//   warp 1       products, one thread of the pair's first CTA
//   warps 4-11   results: tensor memory to dw, or to the f32 sums of a split of the tokens
// 8192^3 bf16: 640 us in short runs (1718 TFLOP/s), 714 to 754 under the power limit.
// (Codes that came by TMA and were made operands inside this kernel, by warps of their own: 8192^3 bf16 2034 us, in
// pieces 640 us.  The tensor cores' own reads take three quarters of the shared memory's rate, so that those warps' loads
// and stores waited 1200 cycles each; 64x16384x4096 to f32 55 us and 54 us.)
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#define TROP_TU 13  // this file's id in a bounds-violation record
#include "block.h"
#include "internal.h"
#include "operands.h"
#include "pack8.h"
#include "packed.h"
#include "tcgen05.h"

namespace trop {
namespace {

constexpr int TK = 64, TM = 256, TN = 256;
// Stages of one chain of accumulations of an f32 result.  A chain loses up to a last place every 16 tokens, 2.2e-10 to 4.3e-10 of its norm
// a token: 2.8e-6 over 8192, 7.0e-6 over 16384, where the plain f32 product is off by 3.1e-7 and 5.1e-7.  Chains of 2048 tokens that the
// copies to memory add up in f32 are off by 4.5e-7 over any number of tokens (8192^3 bf16 to f32 721 to 725 us, one chain 654).
constexpr int CHAIN = 2048 / TK;
constexpr int HALF_BYTES = 128 * TK * 2;  // a CTA's part of either operand in a stage
constexpr int STAGE_BYTES = 2 * HALF_BYTES, STAGES = 6;
constexpr int EPI_WARPS = 8, THREADS = 128 + 32 * EPI_WARPS;
constexpr int BOX_BYTES = 4096;
constexpr int SMEM = STAGES * STAGE_BYTES + EPI_WARPS * BOX_BYTES + 1024;

struct Job {
    int mt, nt, kt, kper, units;
    int chain;       // stages of one accumulation: a unit's chains are added up in memory
    int rows, cols;  // of dw
    void* out;       // null: f32 sums, through map_c
    int64_t ldo;
    int wide, vec;   // out is f32; its rows lie on 16 bytes: through map_c
    int pad_rows;    // rows of one split's sums
    uint32_t* error;
    Span sp_out;
};
struct Unit {
    int m, n, split, k0, k1;
};
__device__ __forceinline__ Unit unit_of(const Job& j, int u)
{
    Unit r;
    // rows of tiles fastest: the units that run together share their columns' codes
    r.m = u % j.mt;
    u /= j.mt;
    r.n = u % j.nt;
    r.split = u / j.nt;
    r.k0 = r.split * j.kper;
    r.k1 = min(j.kt, r.k0 + j.kper);
    return r;
}

template <bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    k_weight_grad(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_c, const __grid_constant__ Job j)
{
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], drain;
    __shared__ uint32_t tmem_slot;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t ring = (smem_u32(dyn) + 1023u) & ~1023u, boxes = ring + STAGES * STAGE_BYTES;
    const int first = blockIdx.x / 2, step = gridDim.x / 2;

    if (warp == 1 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
        for (int b = 0; b < 2; ++b) mbar_init(&tfull[b], 1), mbar_init(&tempty[b], EPI_WARPS * 2);
        mbar_init(&drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) tma_prefetch_map(&map_a), tma_prefetch_map(&map_b);
    if (warp == 2) tmem_alloc_all<2>(&tmem_slot);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {  // loads
            int s = 0;
            uint32_t phase = 0, issued = 0;
            for (int u = first; u < j.units && ok; u += step) {
                const Unit t = unit_of(j, u);
                const int am = t.m * TM + rank * 128, bn = t.n * TN + rank * 128;
                for (int k = t.k0; k < t.k1; ++k) {
                    if (!(ok = mbar_wait(&empty[s], phase ^ 1))) break;
                    if (rank == 0) mbar_expect_tx(&full[s], 2 * STAGE_BYTES);
                    const uint32_t bar = mapa(smem_u32(&full[s]), 0), to = ring + s * STAGE_BYTES;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        tma_load_2d<2>(to + c * 8192, &map_a, am + 64 * c, k * TK, bar);
                        tma_load_2d<2>(to + HALF_BYTES + c * 8192, &map_b, bn + 64 * c, k * TK, bar);
                    }
                    ++issued;
                    if (++s == STAGES) s = 0, phase ^= 1;
                }
            }
            if (!ok && rank == 0)  // no copy may land after the CTA has left
                for (uint32_t i = 0; i < min(issued, (uint32_t)STAGES); ++i) {
                    if (--s < 0) s = STAGES - 1, phase ^= 1;
                    (void)mbar_wait(&full[s], phase);
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {  // products
            constexpr uint32_t idesc = mma_desc(BF16, true, true, TM, TN);
            int s = 0;
            uint32_t phase = 0, tile = 0;
            for (int u = first; u < j.units && ok; u += step) {
                const Unit t = unit_of(j, u);
                for (int k0 = t.k0; k0 < t.k1 && ok; k0 += j.chain, ++tile) {
                    const uint32_t buf = tile & 1, acc = tmem + buf * TN;
                    if (!(ok = mbar_wait_cluster(&tempty[buf], ((tile >> 1) & 1) ^ 1))) break;
                    tc_fence_after();
                    const int k1 = min(t.k1, k0 + j.chain);
                    for (int k = k0; k < k1; ++k) {
                        if (!(ok = mbar_wait_cluster(&full[s], phase))) break;
                        tc_fence_after();
                        const uint32_t at = ring + s * STAGE_BYTES;
                        const uint64_t da = smem_desc(at, 8192), db = smem_desc(at + HALF_BYTES, 8192);
#pragma unroll
                        for (int i = 0; i < TK / 16; ++i) tc_mma<2>(acc, da + i * 128, db + i * 128, idesc, k > k0 || i > 0);
                        tc_commit<2>(&empty[s]);
                        if (++s == STAGES) s = 0, phase ^= 1;
                    }
                    if (ok) tc_commit<2>(&tfull[buf]);
                }
            }
            if (!ok) {  // no product may run after the CTA has left
                tc_commit<2>(&drain);
                (void)mbar_wait(&drain, 0);
            }
        }
    } else if (warp >= 4) {  // results
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t box = boxes + (warp - 4) * BOX_BYTES;
        uint32_t tile = 0;
        for (int u = first; u < j.units && ok; u += step) {
            const Unit t = unit_of(j, u);
            for (int k0 = t.k0; k0 < t.k1; k0 += j.chain, ++tile) {
                const uint32_t buf = tile & 1;
                ok = mbar_wait(&tfull[buf], (tile >> 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const bool add = k0 > t.k0;  // to the chains before, which are in memory by then: in their order
                if (add && lane == 0) tma_store_wait();
                __syncwarp();
                const uint32_t src = tmem + buf * TN + half * 128 + ((uint32_t)(quad * 32) << 16);
                const int row0 = t.m * TM + rank * 128 + quad * 32;
                uint32_t v[2][32];
                tmem_ld32(src, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_wait_ld(v[c & 1]);
                    if (c < 3) tmem_ld32(src + (c + 1) * 32, v[(c + 1) & 1]);
                    else {  // the accumulator is in registers: the next tile may fill it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(mapa(smem_u32(&tempty[buf]), 0));
                    }
                    const int col = t.n * TN + half * 128 + c * 32;
                    if (!j.out || j.wide) {  // f32: a box of 32 columns
                        box_free(lane);
                        to_box<32>(box, lane, 0, v[c & 1]);
                        if (!j.out)
                            store_box(&map_c, box, lane, col, t.split * j.pad_rows + row0, j.cols, t.split * j.pad_rows + j.rows, add);
                        else if (j.vec) store_box(&map_c, box, lane, col, row0, j.cols, j.rows, add);
                        else copy_box<float>(box, lane, col, row0, j.rows, j.cols, j.out, j.ldo, j.sp_out);  // (one chain)
                        continue;
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pack2<BF16>(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1]));
                    if (c % 2 == 0) box_free(lane);  // a box of 64 columns, in two halves
                    to_box<16>(box, lane, (c % 2) * 4, w);
                    if (c % 2 == 0) continue;
                    if (j.vec) store_box(&map_c, box, lane, col - 32, row0, j.cols, j.rows, false);
                    else copy_box<uint16_t>(box, lane, col - 32, row0, j.rows, j.cols, j.out, j.ldo, j.sp_out);
                }
            }
        }
        if (lane == 0) tma_store_wait();
    }
    if (!ok && lane == 0) {
        *(volatile uint32_t*)j.error = 1;
        __threadfence_system();
    }
    __syncwarp();
    pdl_signal();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 2) tmem_free_all<2>(tmem);
}

// The sums [ks][slab][lda], added in order, four columns of a row per thread where rows allow 16-byte loads.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_grad_join(const float* acc, int ks, int64_t slice, int64_t lda, int64_t rows, int64_t cols,
                                                   T* out, int64_t ldo, Span sp_acc, Span sp_out)
{
    pdl_wait();
    pdl_signal();
    constexpr int W = VEC ? 4 : 1;
    const int64_t n = rows * cols / W, per_row = cols / W;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / per_row, c = (i - r * per_row) * W;
        float s[W];
#pragma unroll
        for (int w = 0; w < W; ++w) s[w] = 0.f;
#pragma unroll 4
        for (int k = 0; k < ks; ++k) {
            const float* p = acc + k * slice + r * lda + c;
            Raw<float, W> q;
            if (!TROP_IN(p, 4 * W, sp_acc)) continue;
            q.read(p);
#pragma unroll
            for (int w = 0; w < W; ++w) s[w] += q.get(w);
        }
        Raw<T, W> q;
        q.set(s);
        if (TROP_IN(out + r * ldo + c, W * sizeof(T), sp_out)) q.write(out + r * ldo + c);
    }
}

// Columns of dy summed over rows blockIdx.y, + gridDim.y, ... by eight warps, whose sums are added in warp order: 256 columns a
// block (32 where rows do not lie on 16 bytes).  One block of rows writes db, several their sums.
template <typename T, int VEC, typename TO>
__global__ void __launch_bounds__(256) k_column_sums(const T* dy, int64_t sr, int64_t rows, int64_t cols, float* part, TO* out,
                                                     Span sp_dy, Span sp_part, Span sp_out)
{
    pdl_wait();
    pdl_signal();
    __shared__ float sh[8][32 * VEC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * VEC;
    float a[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = 0.f;
    const int64_t step = (int64_t)gridDim.y * 8;
    for (int64_t r = (int64_t)blockIdx.y * 8 + warp; r < rows; r += step * 4) {
        Raw<T, VEC> q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const T* p = dy + (r + u * step) * sr + c;
            q[u].zero();
            if (r + u * step < rows && c < cols && TROP_IN(p, VEC * sizeof(T), sp_dy)) q[u].read(p);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[i] += (q[0].get(i) + q[1].get(i)) + (q[2].get(i) + q[3].get(i));
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) sh[warp][lane * VEC + i] = a[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * VEC; i += 256) {
        const int64_t col = (int64_t)blockIdx.x * 32 * VEC + i;
        if (col >= cols) break;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += sh[w][i];
        if (part) {
            if (TROP_IN(part + blockIdx.y * cols + col, 4, sp_part)) part[blockIdx.y * cols + col] = v;
        } else if (TROP_IN(out + col, sizeof(TO), sp_out)) {
            out[col] = from_f32<TO>(v);
        }
    }
}

#define GRAD_LAUNCH(kernel, grid, block, ...)                                      \
    do {                                                                           \
        const cudaError_t e_ = launch_pdl(kernel, grid, block, 0, s, __VA_ARGS__); \
        if (e_ != cudaSuccess) return cuda_error(e_, #kernel " launch");           \
        count_launches(1);                                                         \
    } while (0)

template <typename T, typename TO>
int bias_sums(const Operand& o, TO* out, float* part, int parts, cudaStream_t s)
{
    const Matrix16& dy = o.m;  // (rows on 16 bytes)
    const int64_t size[2] = {dy.rows, o.packed ? dy.ld : dy.cols}, stride[2] = {dy.ld, 1};
    const Span sp = span_of(dy.p, 2, 2, size, stride), sp_out = span_bytes(out, dy.cols * sizeof(TO));
    const Span sp_part = span_bytes(part, (size_t)parts * dy.cols * 4);
    const bool vec = dy.cols % 8 == 0 || o.packed;  // (a packed copy's rows reach to the next vector's end)
    const auto kernel = vec ? k_column_sums<T, 8, TO> : k_column_sums<T, 1, TO>;
    GRAD_LAUNCH(kernel, dim3(cdiv(dy.cols, vec ? 256 : 32), parts), dim3(256), (const T*)dy.p, dy.ld, dy.rows, dy.cols,
                parts > 1 ? part : nullptr, out, sp, sp_part, sp_out);
    if (parts > 1)
        GRAD_LAUNCH((k_grad_join<TO, false>), dim3(cdiv(dy.cols, 256)), dim3(256), (const float*)part, parts, dy.cols, dy.cols, (int64_t)1,
                    dy.cols, out, dy.cols, sp_part, sp_out);
    return TROP_OK;
}
// Blocks of rows of the bias's sums: as many as fill the device twice, of 64 rows at least.
int bias_parts(const Mat16& dy, int sm)
{
    const int across = cdiv(dy.cols, 256);
    return (int)std::max<int64_t>(1, std::min<int64_t>(dy.rows / 64, 2 * sm / across));
}

// Splits' sums into columns c0 .. c0 + cols of dw.
template <typename TO>
int join(const float* acc, int ks, int64_t slab, int64_t lda, const WeightGrad& q, int64_t c0, int64_t cols, int sm, cudaStream_t s)
{
    const int64_t rows = q.dy.cols, size[2] = {rows, cols}, stride[2] = {q.ldw, 1};
    TO* const out = (TO*)q.dw + c0;
    const Span sp_out = span_of(out, sizeof(TO), 2, size, stride), sp_acc = span_bytes(acc, (size_t)ks * slab * lda * 4);
    const bool vec = cols % 4 == 0 && q.ldw % 4 == 0 && (uintptr_t)out % (4 * sizeof(TO)) == 0;
    const int grid = (int)std::min<int64_t>((rows * cols / (vec ? 4 : 1) + 255) / 256, (int64_t)sm * 8);
    const auto kernel = vec ? k_grad_join<TO, true> : k_grad_join<TO, false>;
    GRAD_LAUNCH(kernel, dim3(grid), dim3(256), acc, ks, slab * lda, lda, rows, cols, out, q.ldw, sp_acc, sp_out);
    return TROP_OK;
}

int launch(bool bf16, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const Job& j, int sm, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(j.units, sm / 2) * 2);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, k_weight_grad<true>, a, b, c, j)
                               : cudaLaunchKernelEx(&cfg, k_weight_grad<false>, a, b, c, j);
    if (e != cudaSuccess) return cuda_error(e, "k_weight_grad launch");
    count_launches(1);
    return TROP_OK;
}

}  // namespace

int register_weight_grad_kernels()
{
    constexpr cudaFuncAttribute most = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(k_weight_grad<true>, most, SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_weight_grad<false>, most, SMEM);
    return e == cudaSuccess ? (int)TROP_OK : cuda_error(e, "cudaFuncSetAttribute(k_weight_grad)");
}

int launch_weight_grad(const WeightGrad& q, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const int sm = dev->sm_count;
    const int64_t T = q.dy.rows, O = q.dy.cols, C = q.cols;
    const int type = q.bf16 ? TROP_BF16 : TROP_F16;
    Workspace ws(s);
    Operand dy(q.dy, ws);
    // a piece of x's columns: whole tiles, 64 MiB of values, but 1024 columns at least
    const int64_t whole = (C + TN - 1) / TN * TN;
    const int64_t piece = std::min(whole, std::max<int64_t>((32 << 20) / T / TN * TN, 1024));
    const int64_t ldx = (std::min(piece, C) + 7) / 8 * 8;
    const size_t at_x = ws.add((size_t)T * ldx * 2);
    const int mt = cdiv(O, TM), kt = cdiv(T, TK);
    const int ks = C == 0 ? 1 : splits(mt * cdiv(std::min(piece, C), TN), kt, sm / 2, O * std::min(piece, C) * 4);
    const int64_t lda = (std::min(piece, C) + 3) / 4 * 4, pad_rows = (O + 31) / 32 * 32;
    const size_t elem = q.wide ? 4 : 2;
    // (pieces start on whole tiles)
    const bool vec = (uintptr_t)q.dw % 16 == 0 && q.ldw * elem % 16 == 0 && q.ldw >= C && q.ldw < (int64_t)1 << 37;
    // sums in workspace: of splits, and of chains where the result's rows take no copies (8192x4864x2047 bf16 to f32 160 us; added by
    // loads and stores there 308)
    const bool sums = ks > 1 || (q.wide && !vec && kt > CHAIN);
    const size_t at_acc = sums ? ws.add((size_t)ks * pad_rows * lda * 4) : 0;
    const int parts = q.db ? bias_parts(q.dy, sm) : 1;
    const size_t at_part = parts > 1 ? ws.add((size_t)parts * O * 4) : 0;
    if (ws.bytes) TROP_TRY(ws.take());
    TROP_TRY(pack(dy, ws, sm));
    if (q.db) {
        float* part = parts > 1 ? (float*)(ws.base + at_part) : nullptr;
        if (q.bf16)
            TROP_TRY(q.wide ? (bias_sums<__nv_bfloat16, float>(dy, (float*)q.db, part, parts, s))
                            : (bias_sums<__nv_bfloat16, __nv_bfloat16>(dy, (__nv_bfloat16*)q.db, part, parts, s)));
        else
            TROP_TRY(q.wide ? (bias_sums<__half, float>(dy, (float*)q.db, part, parts, s))
                            : (bias_sums<__half, __half>(dy, (__half*)q.db, part, parts, s)));
    }
    void* const x = ws.base + at_x;
    float* const acc = (float*)(ws.base + at_acc);
    for (int64_t c0 = 0; c0 < C; c0 += piece) {
        const int64_t cols = std::min(piece, C - c0);
        TROP_TRY(launch_activation_values(T, cols, {q.x.codes + c0, q.x.sc, q.x.scales + c0 / GROUP8, q.x.ss}, {x, ldx, type}, s));
        Job j = {};
        TROP_TRY(device_error_word(&j.error));
        j.rows = (int)O;
        j.cols = (int)cols;
        j.mt = mt;
        j.nt = cdiv(cols, TN);
        j.kt = kt;
        j.kper = cdiv(kt, ks);
        j.units = j.mt * j.nt * ks;
        j.chain = q.wide ? CHAIN : kt;
        j.wide = q.wide;
        CUtensorMap a, b, c;
        TROP_TRY(make_map(&a, type, dy.m.p, O, T, dy.m.ld, TK));
        TROP_TRY(make_map(&b, type, x, cols, T, ldx, TK));
        c = a;
        if (sums) {
            j.pad_rows = (int)pad_rows;
            TROP_TRY(make_map(&c, TROP_F32, acc, cols, ks * pad_rows, lda, 32));
        } else {
            const int64_t size[2] = {O, cols}, stride[2] = {q.ldw, 1};
            j.out = (char*)q.dw + c0 * elem;
            j.ldo = q.ldw;
            j.vec = vec;
            j.sp_out = span_of(j.out, elem, 2, size, stride);
            if (j.vec) TROP_TRY(make_map(&c, q.wide ? (int)TROP_F32 : type, j.out, cols, O, q.ldw, 32));
        }
        TROP_TRY(launch(q.bf16, a, b, c, j, sm, s));
        if (sums)
            TROP_TRY(q.wide   ? join<float>(acc, ks, pad_rows, lda, q, c0, cols, sm, s)
                     : q.bf16 ? join<__nv_bfloat16>(acc, ks, pad_rows, lda, q, c0, cols, sm, s)
                              : join<__half>(acc, ks, pad_rows, lda, q, c0, cols, sm, s));
    }
    return TROP_OK;
}

}  // namespace trop
