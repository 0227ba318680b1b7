// activation.cu -- activations in 8 bits (the format: pack8.h), written and read back.
//
// Both directions are bound by memory: a 16-bit element is 2 bytes one way and 1 + 1/32 the other.  A thread has the
// elements of 16 bytes, 32 / that many neighbouring lanes a group, whose largest magnitude they find by shuffles; U rows'
// loads are on their way together.  Matrices without gaps are taken as one row.
// Rows that do not lie on 16 bytes keep whole vectors all the same: two aligned loads are shifted together (pack), or
// the vectors are laid where the result's are aligned and the codes shifted (values).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#define TROP_TU 11  // this file's id in a bounds-violation record
#include "block.h"
#include "pack8.h"
#include "rows.h"

namespace trop {
namespace {

struct Job8 {
    int64_t rows, cols;
    const void* x;  // pack: the elements; values: the result
    int64_t sx;
    int8_t* codes;
    int64_t sc;
    uint8_t* scales;
    int64_t ss;
    int wide_codes;  // rows of codes start on a vector's bytes
    Span sp_x, sp_c, sp_s;
};

// VEC elements from any element on, where the aligned 32 bytes around them lie in the matrix; else one by one.  Elements from
// `left` on are zero.
template <typename T, int VEC>
__device__ __forceinline__ void read_any(const T* p, int left, const T* begin, const T* end, Raw<T, VEC>& q, const Span& sp)
{
    (void)sp;
    const uint32_t off = (uint32_t)((uintptr_t)p & 15);
    const char* const at = reinterpret_cast<const char*>(p) - off;
    if (at >= reinterpret_cast<const char*>(begin) && at + (off ? 32 : 16) <= reinterpret_cast<const char*>(end)) {
        uint32_t w[8];
        const bool in = TROP_IN(at, off ? 32 : 16, sp);
        const uint4 a = in ? reinterpret_cast<const uint4*>(at)[0] : make_uint4(0, 0, 0, 0);
        const uint4 b = in && off ? reinterpret_cast<const uint4*>(at)[1] : make_uint4(0, 0, 0, 0);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        if (off & 8)
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        if (off & 4)
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) q.w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
        if (left < VEC)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr int E = 4 / sizeof(T);
                if (i * E >= left) q.w[i] = 0;
                else if (E == 2 && i * E + 1 >= left) q.w[i] &= 0xffffu;
            }
    } else {
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = i < left && TROP_IN(p + i, sizeof(T), sp) ? to_f32(p[i]) : 0.f;
        q.set(v);
    }
}

template <typename T, bool OFF, int U>
__global__ void __launch_bounds__(256, 4) k_pack8(const Job8 j)
{
    pdl_wait();
    pdl_signal();
    constexpr int VEC = 16 / sizeof(T);
    const int c = (int)(blockIdx.x * blockDim.x + threadIdx.x) * VEC, cols = (int)j.cols;
    const T* const begin = (const T*)j.x;
    const T* const end = begin + (j.rows - 1) * j.sx + j.cols;
    const int64_t step = (int64_t)gridDim.y * blockDim.y;
    for (int64_t row0 = (int64_t)blockIdx.y * blockDim.y; row0 < j.rows; row0 += step * U) {
        Raw<T, VEC> q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step + threadIdx.y;
            const bool live = row < j.rows && c < cols;
            const T* p = begin + row * j.sx + c;
            q[u].zero();
            if (OFF) {
                if (live) read_any<T, VEC>(p, cols - c, begin, end, q[u], j.sp_x);
            } else if (live && TROP_IN(p, 16, j.sp_x)) {
                q[u].read(p);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step + threadIdx.y;
            const bool live = row < j.rows && c < cols;
            const uint32_t e = scale8(group_top8<VEC>(top8<T, VEC>(q[u])));
            if (!live) continue;
            Codes<VEC> k;
            codes8<T, VEC>(q[u], e, k.w);
            int8_t* to = j.codes + row * j.sc + c;
            if (!OFF || (j.wide_codes && c + VEC <= cols)) {
                if (TROP_IN(to, VEC, j.sp_c)) k.write(to);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i < cols && TROP_IN(to + i, 1, j.sp_c)) to[i] = (int8_t)(k.w[i / 4] >> 8 * (i % 4));
            }
            uint8_t* s = j.scales + row * j.ss + c / GROUP8;
            if (c % GROUP8 == 0 && TROP_IN(s, 1, j.sp_s)) *s = (uint8_t)e;
        }
    }
}

// (Registers are held down to where the loads of several rows from many warps are on their way: ragged rows at 193 registers
// a thread and with both edges of every row one by one took 232 us for 40950x1001 f16.)
template <typename T, bool OFF, int U>
__global__ void __launch_bounds__(256, 4) k_values8(const Job8 j)
{
    pdl_wait();
    pdl_signal();
    constexpr int VEC = 16 / sizeof(T);
    const int vec = blockIdx.x * blockDim.x + threadIdx.x, cols = (int)j.cols;
    const int64_t step = (int64_t)gridDim.y * blockDim.y;
    const int8_t* const end = j.codes + (j.rows - 1) * j.sc + j.cols;
    // the first column of the thread's vector of a row: where the result's vectors lie on 16 bytes
    auto column = [&](const T* out) { return vec * VEC - (OFF ? (int)((uint32_t)(uintptr_t)out & 15) / (int)sizeof(T) : 0); };
    for (int64_t row0 = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; row0 < j.rows; row0 += step * U) {
        Codes<VEC> q[U];
        uint32_t s0[U], s1[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            const int c = column((const T*)j.x + row * j.sx);
            const int8_t* p = j.codes + row * j.sc + c;
            const uint8_t* s = j.scales + row * j.ss;
            s0[u] = s1[u] = LEAST8;
            if (row < j.rows && c < cols) {
                const int g0 = max(c, 0) / GROUP8, g1 = min(c + VEC - 1, cols - 1) / GROUP8;
                if (TROP_IN(s + g0, 1, j.sp_s)) s0[u] = s[g0];
                if (OFF && TROP_IN(s + g1, 1, j.sp_s)) s1[u] = s[g1];
                if (OFF) codes_any<VEC>(p, -c, cols - c, j.codes, end, q[u], j.sp_c);
                else if (TROP_IN(p, VEC, j.sp_c)) q[u].read(p);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            T* const out = (T*)j.x + row * j.sx;
            const int c = column(out);
            if (row >= j.rows || c >= cols) continue;
            float v[VEC];
            const float unit = unit8(s0[u]);
            if (OFF) {
                const float other = unit8(s1[u]);
                const int edge = max(c, 0) / GROUP8 * GROUP8 + GROUP8 - c;  // elements up to the first group's end
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = coded8(q[u].w[i / 4] ^ 0x80808080u, i % 4) * (i < edge ? unit : other);
            } else {
                values8<VEC>(q[u].w, unit, v);
            }
            if (!OFF || (c >= 0 && c + VEC <= cols)) {
                store<T, VEC>(out + c, v, j.sp_x);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (c + i >= 0 && c + i < cols && TROP_IN(out + c + i, sizeof(T), j.sp_x)) out[c + i] = from_f32<T>(v[i]);
            }
        }
    }
}

// Matrices without gaps, in whole groups: U vectors of a thread, a block's width apart.
template <typename T, int U>
__global__ void __launch_bounds__(256) k_pack8_flat(const T* x, int8_t* codes, uint8_t* scales, int64_t vecs, Span sp_x, Span sp_c,
                                                    Span sp_s)
{
    pdl_wait();
    pdl_signal();
    constexpr int VEC = 16 / sizeof(T);
    const int64_t first = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
    Raw<T, VEC> q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256;
        q[u].zero();
        if (i < vecs && TROP_IN(x + i * VEC, 16, sp_x)) q[u].read(x + i * VEC);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256;
        const uint32_t e = scale8(group_top8<VEC>(top8<T, VEC>(q[u])));
        Codes<VEC> k;
        codes8<T, VEC>(q[u], e, k.w);
        if (i >= vecs) break;
        if (TROP_IN(codes + i * VEC, VEC, sp_c)) k.write(codes + i * VEC);
        if (i % (GROUP8 / VEC) == 0 && TROP_IN(scales + i / (GROUP8 / VEC), 1, sp_s)) scales[i / (GROUP8 / VEC)] = (uint8_t)e;
    }
}
template <typename T, int U>
__global__ void __launch_bounds__(256) k_values8_flat(const int8_t* codes, const uint8_t* scales, T* x, int64_t vecs, Span sp_c, Span sp_s,
                                                      Span sp_x)
{
    pdl_wait();
    pdl_signal();
    constexpr int VEC = 16 / sizeof(T);
    const int64_t first = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
    Codes<VEC> q[U];
    uint32_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256;
        q[u].zero();
        e[u] = LEAST8;
        if (i < vecs && TROP_IN(codes + i * VEC, VEC, sp_c)) q[u].read(codes + i * VEC);
        if (i < vecs && TROP_IN(scales + i / (GROUP8 / VEC), 1, sp_s)) e[u] = scales[i / (GROUP8 / VEC)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256;
        if (i >= vecs) break;
        float v[VEC];
        values8<VEC>(q[u].w, unit8(e[u]), v);
        store<T, VEC>(x + i * VEC, v, sp_x);
    }
}

// Results without gaps between ragged rows: aligned vectors of the whole result, `lead` elements before its first on.  One that
// goes over a row's end takes its codes from both rows.  The row is a product with 2^(31 + s) / cols rounded up, s the bits of
// cols - 1, exact below 2^31 (Granlund and Montgomery, "Division by invariant integers using multiplication", 1994).
// 40950x1001 f16 38 us with one vector a thread, 40 us with two; by rows, of which the first and the last vector are stored
// element by element, 46 us (300000x33 bf16 12 us against 27).
struct Flat8 {
    uint32_t n, vecs, magic, shift, sc, ss;  // elements, vectors; strides of codes and scales
    int lead;
};
template <typename T, int U>
__global__ void __launch_bounds__(256, 4) k_values8_ragged(const Job8 j, const Flat8 f)
{
    pdl_wait();
    pdl_signal();
    constexpr int VEC = 16 / sizeof(T);
    const int cols = (int)j.cols;
    const int8_t* const end = j.codes + (j.rows - 1) * j.sc + j.cols;
    Codes<VEC> q[U];
    uint32_t s0[U], s1[U], s2[U];  // the scales of the row's first and last element here, and of the next row's
    int col[U];
    const uint32_t first = blockIdx.x * (256 * U) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = first + u * 256;
        const int64_t f0 = (int64_t)i * VEC - f.lead;
        s0[u] = s1[u] = s2[u] = LEAST8;
        q[u].zero();
        col[u] = 0;
        if (i >= f.vecs) continue;
        const uint32_t row = f0 < 0 ? 0 : __umulhi((uint32_t)f0, f.magic) >> f.shift;
        const int c = (int)(f0 - (int64_t)((uint64_t)row * (uint32_t)cols)), left = cols - c;
        col[u] = c;
        const int8_t* p = j.codes + (uint64_t)row * f.sc + c;
        const uint8_t* s = j.scales + (uint64_t)row * f.ss;
        const int g0 = max(c, 0) / GROUP8, g1 = (min(left, VEC) + c - 1) / GROUP8;
        if (TROP_IN(s + g0, 1, j.sp_s)) s0[u] = s[g0];
        if (TROP_IN(s + g1, 1, j.sp_s)) s1[u] = s[g1];
        codes_any<VEC>(p, -c, left, j.codes, end, q[u], j.sp_c);
        if (left < VEC && row + 1 < (uint32_t)j.rows) {
            Codes<VEC> next;
            codes_any<VEC>(j.codes + (uint64_t)(row + 1) * f.sc - left, left, VEC, j.codes, end, next, j.sp_c);
            if (TROP_IN(s + f.ss, 1, j.sp_s)) s2[u] = s[f.ss];
#pragma unroll
            for (int w = 0; w < VEC / 4; ++w) {
                const int n = min(max(left - 4 * w, 0), 4);  // bytes of this row
                const uint32_t mask = n == 4 ? 0xffffffffu : (1u << 8 * n) - 1;
                q[u].w[w] = (q[u].w[w] & mask) | (next.w[w] & ~mask);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = first + u * 256;
        if (i >= f.vecs) break;
        const int64_t f0 = (int64_t)i * VEC - f.lead;
        T* const out = (T*)j.x + f0;
        const int c = col[u], left = cols - c, edge = max(c, 0) / GROUP8 * GROUP8 + GROUP8 - c;  // up to the row's end, to the first group's
        const float a = unit8(s0[u]), b = unit8(s1[u]), d = unit8(s2[u]);
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = coded8(q[u].w[e / 4] ^ 0x80808080u, e % 4) * (e >= left ? d : e < edge ? a : b);
        if (f0 >= 0 && f0 + VEC <= f.n) {
            store<T, VEC>(out, v, j.sp_x);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (f0 + e >= 0 && f0 + e < f.n && TROP_IN(out + e, sizeof(T), j.sp_x)) out[e] = from_f32<T>(v[e]);
        }
    }
}

// The threads of a row and of several rows in a block of 256, and the grid: as many rows at a time as fill the device
// with U each.
struct Shape8 {
    dim3 grid, block;
};
Shape8 shape8(int64_t rows, int64_t vecs, int lanes, int u, int sm)
{
    int64_t bx = lanes;
    while (bx < 256 && bx < vecs) bx *= 2;
    const int64_t by = 256 / bx, gx = (vecs + bx - 1) / bx;
    const int64_t most = std::max<int64_t>(1, (int64_t)sm * 16 / gx);
    int64_t gy = (rows + by - 1) / by;
    if (gy > most) gy = std::max<int64_t>(most, 1);
    else if (gy * gx > (int64_t)sm * 8) gy = std::max<int64_t>((gy + u - 1) / u, 1);
    return {dim3((unsigned)gx, (unsigned)std::min<int64_t>(gy, 65535)), dim3((unsigned)bx, (unsigned)by)};
}

template <typename T, bool PACK>
int run8(Job8 j, int sm, cudaStream_t s)
{
    constexpr int VEC = 16 / sizeof(T), U = 4;  // (rows off 16 bytes: 2)
    const bool on16 = j.cols % VEC == 0 && aligned(j.x, j.sx, sizeof(T), VEC, j.rows);
    j.wide_codes = aligned(j.codes, j.sc, 1, VEC, j.rows);
    const bool off = !on16 || !j.wide_codes;
    const int64_t groups = (j.cols + GROUP8 - 1) / GROUP8;
    if (!off && j.cols % GROUP8 == 0 && (j.rows == 1 || (j.sx == j.cols && j.sc == j.cols && j.ss == groups))) {
        const int64_t vecs = j.rows * groups * (GROUP8 / VEC), blocks = (vecs + 256 * U - 1) / (256 * U);
        if (blocks <= INT32_MAX) {
            const dim3 grid((unsigned)blocks), block(256);
            if constexpr (PACK)
                TROP_LAUNCH((k_pack8_flat<T, U>), grid, block, 0, (const T*)j.x, j.codes, j.scales, vecs, j.sp_x, j.sp_c, j.sp_s);
            else
                TROP_LAUNCH((k_values8_flat<T, U>), grid, block, 0, (const int8_t*)j.codes, (const uint8_t*)j.scales, (T*)j.x, vecs, j.sp_c,
                            j.sp_s, j.sp_x);
            return TROP_OK;
        }
    }
    if constexpr (!PACK) {
        const int64_t n = j.rows * j.cols;
        if (off && j.rows > 1 && j.sx == j.cols && j.cols >= 2 * VEC && n < INT32_MAX && j.sc >> 32 == 0 && j.ss >> 32 == 0) {
            const int lead = (int)((uintptr_t)j.x % 16 / sizeof(T));
            uint32_t bits = 0;
            while (((int64_t)1 << bits) < j.cols) ++bits;
            const Flat8 f = {(uint32_t)n, (uint32_t)((n + lead + VEC - 1) / VEC), (uint32_t)((((uint64_t)1 << (31 + bits)) / j.cols) + 1),
                             bits - 1, (uint32_t)j.sc, (uint32_t)j.ss, lead};
            TROP_LAUNCH((k_values8_ragged<T, 1>), dim3((f.vecs + 255) / 256), dim3(256), 0, j, f);
            return TROP_OK;
        }
    }
    const int64_t vecs = (j.cols + VEC - 1) / VEC + (off && !PACK ? 1 : 0);
    const Shape8 h = shape8(j.rows, vecs, GROUP8 / VEC, U, sm);
    if constexpr (PACK) {
        if (off) TROP_LAUNCH((k_pack8<T, true, 2>), h.grid, h.block, 0, j);
        else TROP_LAUNCH((k_pack8<T, false, U>), h.grid, h.block, 0, j);
    } else {
        if (off) TROP_LAUNCH((k_values8<T, true, 2>), h.grid, h.block, 0, j);
        else TROP_LAUNCH((k_values8<T, false, U>), h.grid, h.block, 0, j);
    }
    return TROP_OK;
}

Job8 job8(int64_t rows, int64_t cols, const void* x, int64_t sx, int dtype, const Kept8& k)
{
    Job8 j = {};
    j.rows = rows;
    j.cols = cols;
    j.x = x;
    j.sx = sx;
    j.codes = k.codes;
    j.sc = k.sc;
    j.scales = k.scales;
    j.ss = k.ss;
    const int64_t groups = (cols + GROUP8 - 1) / GROUP8;
    const int64_t size[2] = {rows, cols}, stride[2] = {sx, 1}, cstride[2] = {k.sc, 1}, gsize[2] = {rows, groups}, gstride[2] = {k.ss, 1};
    j.sp_x = span_of(x, model_bytes(dtype), 2, size, stride);
    j.sp_c = span_of(k.codes, 1, 2, size, cstride);
    j.sp_s = span_of(k.scales, 1, 2, gsize, gstride);
    return j;
}

}  // namespace

int launch_activation_pack(int64_t rows, int64_t cols, const NormMat& x, const Kept8& k, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const Job8 j = job8(rows, cols, x.p, x.sr, x.dtype, k);
    return x.dtype == TROP_F32    ? run8<float, true>(j, dev->sm_count, s)
           : x.dtype == TROP_BF16 ? run8<__nv_bfloat16, true>(j, dev->sm_count, s)
                                  : run8<__half, true>(j, dev->sm_count, s);
}
int launch_activation_values(int64_t rows, int64_t cols, const Kept8& k, const NormMat& x, cudaStream_t s)
{
    const DeviceInfo* dev;
    TROP_TRY(ensure_device(&dev));
    const Job8 j = job8(rows, cols, x.p, x.sr, x.dtype, k);
    return x.dtype == TROP_F32    ? run8<float, false>(j, dev->sm_count, s)
           : x.dtype == TROP_BF16 ? run8<__nv_bfloat16, false>(j, dev->sm_count, s)
                                  : run8<__half, false>(j, dev->sm_count, s);
}

}  // namespace trop
