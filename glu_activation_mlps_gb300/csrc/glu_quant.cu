// Quantisation to e4m3 with a scale for each block of 128 (glu_quant.cuh),
// alone and fused with the residual add + RMSNorm before it:
//
//     glu_quantize        q, scale of x by rows (1 x 128) or blocks (128 x 128)
//     glu_add_rmsnorm_q   s = x + residual, h = round(s),
//                         y = s / sqrt(mean(s^2) + eps) * gamma,  q, scale of y by rows
//
// Both are bound by HBM: a value is read once and written once.  A thread owns
// pieces of 32 bytes of a row (V = 16 values of a 16-bit type, 8 of f32; 16
// bytes where the rows are only 16-byte multiples), so a block of 128 columns is
// 128 / V neighbouring lanes of one warp and its largest magnitude a few
// shuffles; the values stay in registers between the load and the store.  Other
// rows take the same code with V = 4 values at stride 32 (element accesses,
// coalesced), a block being one warp.
// y is quantised from fp32: it is never rounded to the input's type.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "glu.h"
#include "glu_internal.h"
#include "glu_kernels.cuh"
#include "glu_quant.cuh"

namespace glu {
namespace quant {

// How a thread's V values of one 128-column block lie in a row: VB contiguous
// bytes in one access (32 or 16), or (VB = 0) at stride 32 with element accesses.
template <class T, int VB>
struct Lanes {
    static constexpr bool VEC = VB > 0;
    static constexpr int V = VEC ? VB / int(sizeof(T)) : 4;
    static constexpr int kWords = VEC ? VB / 4 : V;
    static constexpr int kPer = kBlock / V;         // lanes that share a block
    using C = Codec<T>;
    // first column of the piece number `piece` (counted over the row)
    __device__ __forceinline__ static int col(int piece)
    {
        return VEC ? piece * V : (piece / 32) * kBlock + piece % 32;
    }
    struct Raw {
        uint32_t w[kWords];
    };
    // Values past the row are zeros (single elements past it read column 0).
    __device__ __forceinline__ static Raw load(const char *row, int col, int H)
    {
        Raw r;
        if constexpr (VEC) {
            if (col < H) {
                Access<VB>::load(row + int64_t(col) * sizeof(T), r.w);
            } else {
#pragma unroll
                for (int j = 0; j < kWords; ++j) r.w[j] = 0;    // zeros in every type
            }
        } else {
            if (whole(col, H)) {
                const char *p = row + int64_t(col) * sizeof(T);
#pragma unroll
                for (int i = 0; i < V; ++i) r.w[i] = bits(p + 32 * i * sizeof(T));
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const bool in = col + 32 * i < H;
                    const uint32_t w = bits(row + int64_t(in ? col + 32 * i : 0) * sizeof(T));
                    r.w[i] = in ? w : 0u;
                }
            }
        }
        return r;
    }
    // Single elements: whether this warp's block of 128 columns lies inside the
    // row (the usual case needs no test and one address for each piece) ...
    __device__ __forceinline__ static bool whole(int col, int H) { return (col | (kBlock - 1)) < H; }
    // ... and an element's bits, left to be converted where they are used (a
    // conversion here would wait for the load).
    __device__ __forceinline__ static uint32_t bits(const char *p)
    {
        uint32_t v;
        if constexpr (sizeof(T) == 2)
            asm volatile("ld.global.u16 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        else
            asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        return v;
    }
    __device__ __forceinline__ static float get(const Raw &r, int i)
    {
        if constexpr (VEC)
            return C::get(r.w[i / C::kPerWord], i % C::kPerWord);
        else
            return C::get(r.w[i], 0);
    }
    __device__ __forceinline__ static void store(char *row, int col, int H, const float (&f)[V])
    {
        if constexpr (VEC) {
            if (col < H) {
                uint32_t w[kWords];
#pragma unroll
                for (int j = 0; j < kWords; ++j) w[j] = C::put(f + j * C::kPerWord);
                Access<VB>::store(row + int64_t(col) * sizeof(T), w);
            }
        } else {
            char *p = row + int64_t(col) * sizeof(T);
            const bool all = whole(col, H);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (all || col + 32 * i < H) C::store1(p + 32 * i * sizeof(T), f[i]);
        }
    }
    // V e4m3 values of one row
    __device__ __forceinline__ static void store_q(char *row, int col, int H, const float (&f)[V])
    {
        if constexpr (VEC) {
            if (col < H) {
                if constexpr (V == 16) {
                    const uint32_t w[4] = {pack4(f[0], f[1], f[2], f[3]), pack4(f[4], f[5], f[6], f[7]),
                                           pack4(f[8], f[9], f[10], f[11]), pack4(f[12], f[13], f[14], f[15])};
                    Access<16>::store(row + col, w);
                } else if constexpr (V == 8)
                    asm volatile("st.global.L1::no_allocate.v2.b32 [%0], {%1, %2};" ::"l"(row + col),
                                 "r"(pack4(f[0], f[1], f[2], f[3])), "r"(pack4(f[4], f[5], f[6], f[7]))
                                 : "memory");
                else
                    asm volatile("st.global.L1::no_allocate.b32 [%0], %1;" ::"l"(row + col),
                                 "r"(pack4(f[0], f[1], f[2], f[3]))
                                 : "memory");
            }
        } else {
            const uint32_t w = pack4(f[0], f[1], f[2], f[3]);
            char *p = row + col;
            const bool all = whole(col, H);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (all || col + 32 * i < H) p[32 * i] = char((w >> (8 * i)) & 0xFFu);
        }
    }
    __device__ __forceinline__ static float block_max(float v)
    {
#pragma unroll
        for (int o = kPer / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
        return v;
    }
};

__device__ __forceinline__ float sum32(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ---------------------------------------------------------------- add + RMSNorm

struct NormParams {
    const char *x, *res, *gamma;
    char *h, *q;
    float *scale, *rstd;
    int64_t sx, sr, sh, sq;     // row strides in bytes
    int64_t ss;                 // scale's row stride in floats
    int64_t rows;
    int H;
    int tpr;                    // threads per row, a multiple of 32; the block holds blockDim.x / tpr rows
    float eps;
};

// One row per team of tpr threads, NV pieces per thread, its values kept in
// fp32 registers between the sum of squares and the quantisation: x and the
// residual are read once, h, q and the scales written once.  The sum of squares
// is formed with fused multiply-adds in two chains per thread, then over the
// warp by shuffles and over the row's warps through shared memory.
template <class T, int NV, int VB>
__global__ void __launch_bounds__(512) add_rmsnorm_q_kernel(const NormParams p)
{
    using L = Lanes<T, VB>;
    constexpr int V = L::V;
    __shared__ float red[16];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int team = threadIdx.x / p.tpr, t = threadIdx.x - team * p.tpr;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x / p.tpr) + team;
    const bool on = row < p.rows;               // whole teams, so whole warps
    const int H = on ? p.H : 0;                 // a team without a row stores nothing (and loads row 0's first column)
    const char *xr = p.x + (on ? row : 0) * p.sx, *rr = p.res + (on ? row : 0) * p.sr;
    // four pieces' loads at once; gamma is on its way during the reduction where
    // registers allow
    constexpr int CK = NV < 4 ? NV : 4;
    constexpr bool kEarlyGamma = NV <= 4;
    float s[NV][V], ss[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k0 = 0; k0 < NV; k0 += CK) {
        typename L::Raw a[CK], b[CK];
#pragma unroll
        for (int k = 0; k < CK; ++k) {
            const int c = L::col(t + (k0 + k) * p.tpr);
            a[k] = L::load(xr, c, H);
            b[k] = L::load(rr, c, H);
        }
#pragma unroll
        for (int k = 0; k < CK; ++k) {
            float(&v)[V] = s[k0 + k];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = L::get(a[k], i) + L::get(b[k], i);
                ss[i & 1] = fmaf(v[i], v[i], ss[i & 1]);
            }
            L::store(p.h + row * p.sh, L::col(t + (k0 + k) * p.tpr), H, v);
        }
    }
    typename L::Raw g[kEarlyGamma ? NV : 1];
    if constexpr (kEarlyGamma) {
#pragma unroll
        for (int k = 0; k < NV; ++k) g[k] = L::load(p.gamma, L::col(t + k * p.tpr), H);
    }
    float total = sum32(ss[0] + ss[1]);
    if (p.tpr > 32) {
        const int lane = threadIdx.x & 31, nw = p.tpr >> 5;
        if (lane == 0) red[threadIdx.x >> 5] = total;
        __syncthreads();
        total = sum32(lane < nw ? red[team * nw + lane] : 0.0f);
    }
    const float rstd = 1.0f / sqrtf(total / float(p.H) + p.eps);
    if (on && t == 0 && p.rstd) p.rstd[row] = rstd;
    // y / scale = s gamma 448 / max |s gamma|: rstd cancels, and with it a
    // rounding of every value, and goes into the scale alone; where it is far
    // from 1 it stays with the values, whose products with gamma might leave the
    // range of floats without it (near 1, |s| < 2^18, so gamma may reach 2^100).
    const bool near1 = rstd > 0.0009765625f && rstd < 1024.0f;
    const float pre = near1 ? 1.0f : rstd, post = near1 ? rstd : 1.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int piece = t + k * p.tpr, c = L::col(piece);
        float m = 0.0f;
        if constexpr (!kEarlyGamma) g[0] = L::load(p.gamma, c, H);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[k][i] = s[k][i] * pre * L::get(g[kEarlyGamma ? k : 0], i);
            m = fmaxf(m, fabsf(s[k][i]));
        }
        // (next to nothing, the scale's floor needs the largest y itself)
        m = L::block_max(m);
        const bool tiny = m < kAmaxFloor || m * post < kAmaxFloor;
        const Divider d(tiny ? m * post : m);
        const float f = tiny ? d.factor() * post : d.factor();
#pragma unroll
        for (int i = 0; i < V; ++i) s[k][i] *= f;
        L::store_q(p.q + row * p.sq, c, H, s[k]);
        if (piece % L::kPer == 0 && c < H) p.scale[row * p.ss + piece / L::kPer] = tiny ? d.scale() : d.scale() * post;
    }
}

// ---------------------------------------------------------------- quantisation

struct QuantParams {
    const char *x;
    char *q;
    float *scale;
    int64_t sx, sq;             // row strides in bytes
    int64_t ss;                 // scale's row stride in floats
    int64_t rows;
    int H;
    int tpr;                    // rows form: threads per row (the block holds blockDim.x / tpr rows)
};

// By rows: a team of tpr threads (a multiple of 32) takes NV pieces each of one
// row; blockIdx.y and .z count stretches of NV * tpr pieces along wide rows.
template <class T, int NV, int VB>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantParams p)
{
    using L = Lanes<T, VB>;
    constexpr int V = L::V;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int team = threadIdx.x / p.tpr, t = threadIdx.x - team * p.tpr;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x / p.tpr) + team;
    if (row >= p.rows) return;                  // whole teams, so whole warps
    const int first = int(blockIdx.z * gridDim.y + blockIdx.y) * p.tpr * NV + t;
    const char *xr = p.x + row * p.sx;
    typename L::Raw a[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) a[k] = L::load(xr, L::col(first + k * p.tpr), p.H);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int piece = first + k * p.tpr, c = L::col(piece);
        float f[V], m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = L::get(a[k], i);
            m = fmaxf(m, fabsf(f[i]));
        }
        const Divider d(L::block_max(m));
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = d(f[i]);
        L::store_q(p.q + row * p.sq, c, p.H, f);
        if (piece % L::kPer == 0 && c < p.H) p.scale[row * p.ss + piece / L::kPer] = d.scale();
    }
}

// By blocks: 256 threads hold one 128 x 128 block in registers.
template <class T, int VB>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const QuantParams p)
{
    using L = Lanes<T, VB>;
    constexpr int V = L::V;
    constexpr int kRows = 256 / L::kPer;        // rows of the block loaded at once
    constexpr int NV = kBlock / kRows;
    __shared__ float red[8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = int(blockIdx.x) * kBlock + L::col(int(threadIdx.x) % L::kPer);
    const int64_t r0 = int64_t(blockIdx.y) * kBlock + threadIdx.x / L::kPer;
    typename L::Raw a[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t row = r0 + k * kRows;
        a[k] = L::load(p.x + (row < p.rows ? row : 0) * p.sx, c, row < p.rows ? p.H : 0);
    }
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(L::get(a[k], i)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    const Divider d(m);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int64_t row = r0 + k * kRows;
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = d(L::get(a[k], i));
        L::store_q(p.q + row * p.sq, c, row < p.rows ? p.H : 0, f);
    }
    if (threadIdx.x == 0) p.scale[int64_t(blockIdx.y) * p.ss + blockIdx.x] = d.scale();
}

// ---------------------------------------------------------------- host side

namespace {

using NormFn = void (*)(NormParams);
using QuantFn = void (*)(QuantParams);

// The kernel for nv pieces per thread (a power of two that leaves a row of up to
// 32768 columns to 512 threads, so at most 64 values).
template <class T, int VB, int NV = 1>
NormFn norm_kernel(int nv)
{
    if (nv == NV) return add_rmsnorm_q_kernel<T, NV, VB>;
    if constexpr (NV * Lanes<T, VB>::V < 64)
        return norm_kernel<T, VB, 2 * NV>(nv);
    else
        return nullptr;
}

template <class T>
NormFn norm_kernel(int nv, int vb)
{
    return vb == 32 ? norm_kernel<T, 32>(nv) : vb == 16 ? norm_kernel<T, 16>(nv) : norm_kernel<T, 0>(nv);
}

template <class T, int VB>
QuantFn quant_kernel(bool blocks, int nv)
{
    if (blocks) return quantize_blocks_kernel<T, VB>;
    return nv == 1 ? quantize_rows_kernel<T, 1, VB> : quantize_rows_kernel<T, VB == 16 ? 4 : 2, VB>;
}

template <class T>
QuantFn quant_kernel(bool blocks, int nv, int vb)
{
    return vb == 32 ? quant_kernel<T, 32>(blocks, nv) : vb == 16 ? quant_kernel<T, 16>(blocks, nv)
                                                                  : quant_kernel<T, 0>(blocks, nv);
}

// The widest access (32, 16, or 0 for single elements) that every base and row
// stride of `bits` (their bytes, or-ed) allows.
int access_bytes(uint64_t bits) { return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0; }

// Launches with the programmatic dependency of every kernel here (the kernel
// waits for the previous grid itself), or without where that is refused.
template <class P>
int launch(void (*fn)(P), dim3 grid, int threads, const P &p, glu_stream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    P copy = p;
    void *args[] = {&copy};
    cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(fn), args);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        cfg.attrs = nullptr;
        cfg.numAttrs = 0;
        e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(fn), args);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return glu::cuda_fail(e);
    }
    return GLU_OK;
}

}  // namespace
}  // namespace quant
}  // namespace glu

extern "C" int glu_add_rmsnorm_q(const void *x, int64_t x_stride, const void *residual, int64_t res_stride,
                                 const void *gamma, void *h, int64_t h_stride, void *q, int64_t q_stride,
                                 float *scale, int64_t scale_stride, float *rstd, int64_t n_rows, int64_t n_cols,
                                 float eps, glu_dtype_t dtype, glu_stream_t stream)
{
    using namespace glu::quant;
    bool empty = false;
    // x, residual, gamma, h and rstd under the rules of glu_add_rmsnorm_fwd (h
    // standing in for its y, which has no counterpart here)
    if (int st = glu::validate_add_rmsnorm_inputs(x, x_stride, residual, res_stride, gamma, h, h_stride, rstd, n_rows,
                                                  n_cols, eps, dtype, &empty))
        return st;
    if (empty) {
        glu::record_launch(glu_launch_info_t{});
        return GLU_OK;
    }
    const int E = dtype == GLU_F32 ? 4 : 2;
    const int64_t groups = (n_cols + kBlock - 1) / kBlock;
    if (!q || !scale) return GLU_ERR_NULL;
    if (n_rows == 1) {
        x_stride = res_stride = h_stride = q_stride = n_cols;
        scale_stride = groups;
    }
    if (q_stride < n_cols || scale_stride < groups) return GLU_ERR_STRIDE;
    glu::Span all[7] = {};
    const bool fits = glu::span(x, n_rows, x_stride, n_cols, E, &all[0]) &&
                      glu::span(residual, n_rows, res_stride, n_cols, E, &all[1]) &&
                      glu::span(gamma, 1, n_cols, n_cols, E, &all[2]) &&
                      glu::span(h, n_rows, h_stride, n_cols, E, &all[3]) &&
                      glu::span(rstd, rstd ? n_rows : 0, 1, 1, 4, &all[4]) &&
                      glu::span(q, n_rows, q_stride, n_cols, 1, &all[5]) &&
                      glu::span(scale, n_rows, scale_stride, groups, 4, &all[6]);
    if (!fits) return GLU_ERR_SHAPE;
    for (int o = 5; o < 7; ++o)
        for (int i = 0; i < o; ++i)
            if (glu::overlap(all[i], all[o])) return GLU_ERR_ALIAS;
    if (uintptr_t(scale) % 4 || (rstd && uintptr_t(rstd) % 4)) return GLU_ERR_STRIDE;
    if ((uintptr_t(x) | uintptr_t(residual) | uintptr_t(gamma) | uintptr_t(h)) % uintptr_t(E)) return GLU_ERR_STRIDE;

    // q's accesses are V bytes wide: a quarter or half of the others'
    int vb = access_bytes(uintptr_t(x) | uintptr_t(residual) | uintptr_t(gamma) | uintptr_t(h) |
                          uint64_t(n_cols * E) | uint64_t(x_stride * E) | uint64_t(res_stride * E) |
                          uint64_t(h_stride * E));
    if (vb && (uintptr_t(q) | uint64_t(q_stride)) % uint64_t(vb / E)) vb = 0;
    // Pieces a row has (V values each), and pieces per thread: for 16-bit types
    // and single elements as many as leave 128 threads to a row (bf16 4096 x
    // 4096: 20.6 us against 22.6 with 256 threads, 2048 x 16384: 43.7 against
    // 50.6), but no more than 16 single elements; for f32 pieces 512.
    const int V = vb ? vb / E : 4;
    const int64_t pieces = vb ? n_cols / V : groups * 32;
    int nv = 1;
    while (pieces > int64_t(512) * nv || ((!vb || E == 2) && pieces > int64_t(128) * nv && nv * V < (vb ? 64 : 16))) nv *= 2;
    int tpr = int((pieces + nv - 1) / nv);
    tpr = (tpr + 31) / 32 * 32;
    const int teams = tpr >= 128 ? 1 : 128 / tpr;
    NormParams p{};
    p.x = static_cast<const char *>(x);
    p.res = static_cast<const char *>(residual);
    p.gamma = static_cast<const char *>(gamma);
    p.h = static_cast<char *>(h);
    p.q = static_cast<char *>(q);
    p.scale = scale;
    p.rstd = rstd;
    p.sx = x_stride * E;
    p.sr = res_stride * E;
    p.sh = h_stride * E;
    p.sq = q_stride;
    p.ss = scale_stride;
    p.rows = n_rows;
    p.H = int(n_cols);
    p.tpr = tpr;
    p.eps = eps;
    const int64_t blocks = (n_rows + teams - 1) / teams;
    if (blocks > INT32_MAX) return GLU_ERR_SHAPE;
    const NormFn fn = dtype == GLU_F32   ? norm_kernel<float>(nv, vb)
                      : dtype == GLU_F16 ? norm_kernel<__half>(nv, vb)
                                         : norm_kernel<__nv_bfloat16>(nv, vb);
    if (int st = launch(fn, dim3(unsigned(blocks)), tpr * teams, p, stream)) return st;
    glu_launch_info_t info{};
    info.launched = 1;
    info.vec_bytes = vb ? vb : E;
    info.unroll = nv * V;
    info.threads = tpr * teams;
    info.grid = int32_t(blocks);
    info.path = 9;
    info.vector_units = n_rows;
    glu::record_launch(info);
    return GLU_OK;
}

extern "C" int glu_quantize(const void *x, int64_t x_stride, void *q, int64_t q_stride, float *scale,
                            int64_t scale_stride, int64_t n_rows, int64_t n_cols, int block_rows, glu_dtype_t dtype,
                            glu_stream_t stream)
{
    using namespace glu::quant;
    if (!(dtype == GLU_F32 || dtype == GLU_F16 || dtype == GLU_BF16)) return GLU_ERR_ENUM;
    if (block_rows != 1 && block_rows != kBlock) return GLU_ERR_VALUE;
    if (n_rows < 0 || n_cols < 0 || n_cols > (int64_t(1) << 28)) return GLU_ERR_SHAPE;
    if (n_rows == 0 || n_cols == 0) {
        glu::record_launch(glu_launch_info_t{});
        return GLU_OK;
    }
    if (!x || !q || !scale) return GLU_ERR_NULL;
    const int E = dtype == GLU_F32 ? 4 : 2;
    const bool by_block = block_rows == kBlock;
    const int64_t groups = (n_cols + kBlock - 1) / kBlock;
    const int64_t srows = by_block ? (n_rows - 1) / kBlock + 1 : n_rows;
    if (n_rows == 1) x_stride = q_stride = n_cols;
    if (srows == 1) scale_stride = groups;
    if (x_stride < n_cols || q_stride < n_cols || scale_stride < groups) return GLU_ERR_STRIDE;
    glu::Span sx{}, sq{}, ss{};
    if (!glu::span(x, n_rows, x_stride, n_cols, E, &sx) || !glu::span(q, n_rows, q_stride, n_cols, 1, &sq) ||
        !glu::span(scale, srows, scale_stride, groups, 4, &ss))
        return GLU_ERR_SHAPE;
    if (glu::overlap(sx, sq) || glu::overlap(sx, ss) || glu::overlap(sq, ss)) return GLU_ERR_ALIAS;
    if (uintptr_t(scale) % 4 || uintptr_t(x) % uintptr_t(E)) return GLU_ERR_STRIDE;
    int vb = access_bytes(uintptr_t(x) | uint64_t(n_cols * E) | uint64_t(x_stride * E));
    if (vb && (uintptr_t(q) | uint64_t(q_stride)) % uint64_t(vb / E)) vb = 0;
    const int V = vb ? vb / E : 4;
    QuantParams p{};
    p.x = static_cast<const char *>(x);
    p.q = static_cast<char *>(q);
    p.scale = scale;
    p.sx = x_stride * E;
    p.sq = q_stride;
    p.ss = scale_stride;
    p.rows = n_rows;
    p.H = int(n_cols);
    dim3 grid;
    int nv = 1;
    if (by_block) {
        if (srows > 65535 || groups > INT32_MAX) return GLU_ERR_SHAPE;
        grid = dim3(unsigned(groups), unsigned(srows));
    } else {
        // four 16-byte pieces per thread (two of the others) in rows that fill
        // a block with them, else one
        const int64_t pieces = vb ? n_cols / V : groups * 32;
        const int wide = vb == 16 ? 4 : 2;
        nv = pieces >= 256 * wide ? wide : 1;
        int64_t tpr = (pieces + nv - 1) / nv;
        tpr = tpr > 256 ? 256 : (tpr + 31) / 32 * 32;
        p.tpr = int(tpr);
        const int64_t teams = 256 / tpr;
        const int64_t blocks = (n_rows + teams - 1) / teams;
        const int64_t spans = (pieces + tpr * nv - 1) / (tpr * nv);
        if (blocks > INT32_MAX) return GLU_ERR_SHAPE;
        // stretches in y and, above its limit of 65535, in z (the last ones may lie past the row and do nothing)
        const int64_t layers = (spans + 65534) / 65535;
        grid = dim3(unsigned(blocks), unsigned((spans + layers - 1) / layers), unsigned(layers));
    }
    const int threads = by_block ? 256 : 256 / p.tpr * p.tpr;
    const QuantFn fn = dtype == GLU_F32   ? quant_kernel<float>(by_block, nv, vb)
                       : dtype == GLU_F16 ? quant_kernel<__half>(by_block, nv, vb)
                                          : quant_kernel<__nv_bfloat16>(by_block, nv, vb);
    if (int st = launch(fn, grid, threads, p, stream)) return st;
    glu_launch_info_t info{};
    info.launched = 1;
    info.vec_bytes = vb ? vb : E;
    info.unroll = by_block ? 64 : nv * V;
    info.threads = threads;
    const uint64_t all = uint64_t(grid.x) * grid.y * grid.z;
    info.grid = int32_t(all > INT32_MAX ? INT32_MAX : all);
    info.path = 10;
    info.vector_units = srows * groups;
    glu::record_launch(info);
    return GLU_OK;
}
