// 8-bit floating point with a scale for each block of 128: the number format
// of the quantised MLP, shared by the streaming quantisers (glu_quant.cu) and
// the GEMM (glu_gemm_q.cu).
//
//     scale = max(amax, 2^-100) / 448,   q = e4m3(v / scale)
//
// with amax the block's largest magnitude and 448 the largest e4m3 value, so
// the largest value of every block is held as +-448 exactly.  The floor keeps
// the scale a normal float and its inverse finite; a block of zeros is held as
// zeros.  e4m3 rounds to nearest-even with 4 significant bits (relative error
// at most 2^-4, absolute at most 2^-10 of a unit of the scale below 2^-6).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace glu {
namespace quant {

constexpr int kBlock = 128;                     // columns (and, for weights, rows) that share a scale
constexpr float kFp8Max = 448.0f;
constexpr float kAmaxFloor = 7.888609052e-31f;  // 2^-100

// Four values to four e4m3 bytes, the first in the lowest byte; magnitudes
// above 448 become 448, NaN stays NaN.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return uint32_t(lo) | (uint32_t(hi) << 16);
}

// v / scale for one block, rounded as if once: with top = max(amax, floor),
// v / (top / 448) = 512 (0.875 v / top), where 0.875 v is exact for 16-bit v.
// The quotient by 1 / top is corrected by its remainder, so that a value that
// lies exactly between two e4m3 numbers (amax * 3/4, say) still does and goes
// to the even one; a product with a rounded 448 / amax would move it.
struct Divider {
    float top, inv;
    __device__ __forceinline__ explicit Divider(float amax)
    {
        top = fmaxf(amax, kAmaxFloor);
        inv = 1.0f / top;
    }
    __device__ __forceinline__ float operator()(float v) const
    {
        const float n = 0.875f * v;
        const float q = n * inv;
        return 512.0f * fmaf(fmaf(-q, top, n), inv, q);
    }
    // 1 / scale, for values that carry roundings of their own: v * factor() is
    // off by two roundings, which no longer moves exact ties.  NaN for a block
    // with an infinity, as the corrected quotient is.
    __device__ __forceinline__ float factor() const { return inv > 0.0f ? kFp8Max / top : top - top; }
    __device__ __forceinline__ float scale() const { return top / kFp8Max; }
};

}  // namespace quant
}  // namespace glu
