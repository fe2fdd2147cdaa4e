// 8-bit codes of a row: shared by the kernels that write them (row quantisation,
// the gated norm and the norms around a block).
//
// A row v with largest magnitude m gets the scale s = m / 127 and the codes
// q_k = rint(127 v_k / m), ties to even. A zero row: s = 0, q = 0. A row with a
// NaN or an infinity: s = NaN, q = 0, so that everything computed from it is NaN
// (codes cannot hold either, and clamping them would hide the fault).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tc.cuh"

namespace mate {
namespace i8 {

// |v| running maximum that keeps a NaN once met
__device__ __forceinline__ float amax_nan(float m, float v)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
    return d;
}

// the same over a pair
__device__ __forceinline__ float amax_nan(float m, float2 v)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(v.x), "f"(v.y));
    return d;
}

// What quantises a row: code = rint(v * pre * mul).
struct RowScale {
    float mul, pre, scale;
};

// EXACT: mul = 127 / amax rounded UP, which makes the codes of bf16 rows the correctly
// rounded ones: the rounding of v * mul is done once (a fused multiply-add onto the
// rounding constant, below), and a tie needs 254 |v| = (2n+1) amax, so 127 divides either
// amax's 8-bit significand (254: mul is then an exact power of two) or 2n+1 <= 254, that
// is n = 63, which rounds away from zero as a product slightly above the tie does. Any
// other product is at least 2^-16 of itself away from a border, and mul's rounding moves
// it by 2^-23. Otherwise, for rows of computed fp32 values, which have roundings of their
// own: mul and scale within 2 fp32 steps, without the two divisions (they were a fifth
// of the norms' instructions).
template <bool EXACT> __device__ __forceinline__ RowScale row_scale(float amax)
{
    RowScale r;
    const bool finite = amax < __int_as_float(0x7f800000);  // false for NaN
    r.pre = amax >= 0x1p-100f && finite ? 1.f : amax > 0.f && finite ? 0x1p64f : 0.f;
    if (EXACT) {
        r.mul = r.pre != 0.f ? __fdiv_ru(127.f, amax * r.pre) : 0.f;
        r.scale = __fdiv_rn(amax, 127.f);
    } else {
        float inv;  // of a normal number; results below 2^-126 kept
        asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(amax * r.pre));
        r.mul = r.pre != 0.f ? 127.f * inv : 0.f;
        r.scale = amax * (1.f / 127.f);
    }
    if (!finite) r.scale = __int_as_float(0x7fc00000);
    return r;
}

// 1.5 * 2^23: v + kRound has the rounded integer of |v| < 2^22 in its low bits
// (two's complement), ties to even as any fp32 sum
constexpr float kRound = 12582912.f;

// four codes, the first in the low byte
__device__ __forceinline__ uint32_t codes4(float2 a, float2 b, float mul)
{
    const float2 m = make_float2(mul, mul), k = make_float2(kRound, kRound);
    const float2 x = tc::fma_f32x2(a, m, k), y = tc::fma_f32x2(b, m, k);
    return __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
}

}  // namespace i8
}  // namespace mate
