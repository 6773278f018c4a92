// What the tensor-core kernels of softmax attention share.
#pragma once

#include "tc_ptx.cuh"
#include "tc_tiles.cuh"

namespace sgla {
namespace {

// Registers a thread of a 384-thread kernel: 168 at launch; its eight row warps take 208, the
// others keep 80 (256 * 208 + 128 * 80 = 63488 of 384 * 168 = 64512).
constexpr int kRowRegs = 208, kOtherRegs = 80;
constexpr float kLog2e = 1.4426950408889634f;

// Exponentials on the FMA pipe: with n = round(x), f = x - n, 2^x = 2^n p3(f), p3 the degree-3
// polynomial of least largest relative error on [-1/2, 1/2] (Remez exchange; 7.5e-5, a fiftieth
// of the rounding of p to bf16 that follows).
// (2^x, 2^y) on the FMA pipe for x, y <= 8, finite.  Below -126 the result is 2^-126.
__device__ __forceinline__ float2 exp2_fma(float2 x) {
    const float2 magic = make_float2(12582912.f, 12582912.f);  // 1.5 * 2^23: the sum's low bits are round(x)
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x.x));  // -126, a NaN stays
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x.y));
    const float2 t = __fadd2_rn(x, magic);
    const float2 f = __fadd2_rn(x, __fadd2_rn(magic, make_float2(-t.x, -t.y)));
    float2 p = __ffma2_rn(f, make_float2(0.0551716685f, 0.0551716685f), make_float2(0.2426111251f, 0.2426111251f));
    p = __ffma2_rn(p, f, make_float2(0.6932609677f, 0.6932609677f));
    p = __ffma2_rn(p, f, make_float2(0.9999280572f, 0.9999280572f));
    p = make_float2(__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)),
                    __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23)));
    return __ffma2_rn(x, make_float2(0.f, 0.f), p);  // NaN for NaN
}


}  // namespace
}  // namespace sgla
