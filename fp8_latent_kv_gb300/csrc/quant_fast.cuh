// quant_fast.cuh -- the row quantizer's steps for values that are all finite: the same bytes and scales as quant_row.cuh's with
// a third of the instructions.  A maximum that lets NaN through tells whether that holds; where it does not, or where
// 448 / amax overflows, the callers take quant_row.cuh's steps.
#pragma once

#include "quant_row.cuh"
#include "sm100.cuh"

namespace kv8 {

// max(acc, |a|, |b|), NaN if one of them is
__device__ __forceinline__ float abs_max_nan(float acc, float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(acc), "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// all values finite and 448 / amax a finite number (or all values 0): `mul` and `scale` as row_quant_factors gives them, pre 1
__device__ __forceinline__ bool plain_factors(float amax, float &mul, float &scale) {
    mul = amax != 0.f ? __fdiv_rn(448.f, amax) : 1.f;
    scale = __fdiv_rn(amax, 448.f);
    return amax <= 3.402823466e38f && mul <= 3.402823466e38f;
}
__device__ __forceinline__ uint32_t enc2_finite(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}
// two pairs times `mul`, encoded
__device__ __forceinline__ uint32_t enc4_scaled(uint64_t p, uint64_t q, uint64_t mul) {
    float a, b, c, d;
    sm100::f2_unpack(sm100::f2_mul(p, mul), a, b);
    sm100::f2_unpack(sm100::f2_mul(q, mul), c, d);
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

}  // namespace kv8
