// rope.cuh -- the rotation's angles, shared by every kernel that rotates.
//
// A pair at position p with frequency f (radians a position) turns by the angle p f.  For positions of a million an
// f32 product would be off by 2^-24 of a hundred thousand turns, so the turn is kept as a 64-bit binary fraction:
// with s = frac(f / 2 pi) 2^64, the low 64 bits of the whole-number product p s are frac(p f / 2 pi) 2^64, whatever
// the size of p.  The f64 quotient is good to 2^-53 of itself, so the turn is good to |p f| 2^-56 and, f <= 1, better than an f32
// sine for every int32 position.  The f64 work is done once a thread; a row costs a 64-bit product.
#pragma once

#include "common.cuh"

namespace kv8 {

__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
    const double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of position * frequency, times `scale`.  The turn's nearest quarter is taken off, and the rest, at most an eighth of
// a turn to either side, goes through the Taylor series of both (up to x^9 and x^10: their next terms are below 2^-28).
__device__ __forceinline__ float2 turn_cos_sin(int32_t position, uint64_t turn, float scale) {
    const uint32_t phase = (uint32_t)(((uint64_t)(int64_t)position * turn) >> 32);
    const uint32_t quarter = (phase + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(phase - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float x2 = x * x;
    float s = fmaf(x2, 2.7557319223985893e-6f, -1.984126984126984e-4f);
    s = fmaf(x2, s, 8.3333333333333332e-3f);
    s = fmaf(x2, s, -0.16666666666666666f);
    s = fmaf(x * x2, s, x);
    float c = fmaf(x2, -2.7557319223985888e-7f, 2.4801587301587302e-5f);
    c = fmaf(x2, c, -1.3888888888888889e-3f);
    c = fmaf(x2, c, 4.1666666666666664e-2f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.f);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a * scale : a * scale, quarter & 2 ? -b * scale : b * scale);
}

}  // namespace kv8
