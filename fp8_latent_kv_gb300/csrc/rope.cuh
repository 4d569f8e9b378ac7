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

// cos and sin of position * frequency, times `scale`
__device__ __forceinline__ float2 turn_cos_sin(int32_t position, uint64_t turn, float scale) {
    const int64_t phase = (int64_t)((uint64_t)(int64_t)position * turn);
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077392578125e-10f, &s, &c);  // half turns: 2^-31 of the high word
    return make_float2(c * scale, s * scale);
}

}  // namespace kv8
