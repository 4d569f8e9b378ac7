// rope.cuh -- the rotation's angles, shared by every kernel that rotates.
//
// A pair at position p with frequency f (radians a position) turns by the angle p f.  For positions of a million an
// f32 product would be off by 2^-24 of a hundred thousand turns, so the turn is kept as a 64-bit binary fraction:
// with s = frac(f / 2 pi) 2^64, the low 64 bits of the whole-number product p s are frac(p f / 2 pi) 2^64, whatever
// the size of p.  s is the nearest whole number (for |f| up to 2^40), so the turn is off by |p| 2^-65, 2^-34 of a turn for the largest
// int32 position, and small angles keep all of an f32's bits.
#pragma once

#include "common.cuh"

namespace kv8 {

// f = m 2^e with whole m, so s is m times the first 128 bits of 1 / (2 pi), shifted: whole-number steps, which take less
// time than one product in f64 (a call of one fresh row 2.0 -> 1.9 us, of 1000 2.7 -> 2.2; two pieces in f64 2.6 and 3.8).
__device__ __forceinline__ uint64_t turn_of(float inv_freq) {
    constexpr uint64_t kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;  // 2^128 / (2 pi)
    const uint32_t bits = __float_as_uint(inv_freq);
    const int ex = (bits >> 23) & 255, shift = 214 - max(ex, 1);  // f / 2 pi = m 2^128 / (2 pi) 2^-(shift + 64)
    const uint64_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const uint64_t p0 = m * kLow, c = __umul64hi(m, kLow), h = m * kHigh, p1 = h + c, p2 = __umul64hi(m, kHigh) + (p1 < c ? 1 : 0);
    const int k = shift & 63;
    const bool near = shift < 64, far = shift >= 128;
    const uint64_t below = near ? 0 : far ? p1 : p0, low = near ? p0 : far ? p2 : p1, high = near ? p1 : far ? 0 : p2;
    uint64_t turn = k ? (low >> k | high << (64 - k)) + (low >> (k - 1) & 1) : low + (below >> 63);
    if (shift < 0 || shift >= 192) turn = 0;
    return bits >> 31 ? 0 - turn : turn;
}

// cos and sin of position * frequency, times `scale`.  The turn's nearest quarter is taken off, and the rest, at most an eighth of
// a turn to either side, goes through the Taylor series of both (up to x^9 and x^10: their next terms are below 2^-28).
__device__ __forceinline__ float2 turn_cos_sin(int32_t position, uint64_t turn, float scale) {
    const uint64_t phase = (uint64_t)(int64_t)position * turn;
    const uint32_t quarter = ((uint32_t)(phase >> 32) + 0x20000000u) >> 30;
    const float x = __ll2float_rn((int64_t)(phase - ((uint64_t)quarter << 62))) * 3.4061215800865545e-19f;  // 2 pi / 2^64
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
