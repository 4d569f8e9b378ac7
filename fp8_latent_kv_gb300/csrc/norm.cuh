// norm.cuh -- the root-mean-square norm's factor where f32 does not carry the sum of squares.
#pragma once

#include "common.cuh"

namespace kv8 {

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The factor of a root-mean-square norm, y = ((x * pre) * inv) * w, where the f32 sum of squares left its range: from the f64 mean
// square (eps included).  pre, a power of two, keeps inv a normal f32.  A mean square that is not finite gives NaN, so that all bytes
// of the row are 0 (a factor of 0 would keep the signs of its finite values, and leave 0x80 for the negative ones).
static __device__ __noinline__ void norm_factor_f64(double mean_square, float &pre, float &inv) {
    const double f = 1.0 / sqrt(mean_square);
    const double p = f < 5.421010862427522e-20 ? 5.421010862427522e-20 : f > 18446744073709551616.0 ? 18446744073709551616.0 : 1.0;
    pre = (float)p;
    inv = mean_square <= 1.7976931348623157e308 ? (float)(f / p) : __int_as_float(0x7FC00000);
}

}  // namespace kv8
