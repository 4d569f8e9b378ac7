// elem.cuh -- f32 / bf16 values in memory, eight (16 or 32 bytes), two or one at a time, as f32 in registers.
#pragma once

#include "common.cuh"

namespace kv8 {

template <bool kBf16>
struct Elem;
template <>
struct Elem<true> {
    using T = __nv_bfloat16;
};
template <>
struct Elem<false> {
    using T = float;
};

__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&v)[V]) {
    if constexpr (V == 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        unpack2(w.x, v[0], v[1]);
        unpack2(w.y, v[2], v[3]);
        unpack2(w.z, v[4], v[5]);
        unpack2(w.w, v[6], v[7]);
    } else if constexpr (V == 2) {
        unpack2(*reinterpret_cast<const uint32_t *>(p), v[0], v[1]);
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void load(const float *p, float (&v)[V]) {
    if constexpr (V == 8) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (V == 2) {
        const float2 a = *reinterpret_cast<const float2 *>(p);
        v[0] = a.x, v[1] = a.y;
    } else {
        v[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    else
        *p = __float2bfloat16_rn(v[0]);
}
template <int V>
__device__ __forceinline__ void store(float *p, const float (&v)[V]) {
    if constexpr (V == 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}

}  // namespace kv8
