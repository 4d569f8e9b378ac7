// elem.cuh -- f32 / bf16 values in memory, sixteen bytes or one value at a time, as f32 in registers.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

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

// A run of V values as it lies in memory, so that a load in flight takes no more registers than its bytes: V values are 16
// or 32 bytes, or one value.
template <bool kBf16, int V>
struct Raw {
    static constexpr int kWords = V == 1 ? 1 : V * (kBf16 ? 2 : 4) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const typename Elem<kBf16>::T *p) {
        if constexpr (V == 1) {
            if constexpr (kBf16)
                w[0] = __bfloat16_as_ushort(*p);
            else
                w[0] = __float_as_uint(*p);
        } else if constexpr (kWords < 4) {
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) {
                const uint2 a = reinterpret_cast<const uint2 *>(p)[i];
                w[2 * i] = a.x, w[2 * i + 1] = a.y;
            }
            if constexpr (kWords % 2) w[kWords - 1] = reinterpret_cast<const uint32_t *>(p)[kWords - 1];
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
        }
    }
    __device__ __forceinline__ void store(typename Elem<kBf16>::T *p) const {  // as loaded
        if constexpr (V == 1) {
            if constexpr (kBf16)
                *p = __ushort_as_bfloat16((uint16_t)w[0]);
            else
                *p = __uint_as_float(w[0]);
        } else {
            static_assert(kWords % 4 == 0, "whole 16 bytes");
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        if constexpr (V == 1) {
            v[0] = kBf16 ? __uint_as_float(w[0] << 16) : __uint_as_float(w[0]);
        } else if constexpr (kBf16) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) unpack2(w[i], v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
        }
    }
    // values 2 i, 2 i + 1 as a pair of f32
    __device__ __forceinline__ uint64_t pair(int i) const {
        if constexpr (kBf16)
            return sm100::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
        else
            return sm100::f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&v)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    else if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    else
        *p = __float2bfloat16_rn(v[0]);
}
template <int V>
__device__ __forceinline__ void store(float *p, const float (&v)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        *p = v[0];
    }
}

}  // namespace kv8
