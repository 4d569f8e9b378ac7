// quant_blocks.cu -- rows to e4m3 with one f32 scale for each block of 128 columns, a root-mean-square norm before it
// where asked for: the form in which kv8_matmul8 takes its left operand.
//
//     y = x                                         or  y[i] = x[i] w[i] / sqrt(mean(x^2) + eps)
//     scale[k] = amax over block k of |y| / 448;    q[i] = e4m3(y[i] * 448 / amax)     (the row quantizer's steps, per block)
//
// Every value is read once and every byte written once, so DRAM bounds both kernels: sixteen lanes hold a block (eight
// values each) in registers between its maximum and its bytes, and a normed row stays in registers between the sum of
// its squares and its scaling.
#include "elem.cuh"
#include "internal.h"
#include "norm.cuh"
#include "quant_row.cuh"

#include <type_traits>

namespace kv8 {
namespace {

constexpr int kQThreads = 256, kQBlk = KV8_KVB_BLOCK;

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Quantizes a lane's eight values of a block that its half warp holds; returns the block's scale.
__device__ __forceinline__ float quant8(const float (&y)[8], uint2 &bytes) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = finite_abs_max(amax, y[i]);
    amax = half_warp_max(amax);
    float pre, mul, scale;
    row_quant_factors(amax, pre, mul, scale);
    bytes.x = enc4(scale4(make_float4(y[0], y[1], y[2], y[3]), pre, mul));
    bytes.y = enc4(scale4(make_float4(y[4], y[5], y[6], y[7]), pre, mul));
    return scale;
}

// No norm: a block of threads takes 8 rows (a warp each) x kQCols blocks of 128 columns, so that its scales, 8
// neighbours for each column block, go out as whole 32-byte sectors.
constexpr int kQCols = 8, kQRows = kQThreads / 32;

template <bool kBf16>
__global__ void __launch_bounds__(kQThreads) quant_blocks_kernel(const void *__restrict__ xv, int64_t n, int width,
                                                                 int64_t x_stride, uint8_t *__restrict__ q,
                                                                 float *__restrict__ scale, int64_t scale_stride,
                                                                 int col_parts) {
    using T = typename Elem<kBf16>::T;
    __shared__ float sc[kQCols][kQRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tile = blockIdx.x / col_parts;
    const int kb0 = (int)(blockIdx.x - tile * col_parts) * kQCols;
    const int64_t row = tile * kQRows + warp;
    const T *x = static_cast<const T *>(xv) + row * x_stride;
    Raw<kBf16, 8> raw[kQCols / 2];
#pragma unroll
    for (int j = 0; j < kQCols / 2; ++j) {
        const int col = (kb0 + 2 * j) * kQBlk + 8 * lane;
        if (row < n && col < width)
            raw[j].load(x + col);
        else
            raw[j].zero();
    }
#pragma unroll
    for (int j = 0; j < kQCols / 2; ++j) {
        const int col = (kb0 + 2 * j) * kQBlk + 8 * lane;
        float y[8];
        raw[j].get(y);
        uint2 b;
        const float s = quant8(y, b);
        if (row < n && col < width) *reinterpret_cast<uint2 *>(q + row * width + col) = b;
        if ((lane & 15) == 0) sc[2 * j + (lane >> 4)][warp] = s;
    }
    __syncthreads();
    if (threadIdx.x < kQCols * kQRows) {
        const int k = threadIdx.x / kQRows, r = threadIdx.x % kQRows;
        if (tile * kQRows + r < n && (kb0 + k) * kQBlk < width) scale[(kb0 + k) * scale_stride + tile * kQRows + r] = sc[k][r];
    }
}

// With a norm: kT threads a row (a warp, or the whole block), kJ vectors of eight values each.
template <bool kBf16, int kT, int kJ>
__global__ void __launch_bounds__(kQThreads) norm_quant_blocks_kernel(const void *__restrict__ xv, int64_t n, int width,
                                                                      int64_t x_stride, const float *__restrict__ norm_w,
                                                                      float eps, uint8_t *__restrict__ q,
                                                                      float *__restrict__ scale, int64_t scale_stride) {
    using T = typename Elem<kBf16>::T;
    __shared__ float part[kQThreads / 32];
    __shared__ double part_d[kQThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = kT == 32 ? lane : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * (kQThreads / kT) + (kT == 32 ? warp : 0);
    if (row >= n) return;  // (whole warps; with kT == kQThreads no block)
    const T *x = static_cast<const T *>(xv) + row * x_stride;
    Raw<kBf16, 8> raw[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int col = 8 * (t + kT * j);
        if (col < width)
            raw[j].load(x + col);
        else
            raw[j].zero();
    }
    float y[kJ][8], ss = 0.f;
#pragma unroll
    for (int j = 0; j < kJ; ++j) raw[j].get(y[j]);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[j][i], y[j][i], ss);
    ss = warp_sum(ss);
    if constexpr (kT > 32) {
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < kT / 32; ++i) ss += part[i];
    }
    const float ms = ss / (float)width + eps;
    float pre = 1.f, inv = __frsqrt_rn(ms);
    if (!(ms >= 1e-32f && ss <= 1e30f)) {  // squares that leave the f32 range, infinities, NaN: the same for the whole row
        double sd = 0.0;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sd += (double)y[j][i] * (double)y[j][i];
        sd = warp_sum_f64(sd);
        if constexpr (kT > 32) {
            if (lane == 0) part_d[warp] = sd;
            __syncthreads();
            sd = 0.0;
            for (int i = 0; i < kT / 32; ++i) sd += part_d[i];
        }
        norm_factor_f64(sd / width + (double)eps, pre, inv);
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int col = 8 * (t + kT * j);
        if (8 * ((t & ~31) + kT * j) >= width) break;  // (whole warps)
        if (col < width) {
            float w[8];
            load<8>(norm_w + col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] = y[j][i] * pre * inv * w[i];
        }
        uint2 b;
        const float s = quant8(y[j], b);
        if (col < width) {
            *reinterpret_cast<uint2 *>(q + row * width + col) = b;
            if ((lane & 15) == 0) scale[col / kQBlk * scale_stride + row] = s;
        }
    }
}

}  // namespace

cudaError_t launch_quant_blocks(const void *x, int x_bf16, int64_t n, int width, int64_t x_stride, const float *norm_w,
                                float eps, uint8_t *q, float *scale, int64_t scale_stride, cudaStream_t st) {
    if (!norm_w) {
        const int parts = (width + kQCols * kQBlk - 1) / (kQCols * kQBlk);
        const int64_t blocks = (n + kQRows - 1) / kQRows * parts;
        if (x_bf16)
            quant_blocks_kernel<true><<<(unsigned)blocks, kQThreads, 0, st>>>(x, n, width, x_stride, q, scale, scale_stride, parts);
        else
            quant_blocks_kernel<false><<<(unsigned)blocks, kQThreads, 0, st>>>(x, n, width, x_stride, q, scale, scale_stride, parts);
        return cudaGetLastError();
    }
    // a warp a row up to 1024 columns, from there a block
    auto go = [&](auto kernel, int threads) {
        const int per = kQThreads / threads;
        kernel<<<(unsigned)((n + per - 1) / per), kQThreads, 0, st>>>(x, n, width, x_stride, norm_w, eps, q, scale, scale_stride);
    };
    auto pick = [&](auto bf16) {
        constexpr bool b = decltype(bf16)::value;
        if (width <= 512) go(norm_quant_blocks_kernel<b, 32, 2>, 32);
        else if (width <= 1024) go(norm_quant_blocks_kernel<b, 32, 4>, 32);
        else if (width <= 2048) go(norm_quant_blocks_kernel<b, 256, 1>, 256);
        else if (width <= 4096) go(norm_quant_blocks_kernel<b, 256, 2>, 256);
        else if (width <= 8192) go(norm_quant_blocks_kernel<b, 256, 4>, 256);
        else go(norm_quant_blocks_kernel<b, 256, 8>, 256);
    };
    if (x_bf16) pick(std::true_type{});
    else pick(std::false_type{});
    return cudaGetLastError();
}

}  // namespace kv8
