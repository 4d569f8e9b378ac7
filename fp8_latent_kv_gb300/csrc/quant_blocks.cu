// quant_blocks.cu -- rows to e4m3 with one f32 scale for each block of 128 columns, a root-mean-square norm before it
// where asked for: the form in which kv8_matmul8 takes its left operand.
//
//     y = x                                         or  y[i] = x[i] w[i] / sqrt(mean(x^2) + eps)
//     scale[k] = amax over block k of |y| / 448;    q[i] = e4m3(y[i] * 448 / amax)     (the row quantizer's steps, per block)
//
// Every value is read once and every byte written once, so DRAM is the floor of both kernels: eight values a lane stay in
// registers between their block's maximum and its bytes, and a normed row between the sum of its squares and its scaling.
// Without a norm they reach it (8192 x 16384: f32 93 us, 7.3 TB/s, part of the bytes still in L2 at the end; bf16 61 us, 6.6 TB/s).
// With one f32 rows of 16384 take 111 us (6.1 TB/s), bf16 rows 93 (4.4), of 8192 47, of 4096 25, of 2048 15 (3.4): the row, the next
// row and the products lie in 80 to 120 registers, so that few warps an SM (36 % of the most at 8192 columns) have a row's chain of sum, barrier,
// root, maxima and divisions to cover; neither DRAM (51 %) nor issue slots (57 %) are full.
#include "elem.cuh"
#include "internal.h"
#include "launch.h"
#include "norm.cuh"
#include "quant_fast.cuh"

#include <type_traits>

namespace kv8 {
namespace {

constexpr int kQThreads = 256, kQBlk = KV8_KVB_BLOCK;

using sm100::f2_fma;
using sm100::f2_mul;
using sm100::f2_pack;
using sm100::f2_unpack;

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Quantizes J times eight values a lane, of which each sixteen lanes hold J blocks (z[j], as pairs): bytes, and the scale of one
// block, number `mine`, which every lane (lane & 15) / (16 / J) == mine returns.
// The maxima of the J blocks are taken together: with each exchange a lane keeps half of the blocks that it still
// carries, so J = 4 takes 5 exchanges instead of 16 and the divisions are made once.
template <int J>
__device__ __forceinline__ float quant_blocks_of(const uint64_t (&z)[J][4], uint2 (&bytes)[J], int &mine) {
    const int lane = threadIdx.x & 31;
    float m[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        m[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(z[j][i], a, b);
            m[j] = abs_max_nan(m[j], a, b);
        }
    }
    int left = 8;
    mine = 0;
#pragma unroll
    for (int k = J; k > 1; k /= 2, left /= 2) {
        const bool up = lane & left;
#pragma unroll
        for (int j = 0; j < k / 2; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? m[j] : m[j + k / 2], left);
            m[j] = max_nan(up ? m[j + k / 2] : m[j], other);
        }
        mine += up ? k / 2 : 0;
    }
#pragma unroll
    for (; left > 0; left /= 2) m[0] = max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], left));
    float mul, scale;
    const bool plain = plain_factors(m[0], mul, scale);
    if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float f = __shfl_sync(0xffffffffu, mul, (lane & 16) | j * (16 / J));
            const uint64_t ff = f2_pack(f, f);
            bytes[j] = make_uint2(enc4_scaled(z[j][0], z[j][1], ff), enc4_scaled(z[j][2], z[j][3], ff));
        }
        return scale;
    }
    float of_mine = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        float y[8], amax = 0.f, pre;
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(z[j][i], y[2 * i], y[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = finite_abs_max(amax, y[i]);
        row_quant_factors(half_warp_max(amax), pre, mul, scale);
        bytes[j].x = enc4(scale4(make_float4(y[0], y[1], y[2], y[3]), pre, mul));
        bytes[j].y = enc4(scale4(make_float4(y[4], y[5], y[6], y[7]), pre, mul));
        if (j == mine) of_mine = scale;
    }
    return of_mine;
}

// No norm: a block of threads takes 8 rows (a warp each) x kQCols blocks of 128 columns, so that its scales, 8
// neighbours for each column block, go out as whole 32-byte sectors.
constexpr int kQCols = 8, kQRows = kQThreads / 32;

template <bool kBf16>
__global__ void __launch_bounds__(kQThreads) quant_blocks_kernel(const void *xv, int64_t n, int width, int64_t x_stride, uint8_t *q,
                                                                 float *scale, int64_t scale_stride, int col_parts) {
    using T = typename Elem<kBf16>::T;
    __shared__ float sc[kQCols][kQRows];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
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
    uint64_t z[kQCols / 2][4];
#pragma unroll
    for (int j = 0; j < kQCols / 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[j][i] = raw[j].pair(i);
    uint2 b[kQCols / 2];
    int mine;
    const float s = quant_blocks_of<kQCols / 2>(z, b, mine);
#pragma unroll
    for (int j = 0; j < kQCols / 2; ++j) {
        const int col = (kb0 + 2 * j) * kQBlk + 8 * lane;
        if (row < n && col < width) *reinterpret_cast<uint2 *>(q + row * width + col) = b[j];
    }
    if (lane % (32 / kQCols) == 0) sc[2 * mine + (lane >> 4)][warp] = s;
    __syncthreads();
    if (threadIdx.x < kQCols * kQRows) {
        const int k = threadIdx.x / kQRows, r = threadIdx.x % kQRows;
        if (tile * kQRows + r < n && (kb0 + k) * kQBlk < width) scale[(kb0 + k) * scale_stride + tile * kQRows + r] = sc[k][r];
    }
}

// With a norm: kT threads a row (a warp, or the whole block), kJ vectors of eight values each, row after row; a row is loaded
// while the one before is worked on.
template <bool kBf16, int kT, int kJ, int kBlocks>
__global__ void __launch_bounds__(kT == 32 ? kQThreads : kT, kBlocks)
    norm_quant_blocks_kernel(const void *xv, int64_t n, int width, int64_t x_stride, const float *norm_w, float eps, uint8_t *q,
                             float *scale, int64_t scale_stride) {
    using T = typename Elem<kBf16>::T;
    constexpr int kRows = kT == 32 ? kQThreads / kT : 1;  // of a block at a time
    __shared__ float part[2][kT / 32];
    __shared__ double part_d[2][kT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = kT == 32 ? lane : threadIdx.x;
    const T *x = static_cast<const T *>(xv);
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    Raw<kBf16, 8> raw[kJ];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int col = 8 * (t + kT * j);
            if (row < n && col < width)
                raw[j].load(x + row * x_stride + col);
            else
                raw[j].zero();
        }
    };
    int64_t row = (int64_t)blockIdx.x * kRows + (kT == 32 ? warp : 0);
    fetch(row);
    for (int turn = 0; row < n; row += (int64_t)gridDim.x * kRows, turn ^= 1) {  // (one row a warp, or a block: no thread leaves others behind)
        uint64_t z[kJ][4], s2 = 0;
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[j][i] = raw[j].pair(i);
        fetch(row + (int64_t)gridDim.x * kRows);
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = f2_fma(z[j][i], z[j][i], s2);
        float ss, s_hi;
        f2_unpack(s2, ss, s_hi);
        ss += s_hi;
        ss = warp_sum(ss);
        if constexpr (kT > 32) {
            if (lane == 0) part[turn][warp] = ss;
            __syncthreads();
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < kT / 32; ++i) ss += part[turn][i];
        }
        const float ms = ss / (float)width + eps;
        float pre = 1.f, inv = __frsqrt_rn(ms);
        if (!(ms >= 1e-32f && ss <= 1e30f)) {  // squares that leave the f32 range, infinities, NaN: the same for the whole row
            double sd = 0.0;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    f2_unpack(z[j][i], lo, hi);
                    sd += (double)lo * (double)lo + (double)hi * (double)hi;
                }
            sd = warp_sum_f64(sd);
            if constexpr (kT > 32) {
                if (lane == 0) part_d[turn][warp] = sd;
                __syncthreads();
                sd = 0.0;
                for (int i = 0; i < kT / 32; ++i) sd += part_d[turn][i];
            }
            norm_factor_f64(sd / width + (double)eps, pre, inv);
        }
        if (pre != 1.f) {
#pragma unroll
            for (int j = 0; j < kJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] = f2_mul(z[j][i], f2_pack(pre, pre));
        }
        // (the norm's factor first: then no row's size and no weight's can take the product out of range)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int col = 8 * (t + kT * j);
            if (col < width) {
                Raw<false, 8> w;
                w.load(norm_w + col);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] = f2_mul(f2_mul(z[j][i], f2_pack(inv, inv)), w.pair(i));
            }
        }
        uint2 b[kJ];
        int mine;
        const float sc = quant_blocks_of<kJ>(z, b, mine);
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
            const int col = 8 * (t + kT * j);
            if (col < width) *reinterpret_cast<uint2 *>(q + row * width + col) = b[j];
        }
        const int block = (8 * (t + kT * mine)) / kQBlk;
        if (lane % (16 / kJ) == 0 && block * kQBlk < width) scale[block * scale_stride + row] = sc;
    }
}

}  // namespace

cudaError_t launch_quant_blocks(const void *x, int x_bf16, int64_t n, int width, int64_t x_stride, const float *norm_w,
                                float eps, uint8_t *q, float *scale, int64_t scale_stride, cudaStream_t st) {
    if (!norm_w) {
        const int parts = (width + kQCols * kQBlk - 1) / (kQCols * kQBlk);
        const int64_t blocks = (n + kQRows - 1) / kQRows * parts;
        return launch_dependent(x_bf16 ? quant_blocks_kernel<true> : quant_blocks_kernel<false>, (unsigned)blocks, kQThreads, 0, st, x, n,
                                width, x_stride, q, scale, scale_stride, parts);
    }
    // A warp a row up to 1024 columns, from there a block, of as few threads as hold a row: what a thread's blocks of columns
    // share (their maxima, the divisions) is made once for them.  (8192 bf16 rows of 2048, partly in the L2: 64 threads 12.8 us, 256
    // threads 18.0; of 4096: 128 threads 21.1, 256 threads 25.0; f32 rows of 4096, with twice the bytes on their way: 32.1 and 30.0.)
    auto go = [&](auto kernel, int threads, int rows, int blocks_per_sm) {
        const int64_t need = (n + rows - 1) / rows, most = (int64_t)device_sm_count() * blocks_per_sm;
        return launch_dependent(kernel, (unsigned)(need < most ? need : most), threads, 0, st, x, n, width, x_stride, norm_w, eps, q, scale,
                                scale_stride);
    };
    auto pick = [&](auto bf16) {
        constexpr bool b = decltype(bf16)::value;
        if (width <= 512) return go(norm_quant_blocks_kernel<b, 32, 2, 4>, 256, 8, 4);
        if (width <= 1024) return go(norm_quant_blocks_kernel<b, 32, 4, 2>, 256, 8, 2);
        if (width <= 2048) return go(norm_quant_blocks_kernel<b, 64, 4, b ? 12 : 8>, 64, 1, b ? 12 : 8);
        if (width <= 4096) {
            if constexpr (b)
                return go(norm_quant_blocks_kernel<b, 128, 4, 6>, 128, 1, 6);
            else
                return go(norm_quant_blocks_kernel<b, 256, 2, 4>, 256, 1, 4);
        }
        if (width <= 8192) return go(norm_quant_blocks_kernel<b, 256, 4, b ? 3 : 2>, 256, 1, b ? 3 : 2);
        return go(norm_quant_blocks_kernel<b, 512, 4, 1>, 512, 1, 1);
    };
    return x_bf16 ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace kv8
