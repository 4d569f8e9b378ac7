// rope_rows.cu -- rotary positions of a part of each head, and a projection's fresh rows made into cache rows.
//
// The rotation of dims [at, at + dim) of a head at position p, for i < dim / 2 with the pair (u, v) = elements
// (2 i, 2 i + 1) (interleaved layout) or (i, i + dim / 2) (half layout):
//     a = p inv_freq[i];   u' = scale (u cos a - v sin a);   v' = scale (u sin a + v cos a)
// All arithmetic is f32; an output in bf16 is rounded once.
//
// Both kernels read every value once and write every value once, so DRAM is their floor.  kv8_rope reaches it: 8192 tokens of
// 128 bf16 heads of 192, 805 MB, in 121 us (6.65 TB/s, a plain copy's rate).  kv8_norm_rope_rows does not: 26.1 us for 65536 bf16 rows
// (114 MB, 4.4 TB/s; half layout 26.5) and 31.5 us for f32 rows (6.0 TB/s).  With bf16 rows neither DRAM (37 %) nor the issue slots
// (67 %) are full: a row is about 300 instructions in a chain of sum, root, products, maximum, division and bytes, and 24 warps an SM
// do not cover it all.  A half warp a row halves what a row costs once, but holds twice the registers, and was no faster (24.5 us where
// a warp a row took 25.3, and 1000 rows 2.6 -> 3.9 us).
#include "elem.cuh"
#include "internal.h"
#include "launch.h"
#include "norm.cuh"
#include "quant_fast.cuh"
#include "rope.cuh"
#include "sm100.cuh"

namespace kv8 {
namespace {

using sm100::f2_fma;
using sm100::f2_mul;
using sm100::f2_pack;
using sm100::f2_unpack;

// ---------------------------------------------------------------------------------------------------------
// kv8_rope
// ---------------------------------------------------------------------------------------------------------
constexpr int kRopeThreads = 256, kRopeUnroll = 2, kRestUnroll = 4;  // items of a thread in flight
constexpr int kRopeTable = 1024;                                        // cos / sin pairs of a block's tokens

struct RopeArgs {
    const void *x;
    int64_t x_row, x_head;  // strides in elements
    void *rot, *rest;
    int64_t rot_row, rot_head, rest_row, rest_head;
    const int32_t *position;
    const float *inv_freq;
    float scale;
    int64_t n;
    int heads, at, dim, n_rest;      // n_rest: elements of a head that are not turned, 0 where `rest` is not asked for
    int tokens, head_part, n_parts;  // a block: `tokens` tokens of `head_part` heads, n_parts blocks for all heads
    uint32_t rest_inv, rot_inv;      // 2^32 / items of a head, rounded up: (it * that) >> 32 divides the few items of a block
};

// A block takes some tokens and heads: first it copies their rest, V values an item (V: 16 bytes of x, or one value), while
// the rotated part's first values are on their way, then it turns the rotated part, V / 2 interleaved pairs or V pairs of the
// half layout an item.  (Both kinds in one sequence of items made every warp walk both paths: 160 us for 8192 tokens of 128
// heads of 192.)  An item reads all it needs before it writes, so the rotated part may be written over x.
template <bool kInBf16, bool kOutBf16, bool kHalf, int V>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeArgs a) {
    using In = typename Elem<kInBf16>::T;
    using Out = typename Elem<kOutBf16>::T;
    constexpr int P = kHalf ? V : (V == 1 ? 1 : V / 2);  // pairs of a rotated item
    constexpr bool kTwo = kHalf || V == 1;               // which lies in two places
    constexpr int U = kRopeUnroll;
    __shared__ float2 table[kRopeTable];
    __shared__ uint64_t turns[KV8_MAX_ROPE / 2];
    const int half_dim = a.dim / 2;
    const int64_t block = blockIdx.x / a.n_parts;
    const int part = (int)(blockIdx.x - block * a.n_parts);
    const int64_t n0 = block * a.tokens;
    const int tokens = (int)(a.n - n0 < a.tokens ? a.n - n0 : a.tokens);
    const int h0 = part * a.head_part, heads = min(a.head_part, a.heads - h0), runs = tokens * heads;
    const In *xb = static_cast<const In *>(a.x) + n0 * a.x_row + h0 * a.x_head;
    // item -> token and head of the block, number within the head
    auto place = [&](int it, int per_head, uint32_t inv, int &t, int &h, int &k) {
        const int th = per_head == 1 ? it : (int)__umulhi((uint32_t)it, inv);
        k = it - th * per_head;
        t = tokens == 1 ? 0 : th / heads;
        h = th - t * heads;
    };

    struct Item {
        Raw<kInBf16, V> u, v;  // (v: the second place)
        int t, h, k;
    };
    const int per_head = half_dim / P, items = runs * per_head;
    auto fetch = [&](int base, Item(&w)[U]) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int it = base + j * kRopeThreads;
            if (it < items) {
                place(it, per_head, a.rot_inv, w[j].t, w[j].h, w[j].k);
                const In *x = xb + w[j].t * a.x_row + w[j].h * a.x_head + a.at + w[j].k * (kHalf ? P : 2 * P);
                w[j].u.load(x);
                if constexpr (kTwo) w[j].v.load(x + (kHalf ? half_dim : 1));
            }
        }
    };
    Item w0[U], w1[U];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    fetch(threadIdx.x, w0);
    if (threadIdx.x < half_dim) turns[threadIdx.x] = turn_of(a.inv_freq[threadIdx.x]);

    if (a.n_rest > 0) {
        Out *rest = static_cast<Out *>(a.rest) + n0 * a.rest_row + h0 * a.rest_head;
        const int per_rest = a.n_rest / V, all = runs * per_rest;
        for (int base = threadIdx.x; base < all; base += kRopeThreads * kRestUnroll) {
            Raw<kInBf16, V> r[kRestUnroll];
            int64_t to[kRestUnroll];
#pragma unroll
            for (int j = 0; j < kRestUnroll; ++j) {
                const int it = base + j * kRopeThreads;
                if (it < all) {
                    int t, h, k;
                    place(it, per_rest, a.rest_inv, t, h, k);
                    r[j].load(xb + t * a.x_row + h * a.x_head + (k * V < a.at ? k * V : k * V + a.dim));
                    to[j] = t * a.rest_row + h * a.rest_head + k * V;
                }
            }
#pragma unroll
            for (int j = 0; j < kRestUnroll; ++j) {
                if (base + j * kRopeThreads < all) {
                    if constexpr (kInBf16 == kOutBf16) {
                        r[j].store(rest + to[j]);
                    } else {
                        float x[V];
                        r[j].get(x);
                        store<V>(rest + to[j], x);
                    }
                }
            }
        }
    }

    __syncthreads();
    for (int i = threadIdx.x; i < tokens * half_dim; i += kRopeThreads) {
        const int t = i / half_dim;
        table[i] = turn_cos_sin(a.position[n0 + t], turns[i - t * half_dim], a.scale);
    }
    __syncthreads();
    Out *rot = static_cast<Out *>(a.rot) + n0 * a.rot_row + h0 * a.rot_head;
    auto turn = [&](int base, const Item(&w)[U]) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (base + j * kRopeThreads >= items) continue;
            float x[V], y[V];
            w[j].u.get(x);
            const int i = w[j].k * P;
            Out *o = rot + w[j].t * a.rot_row + w[j].h * a.rot_head + (kHalf ? i : 2 * i);
            const float2 *cs = table + w[j].t * half_dim + i;
            if constexpr (kTwo) {
                w[j].v.get(y);
#pragma unroll
                for (int m = 0; m < V; ++m) {
                    const float p = x[m], q = y[m];
                    x[m] = p * cs[m].x - q * cs[m].y;
                    y[m] = p * cs[m].y + q * cs[m].x;
                }
                store<V>(o, x);
                store<V>(o + (kHalf ? half_dim : 1), y);
            } else {
#pragma unroll
                for (int m = 0; m < P; ++m) {
                    const float p = x[2 * m], q = x[2 * m + 1];
                    x[2 * m] = p * cs[m].x - q * cs[m].y;
                    x[2 * m + 1] = p * cs[m].y + q * cs[m].x;
                }
                store<V>(o, x);
            }
        }
    };
    for (int base = threadIdx.x; base < items; base += 2 * kRopeThreads * U) {
        fetch(base + kRopeThreads * U, w1);
        turn(base, w0);
        fetch(base + 2 * kRopeThreads * U, w0);
        turn(base + kRopeThreads * U, w1);
    }
}

template <bool kInBf16, bool kOutBf16, bool kHalf>
cudaError_t rope_go(const RopeArgs &a, bool wide, int64_t blocks, cudaStream_t st) {
    return launch_dependent(wide ? rope_kernel<kInBf16, kOutBf16, kHalf, kInBf16 ? 8 : 4> : rope_kernel<kInBf16, kOutBf16, kHalf, 1>,
                            (unsigned)blocks, kRopeThreads, 0, st, a);
}

// ---------------------------------------------------------------------------------------------------------
// kv8_norm_rope_rows
// ---------------------------------------------------------------------------------------------------------
constexpr int kRowsThreads = 256;
constexpr int kRowsAhead = 3;  // rows of a warp in shared memory or on their way
constexpr int kRowsBlocks = 3;  // an SM
constexpr int row_bytes(bool bf16) { return kRow * (bf16 ? 2 : 4); }

// One warp a row, grid-stride, the next rows on their way to shared memory meanwhile (each warp for itself): lane l holds latent
// elements 8 l .. and 256 + 8 l .., rotary elements 2 l, 2 l + 1 (a pair of the interleaved layout; of the half layout the partners sit in
// lane l xor 16), and the angle of pair l.
template <bool kBf16, bool kHalf>
__global__ void __launch_bounds__(kRowsThreads, kRowsBlocks) norm_rope_rows_kernel(
    const void *xv, int64_t n, int64_t x_stride, const float *norm_w, float eps, const int32_t *position, const float *inv_freq,
    float rope_scale, const int64_t *dst, uint8_t *kv8, float *kv_scale, int64_t cache_rows, int *err_word) {
    using T = typename Elem<kBf16>::T;
    const T *x = static_cast<const T *>(xv);
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kRowsThreads / 32);
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const uint64_t turn = turn_of(inv_freq[lane]);
    uint64_t w[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        Raw<false, 8> a;
        a.load(norm_w + 256 * j + 8 * lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * j + i] = a.pair(i);
    }
    extern __shared__ __align__(16) uint8_t rows_smem[];
    uint8_t *ring = rows_smem + (threadIdx.x >> 5) * (kRowsAhead * row_bytes(kBf16));
    int32_t next_pos;
    int64_t next_row;
    auto ask = [&](int64_t r, int slot) {  // (a group for every row, empty past the last one)
        if (r < n) {
            const uint8_t *from = reinterpret_cast<const uint8_t *>(x + r * x_stride);
#pragma unroll
            for (int c = 0; c < row_bytes(kBf16); c += 512)
                if (c + 16 * lane < row_bytes(kBf16)) sm100::cp_async_16(ring + slot * row_bytes(kBf16) + c + 16 * lane, from + c + 16 * lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto ask_place = [&](int64_t r) {
        if (r < n) {
            next_pos = position[r];
            next_row = dst[r];
        }
    };
    int64_t r = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
#pragma unroll
    for (int i = 0; i < kRowsAhead - 1; ++i) ask(r + i * warps, i);
    ask_place(r);
    for (int slot = 0; r < n; r += warps, slot = (slot + 1) % kRowsAhead) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead - 2) : "memory");
        __syncwarp();
        uint64_t z[8];
        float k[2];
        {
            const T *xr = reinterpret_cast<const T *>(ring + slot * row_bytes(kBf16));
            Raw<kBf16, 8> raw[2];
            Raw<kBf16, 2> raw_k;
            raw[0].load(xr + 8 * lane);
            raw[1].load(xr + 256 + 8 * lane);
            raw_k.load(xr + kKL + 2 * lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = raw[j / 4].pair(j % 4);
            raw_k.get(k);
        }
        __syncwarp();
        ask(r + (kRowsAhead - 1) * warps, (slot + kRowsAhead - 1) % kRowsAhead);  // (the slot of the row before this one)
        const int32_t pos = next_pos;
        const int64_t row = next_row;
        ask_place(r + warps);
        if (row < 0 || row >= cache_rows) {
            if (lane == 0 && err_word) atomicOr(err_word, (int)KV8_ERR_INDEX);
            continue;
        }
        uint64_t s2 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) s2 = f2_fma(z[j], z[j], s2);
        float ss, s_hi;
        f2_unpack(s2, ss, s_hi);
        ss = warp_sum(ss + s_hi);
        float2 c0 = turn_cos_sin(pos, turn, rope_scale);
        if constexpr (kHalf) {  // (a lane's two pairs are numbers 2 (l mod 16) and the next: their angles are two other lanes')
            const int from = 2 * (lane & 15);
            const float2 c1 = make_float2(__shfl_sync(0xffffffffu, c0.x, from + 1), __shfl_sync(0xffffffffu, c0.y, from + 1));
            c0 = make_float2(__shfl_sync(0xffffffffu, c0.x, from), __shfl_sync(0xffffffffu, c0.y, from));
            const float sign = lane < 16 ? -1.f : 1.f;
            const float o0 = __shfl_xor_sync(0xffffffffu, k[0], 16), o1 = __shfl_xor_sync(0xffffffffu, k[1], 16);
            k[0] = k[0] * c0.x + sign * o0 * c0.y;
            k[1] = k[1] * c1.x + sign * o1 * c1.y;
        } else {
            const float u = k[0], v = k[1];
            k[0] = u * c0.x - v * c0.y;
            k[1] = u * c0.y + v * c0.x;
        }
        const float ms = ss * (1.f / kKL) + eps;
        float pre = 1.f, inv = __frsqrt_rn(ms);
        if (!(ms >= 1e-32f && ss <= 1e30f)) {  // squares that leave the f32 range, infinities, NaN
            double sd = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float lo, hi;
                f2_unpack(z[j], lo, hi);
                sd += (double)lo * (double)lo + (double)hi * (double)hi;
            }
            norm_factor_f64(warp_sum_f64(sd) / kKL + (double)eps, pre, inv);
        }
        if (pre != 1.f) {
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = f2_mul(z[j], f2_pack(pre, pre));
        }
        // (the norm's factor first: then no row's size and no weight's can take the product out of range)
        float amax = 0.f, mul, sc;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[j] = f2_mul(f2_mul(z[j], f2_pack(inv, inv)), w[j]);
            float lo, hi;
            f2_unpack(z[j], lo, hi);
            amax = abs_max_nan(amax, lo, hi);
        }
        amax = warp_max_nan(abs_max_nan(amax, k[0], k[1]));
        uint2 b[2];
        uint32_t bk;
        if (plain_factors(amax, mul, sc)) {
            const uint64_t f = f2_pack(mul, mul);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                b[j] = make_uint2(enc4_scaled(z[4 * j], z[4 * j + 1], f), enc4_scaled(z[4 * j + 2], z[4 * j + 3], f));
            bk = enc2_finite(k[0] * mul, k[1] * mul);
        } else {
            float y[16], qpre;
            amax = finite_abs_max(finite_abs_max(0.f, k[0]), k[1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) f2_unpack(z[j], y[2 * j], y[2 * j + 1]);
#pragma unroll
            for (int j = 0; j < 16; ++j) amax = finite_abs_max(amax, y[j]);
            amax = warp_max(amax);
            row_quant_factors(amax, qpre, mul, sc);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                b[j] = make_uint2(enc4(scale4(make_float4(y[8 * j], y[8 * j + 1], y[8 * j + 2], y[8 * j + 3]), qpre, mul)),
                                  enc4(scale4(make_float4(y[8 * j + 4], y[8 * j + 5], y[8 * j + 6], y[8 * j + 7]), qpre, mul)));
            bk = enc2(__fmul_rn(__fmul_rn(k[0], qpre), mul), __fmul_rn(__fmul_rn(k[1], qpre), mul));
        }
        if (lane == 0) kv_scale[row] = sc;
        uint8_t *q = kv8 + row * kRow;
        *reinterpret_cast<uint2 *>(q + 8 * lane) = b[0];
        *reinterpret_cast<uint2 *>(q + 256 + 8 * lane) = b[1];
        *reinterpret_cast<uint16_t *>(q + kKL + 2 * lane) = (uint16_t)bk;
    }
}

}  // namespace

cudaError_t launch_rope(const void *x, int x_bf16, int64_t n, int heads, int width, int rope_at, int rope_dim,
                        int64_t x_row, int64_t x_head, const int32_t *position, const float *inv_freq, float scale,
                        int half_layout, void *rot, int64_t rot_row, int64_t rot_head, void *rest, int64_t rest_row,
                        int64_t rest_head, int out_bf16, cudaStream_t st) {
    RopeArgs a{};
    a.x = x, a.x_row = x_row, a.x_head = x_head;
    a.rot = rot, a.rot_row = rot_row, a.rot_head = rot_head;
    a.rest = rest, a.rest_row = rest_row, a.rest_head = rest_head;
    a.position = position, a.inv_freq = inv_freq, a.scale = scale;
    a.n = n, a.heads = heads, a.at = rope_at, a.dim = rope_dim;
    a.n_rest = rest ? width - rope_dim : 0;
    // 16 bytes of x at a time where every run of eight values lies on 16 bytes
    const int64_t odd = x_row | x_head | rot_row | rot_head | (rest ? rest_row | rest_head : 0) | rope_at | (width - rope_dim) |
                        (half_layout ? rope_dim / 2 : rope_dim);
    const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rot) | reinterpret_cast<uintptr_t>(rest);
    const bool wide = odd % 8 == 0 && at % 16 == 0;
    const int V = wide ? (x_bf16 ? 8 : 4) : 1;
    const int per_rest = a.n_rest / V, per_rot = half_layout ? rope_dim / 2 / V : rope_dim / (wide ? V : 2), per_head = per_rest + per_rot;
    auto inverse = [](int d) { return (uint32_t)(((1ull << 32) + d - 1) / d); };
    a.rest_inv = per_rest > 0 ? inverse(per_rest) : 0;
    a.rot_inv = inverse(per_rot);
    // a block's items: sixteen a thread, or fewer where that would leave fewer than two blocks an SM
    const int64_t each = n * heads * (int64_t)per_head / ((int64_t)device_sm_count() * 2 * kRopeThreads);
    const int target = kRopeThreads * (int)(each < 1 ? 1 : each < 16 ? each : 16);
    int hp = target / per_head;
    a.head_part = hp < 1 ? 1 : hp < heads ? hp : heads;
    a.n_parts = (heads + a.head_part - 1) / a.head_part;
    a.head_part = (heads + a.n_parts - 1) / a.n_parts;  // even parts
    int tokens = a.n_parts > 1 ? 1 : target / (heads * per_head);
    const int most = kRopeTable / (rope_dim / 2);
    a.tokens = tokens < 1 ? 1 : tokens < most ? tokens : most;
    const int64_t blocks = (n + a.tokens - 1) / a.tokens * a.n_parts;
    switch ((x_bf16 ? 4 : 0) | (out_bf16 ? 2 : 0) | (half_layout ? 1 : 0)) {
        case 0: return rope_go<false, false, false>(a, wide, blocks, st);
        case 1: return rope_go<false, false, true>(a, wide, blocks, st);
        case 2: return rope_go<false, true, false>(a, wide, blocks, st);
        case 3: return rope_go<false, true, true>(a, wide, blocks, st);
        case 4: return rope_go<true, false, false>(a, wide, blocks, st);
        case 5: return rope_go<true, false, true>(a, wide, blocks, st);
        case 6: return rope_go<true, true, false>(a, wide, blocks, st);
        default: return rope_go<true, true, true>(a, wide, blocks, st);
    }
}

cudaError_t launch_norm_rope_rows(const void *x, int x_bf16, int64_t n, int64_t x_stride, const float *norm_w, float eps,
                                  const int32_t *position, const float *inv_freq, float rope_scale, int half_layout,
                                  const int64_t *dst, uint8_t *kv8, float *kv_scale, int64_t cache_rows, int *err_word,
                                  cudaStream_t st) {
    int64_t blocks = (n + kRowsThreads / 32 - 1) / (kRowsThreads / 32);
    const int64_t cap = (int64_t)device_sm_count() * kRowsBlocks;
    if (blocks > cap) blocks = cap;
    const int smem = kRowsThreads / 32 * kRowsAhead * row_bytes(x_bf16 != 0);
    auto go = [&](auto kernel) -> cudaError_t {
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        return launch_dependent(kernel, (unsigned)blocks, kRowsThreads, smem, st, x, n, x_stride, norm_w, eps, position, inv_freq, rope_scale,
                                dst, kv8, kv_scale, cache_rows, err_word);
    };
    if (x_bf16) return half_layout ? go(norm_rope_rows_kernel<true, true>) : go(norm_rope_rows_kernel<true, false>);
    return half_layout ? go(norm_rope_rows_kernel<false, true>) : go(norm_rope_rows_kernel<false, false>);
}

}  // namespace kv8
