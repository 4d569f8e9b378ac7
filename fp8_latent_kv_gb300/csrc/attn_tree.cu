// attn_tree.cu -- attention of drafted tokens over a paged latent cache: the kernel for f32 queries, and the merge of the
// groups that a share boundary cuts.
//
// For column (token i, head h) of a sequence and row t:  s_t = sm_scale * scale_t * q.e4m3(row_t),
// out = sum_t 2^((s_t - m) log2 e) scale_t e4m3(Lc_t) / sum_t 2^((s_t - m) log2 e), one pass over the rows with
// the running maximum m.  All columns of a sequence read the same rows.
//
// The products run on the tensor cores with f16 operands, which hold every e4m3 value: a query element, scaled by its
// column's power of two, is the sum of two f16 values to 2^-22 of itself (or 2^-39 of the column's largest), and so is a
// weight p * scale, scaled by a power of two for its column and step.  The sums are kept in f32: the context's over 64 rows
// at most in the tensor core, whose additions are not rounded to nearest, then by f32 additions.
// These are register-operand MMAs (3 cycles of an SM for 16 x 8 x 16, measured here), which take the rows' e4m3 pairs
// converted in registers; tcgen05 would want the rows as f16 in shared memory, 74 KB of 64 rows written by the threads beside 76 KB of
// queries.  8 x 8 tokens of 128 heads over 4096 rows: 550 us, 133 TFLOP/s (38.6 on the CUDA cores); a step of 64 rows
// takes 9.3 thousand cycles, 3.4 in the scores and 3.5 in the context, which the MMAs' rate bounds, the rest between the
// barriers of the softmax.
#include "sm100.cuh"
#include "tree.cuh"

#include <math.h>

#include <algorithm>

namespace kv8 {
namespace {

using namespace sm100;

constexpr int kCols = 32;      // (token, head) columns per block
constexpr int kUnit = 32;      // rows that the shares count
constexpr int kRows = 64;      // rows per step: two units where there are two
// A segment's start and end cost as much as this many units: 16 sequences of up to 4 tokens of 32 heads over up to 700 rows
// took 42.2 us with 0, 34.2 with 1, 30.7 with 2, 28.6 with 4, 32.3 with 8; 30 of up to 3 tokens of 20 heads over up to 3000
// rows 78.1, 77.2, 72.0, 72.6, 77.1.
constexpr int kSegment = 4;
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
// Strides in bytes.  A tile's: 16-byte copies, and 148 words put eight rows' four words into 32 banks.  A query column's: four
// columns' four 8-byte pieces in 32 banks.
constexpr int kTileStride = 592, kQStride = 2 * kRow + 32;
constexpr int kSStride = kCols + 8;        // words
// A step's weights are measured by its largest score plus a scale's logarithm, a sum that from here on may be binary orders off: weights
// would leave their f16 pieces.  Such a column is NaN.  (Measuring them again, with the maximum taken off first: 555 us against 550
// for the largest case, which does not do it.)
constexpr float kFar = 33554432.f;
constexpr int kSteps = kRow / 16 / 4;      // 16-byte steps of a row that a warp's part of the scores covers
static_assert(kSteps * 64 == kRow, "a row's quarters");

struct Smem {
    alignas(16) uint8_t q[2][kCols][kQStride];  // the columns' queries: f16 pieces
    alignas(16) uint8_t tile[2][kRows][kTileStride];  // this step's cache rows and the next's; rows left out are zero
    union {
        float s[4][kRows][kSStride];       // the dot products, by quarter of the row
        alignas(16) uint8_t w[2][kCols][2 * kRows];  // weights: f16 pieces, a 16-row step's rows as 0 1 8 9 2 3 10 11 ...
    };
    uint64_t full[2];                      // a step's rows have landed
    float scale[2][kRows], log_scale[2][kRows];
    alignas(4) uint8_t there[2][kRows];
    int m_max[2][kCols], e_max[2][kCols];  // of a step's scores and of the weights' logarithms, in the order of whole numbers
    float z_part[kWarps][kCols];
    int abort_flag;
    float corr[kCols], unit[kCols];        // the accumulators' factor, the step's weights'
    float factor[kCols];                   // scores: sm_scale log2(e) / the column's power of two
};

__global__ void __launch_bounds__(288) tree_sched_kernel(TreeArgs a) {
    __shared__ TreeScan scan;
    grid_dependency_wait();
    grid_launch_dependents();
    tree_schedule<kCols, kUnit, kSegment, 1>(a, scan);
}

// Floats as whole numbers of the same order, and back.
__device__ __forceinline__ int float_order(float v) {
    const int i = __float_as_int(v);
    return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }
// A column's 8-byte piece u of 16 (four rows of a 16-row step): where a load of four columns by four pieces, and a store of
// one piece of 16 columns, meet 32 banks.
__device__ __forceinline__ int weight_offset(int col, int u) { return 8 * (u ^ (4 * (col & 3)) ^ (col >> 2 & 3)); }

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
    return r;
}
// d += a b: a [16][16], b [16][8] f16, d [16][8] f32.  Lane 4 g + c holds of a rows g and g + 8, columns 2 c, 2 c + 1 (a0, a1)
// and 8 on (a2, a3); of b column g, the same rows (b0, b1); of d rows g (d0, d1) and g + 8, columns 2 c, 2 c + 1.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two values -> f16 pieces: the nearest, and the nearest to what is left.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Dot products: a warp takes 32 rows and a quarter of their bytes against 16 columns, a thread's four bytes of a 16-byte
// step standing for rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the contraction on both sides.
__device__ __forceinline__ void partial_scores(Smem &sm, const uint8_t (*tile)[kTileStride], int warp, int lane) {
    const int g = lane >> 2, c = lane & 3, r0 = 32 * (warp & 1) + g, part = warp >> 1 & 3, n0 = 16 * (warp >> 3);
    float acc[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
#pragma unroll 3
    for (int k = 0; k < kSteps; ++k) {
        const int at = 16 * (part * kSteps + k) + 4 * c;
        uint32_t a[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t v = *reinterpret_cast<const uint32_t *>(&tile[r0 + 16 * m + 8 * i][at]);
                a[m][i] = e4m3x2_to_f16x2(v);
                a[m][2 + i] = e4m3x2_to_f16x2(v >> 16);
            }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int piece = 1; piece >= 0; --piece) {
                const uint2 b = *reinterpret_cast<const uint2 *>(&sm.q[piece][n0 + 8 * n + g][2 * at]);
#pragma unroll
                for (int m = 0; m < 2; ++m) mma_f16(acc[m][n], a[m], b.x, b.y);
            }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float2 *>(&sm.s[part][r0 + 16 * m + 8 * i][n0 + 8 * n + 2 * c]) = make_float2(acc[m][n][2 * i], acc[m][n][2 * i + 1]);
}

// acc = acc * corr + weights x rows * unit: a warp has all columns by 32 latent dims.  A thread's bytes
// 4 g .. 4 g + 3 of two rows make the operand's pairs for four products of 8 dims (4 g + n, g < 8); so it ends with columns
// g + 8 i + 16 m, dims 8 c + n and 8 c + 4 + n.
__device__ __forceinline__ void context(const Smem &sm, const uint8_t (*tile)[kTileStride], int steps, int warp, int lane, float (&acc)[2][4][4]) {
    const int g = lane >> 2, c = lane & 3;
    {
        float t[2][4][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) t[m][n][i] = 0.f;
#pragma unroll 2
        for (int k = 0; k < steps; ++k) {
            uint32_t b[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *src = &tile[16 * k + 8 * i + 2 * c][32 * warp + 4 * g];
                const uint32_t x = *reinterpret_cast<const uint32_t *>(src), y = *reinterpret_cast<const uint32_t *>(src + kTileStride);
                const uint32_t lo = __byte_perm(x, y, 0x5140), hi = __byte_perm(x, y, 0x7362);
                b[i][0] = e4m3x2_to_f16x2(lo);
                b[i][1] = e4m3x2_to_f16x2(lo >> 16);
                b[i][2] = e4m3x2_to_f16x2(hi);
                b[i][3] = e4m3x2_to_f16x2(hi >> 16);
            }
#pragma unroll
            for (int piece = 1; piece >= 0; --piece)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(&sm.w[piece][16 * m + g][weight_offset(g, 4 * k + c)]);
                    const uint2 v = *reinterpret_cast<const uint2 *>(&sm.w[piece][16 * m + 8 + g][weight_offset(8 + g, 4 * k + c)]);
                    const uint32_t a[4] = {u.x, v.x, u.y, v.y};
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma_f16(t[m][n], a, b[0][n], b[1][n]);
                }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float f = sm.corr[16 * m + 8 * i + g], u = sm.unit[16 * m + 8 * i + g];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    acc[m][n][2 * i] = fmaf(acc[m][n][2 * i], f, t[m][n][2 * i] * u);
                    acc[m][n][2 * i + 1] = fmaf(acc[m][n][2 * i + 1], f, t[m][n][2 * i + 1] * u);
                }
            }
    }
}

__global__ void __launch_bounds__(kThreads, 1) attn_tree_f32_kernel(TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad_page = false, ok = true;
    if (tid == 0) {
        mbar_init(&sm.full[0], kRows);
        mbar_init(&sm.full[1], kRows);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (tid < 2 * kCols) (&sm.m_max[0][0])[tid] = (&sm.e_max[0][0])[tid] = float_order(-INFINITY);
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    TreeWalk walk;
    walk.begin(a, blockIdx.x);
    TreeSegment seg;
    uint32_t step = 0;  // of all segments
    while (ok && walk.next<kCols, kUnit>(a, seg)) {
        const int g0 = seg.g * kCols, nc = min(kCols, seg.q.n * a.H - g0);
        const int64_t q_base = (int64_t)seg.q.q0 * a.H + g0, rows_end = seg.q.len + seg.q.n;
        const int64_t p_begin = (int64_t)seg.t0 * kUnit, p_end = min((int64_t)seg.t1 * kUnit, rows_end);
        // the step's cache rows from position p0 on, of which a warp's first lanes hold one each
        const int r_own = 4 * warp + lane;
        int64_t row = -1;
        float scale = 0.f;
        auto fetch_row = [&](int64_t p0) {
            row = -1;
            if (lane < 4 && p0 + r_own < p_end) {
                row = tree_row(a, seg.b, p0 + r_own);
                bad_page |= row < 0;
            }
            scale = row >= 0 ? __ldg(a.kv_scale + row) : 0.f;
        };
        // and brings into a buffer that all threads are done with
        auto copy_row = [&](int buf) {
            if (lane >= 4) return;
            const bool there = row >= 0;
            if (scale > 3.402823466e38f) scale = NAN;  // (a score of -inf would say that nobody attends the row)
            sm.scale[buf][r_own] = scale;
            sm.log_scale[buf][r_own] = log2f(scale);
            sm.there[buf][r_own] = there;
            if (there) {
                fence_proxy_async_smem();  // (the threads have read the buffer; the copy writes it)
                mbar_arrive_expect_tx(&sm.full[buf], kRow);
                bulk_load(sm.tile[buf][r_own], a.kv8 + row * kRow, kRow, &sm.full[buf]);
            } else {
                for (int i = 0; i < kRow; i += 16) *reinterpret_cast<uint4 *>(&sm.tile[buf][r_own][i]) = make_uint4(0u, 0u, 0u, 0u);
                mbar_arrive(&sm.full[buf]);
            }
        };
        fetch_row(p_begin);
        __syncthreads();  // the segment before is done with all of this
        copy_row(step & 1);
        {
            // sixteen threads split a column
            const int c = tid >> 4;
            float4 v[kRow / 64];
            float mx = 0.f;
            bool fine = true;
#pragma unroll
            for (int j = 0; j < kRow / 64; ++j) {
                const int k4 = (tid & 15) + 16 * j;
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < nc)
                    v[j] = k4 < kKL / 4 ? __ldg(static_cast<const float4 *>(a.q_lat) + (q_base + c) * (kKL / 4) + k4)
                                        : __ldg(static_cast<const float4 *>(a.q_rope) + (q_base + c) * (kKR / 4) + (k4 - kKL / 4));
            }
#pragma unroll
            for (int j = 0; j < kRow / 64; ++j) {
                const float most = fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)), fmaxf(fabsf(v[j].z), fabsf(v[j].w)));
                mx = fmaxf(mx, most);
                fine = fine && v[j].x == v[j].x && v[j].y == v[j].y && v[j].z == v[j].z && v[j].w == v[j].w;
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // a NaN or an infinity makes all of the column's pieces NaN
            const uint32_t odd = __ballot_sync(0xffffffffu, !fine || mx > 3.402823466e38f);
            fine = (odd >> (lane & 16) & 0xFFFFu) == 0u;
            int E = 0;
            if (fine && mx > 0.f) frexpf(mx, &E);
            const int up = fine && mx > 0.f ? min(15 - E, 100) : 0;  // max |q| 2^up in [2^14, 2^15), or less below 2^-86
            const float f = fine ? ldexpf(1.f, up) : NAN;
            if ((tid & 15) == 0) sm.factor[c] = ldexpf(a.sm_scale_log2, -up);
#pragma unroll
            for (int j = 0; j < kRow / 64; ++j) {
                uint2 hi, lo;
                split_f16(v[j].x * f, v[j].y * f, hi.x, lo.x);
                split_f16(v[j].z * f, v[j].w * f, hi.y, lo.y);
                *reinterpret_cast<uint2 *>(&sm.q[0][c][8 * ((tid & 15) + 16 * j)]) = hi;
                *reinterpret_cast<uint2 *>(&sm.q[1][c][8 * ((tid & 15) + 16 * j)]) = lo;
            }
        }
        float acc[2][4][4];
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i >> 4][i >> 2 & 3][i & 3] = 0.f;
        const int node = (g0 + lane) / a.H;      // of column `lane`
        float m_run = -INFINITY, z_run = 0.f;    // of column `lane`: the maximum so far, and the sum over this warp's rows

        for (int64_t p0 = p_begin; p0 < p_end; p0 += kRows, ++step) {
            const int nr = (int)min((int64_t)kRows, p_end - p0), buf = step & 1;
            const bool more = p0 + kRows < p_end;
            ok = mbar_wait(&sm.full[buf], step >> 1 & 1, &sm.abort_flag, a.err_word);
            // the rows are there; the step before is done with its weights and its rows
            ok = __syncthreads_and(ok);
            if (!ok) break;
            if (more) fetch_row(p0 + kRows);
            if (nr > 32 * (warp & 1)) partial_scores(sm, sm.tile[buf], warp, lane);
            __syncthreads();
            if (more) copy_row(buf ^ 1);
            // ---- softmax: warp w has rows 4 w .. 4 w + 3, lane = column
            float s[4];
            float m_new = -INFINITY, e_max = -INFINITY;  // of the scores, and of the weights' logarithms
            const float factor = sm.factor[lane];
            auto dot = [&](int r) -> float { return (sm.s[0][r][lane] + sm.s[1][r][lane]) + (sm.s[2][r][lane] + sm.s[3][r][lane]); };
            if (p0 + kRows <= seg.q.len && nc == kCols && *reinterpret_cast<const uint32_t *>(&sm.there[buf][4 * warp]) == 0x01010101u) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // every column attends every row
                    const int r = 4 * warp + j;
                    s[j] = dot(r) * (sm.scale[buf][r] * factor);
                    m_new = fmaxf(m_new, s[j]);
                    e_max = fmaxf(e_max, s[j] + sm.log_scale[buf][r]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * warp + j;
                    s[j] = -INFINITY;
                    if (r >= nr || !sm.there[buf][r] || lane >= nc) continue;
                    const int64_t draft = p0 + r - seg.q.len;  // the row's index in the draft
                    if (draft >= 0 && !tree_sees(a, seg.q.q0, node, (int)draft)) continue;
                    s[j] = dot(r) * (sm.scale[buf][r] * factor);
                    m_new = fmaxf(m_new, s[j]);
                    e_max = fmaxf(e_max, s[j] + sm.log_scale[buf][r]);
                }
            }
            atomicMax(&sm.m_max[buf][lane], float_order(m_new));
            atomicMax(&sm.e_max[buf][lane], float_order(e_max));
            // codes that a weight of 0 must not meet: NaN in drafted rows (a column that attends them has NaN weights)
            if (p0 + nr > seg.q.len)
                for (int i = tid; i < nr * (kKL / 16); i += kThreads) {
                    const int r = i / (kKL / 16);
                    if (p0 + r < seg.q.len) continue;
                    uint4 *p = reinterpret_cast<uint4 *>(&sm.tile[buf][r][16 * (i % (kKL / 16))]);
                    *p = make_uint4(without_nan(p->x), without_nan(p->y), without_nan(p->z), without_nan(p->w));
                }
            __syncthreads();  // (and the dot products are read: the weights take their place)
            m_new = fmaxf(m_run, order_float(sm.m_max[buf][lane]));
            e_max = order_float(sm.e_max[buf][lane]);
            if (warp == 1) sm.m_max[buf ^ 1][lane] = sm.e_max[buf ^ 1][lane] = float_order(-INFINITY);  // (read in the step before)
            const float ref = fabsf(m_new) <= kFar ? m_new : m_new == -INFINITY ? 0.f : NAN;
            const float corr = exp2f(m_run - ref);  // 0 before any row
            m_run = m_new;
            // the step's largest weight, of a column, times 2^(14 - top) in (2^13, 2^14]
            const float top = fminf(fmaxf(ceilf(e_max - ref), -110.f), 127.f), up = exp2f(14.f - top);
            if (warp == 0) {
                sm.corr[lane] = corr;
                sm.unit[lane] = exp2f(top - 14.f);
            }
            z_run *= corr;
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                float w[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // a row that the column does not attend weighs 0 whatever its scale holds
                    const float pr = s[j + k] == -INFINITY ? 0.f : exp2f(s[j + k] - ref);
                    z_run += pr;
                    w[k] = s[j + k] == -INFINITY ? 0.f : pr * up * sm.scale[buf][4 * warp + j + k];
                }
                uint32_t hi, lo;
                split_f16(w[0], w[1], hi, lo);
                const int r = 4 * (warp & 3) + j;  // rows r and r + 1 of 16: half of piece r / 2 % 4
                const int at = weight_offset(lane, 4 * (warp >> 2) + (r >> 1 & 3)) + 4 * (r >> 3);
                *reinterpret_cast<uint32_t *>(&sm.w[0][lane][at]) = hi;
                *reinterpret_cast<uint32_t *>(&sm.w[1][lane][at]) = lo;
            }
            __syncthreads();
            context(sm, sm.tile[buf], (nr + 15) / 16, warp, lane, acc);
        }
        __syncthreads();
        sm.z_part[warp][lane] = z_run;
        __syncthreads();
        float z = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) z += sm.z_part[w][lane];
        const bool whole = seg.first && seg.last;
        float *part = a.part + ((int64_t)blockIdx.x * 2 + (seg.first ? 1 : 0)) * tree_part_floats(kCols);
        if (!whole && warp == 0 && lane < nc) {
            part[kCols * kKL + lane] = tree_part_exponent(m_run, z);
            part[kCols * (kKL + 1) + lane] = z;
            part[kCols * (kKL + 2) + lane] = 0.f;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 16 * m + 8 * i + (lane >> 2);
                const float zc = __shfl_sync(0xffffffffu, z, c);
                if (c >= nc) continue;
                const float inv = !whole ? 1.f : zc == 0.f ? 0.f : 1.f / zc;
                {
                    const int d = 32 * warp + 8 * (lane & 3);
                    float o[8];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        o[n] = acc[m][n][2 * i] * inv;
                        o[4 + n] = acc[m][n][2 * i + 1] * inv;
                    }
                    if (whole && a.out_bf16) {
                        __nv_bfloat162 b[4];
#pragma unroll
                        for (int n = 0; n < 4; ++n) b[n] = __floats2bfloat162_rn(o[2 * n], o[2 * n + 1]);
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (q_base + c) * kKL + d) = *reinterpret_cast<uint4 *>(b);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>((whole ? static_cast<float *>(a.out) + (q_base + c) * kKL : part + c * kKL) + d);
                        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
    }
    if (bad_page && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
}

// Joins the parts of the cut groups: out = sum_p 2^(m_p - M) cl_p / (sum_p 2^(m_p - M) z_p + 2^-M sum_p n0_p) with
// M = max_p m_p.  (A set of NaN sums has m_p = +inf: its factor is NaN, the others' are 0.)
// A warp takes one column of one cut group and reads its parts in order: four dims a lane, of 128 or (kQuarters 4) all of
// them.  With a quarter each, and where the warps outnumber these (few columns, so many parts each), up to eight warps of a
// block share the parts.
constexpr int kMergeWarps = 8, kMergeBlocksPerSm = 4;

template <int kQuarters>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(TreeArgs a, int cols) {
    __shared__ float4 other[kMergeWarps][32];
    grid_dependency_wait();
    constexpr int kPer = 4 / kQuarters;  // tasks a column
    const int64_t tasks = (int64_t)a.sched->jobs * cols * kPer, warps = (int64_t)gridDim.x * kMergeWarps;
    int slices = kQuarters == 1 ? kMergeWarps : 1;
    while (slices > 1 && tasks * slices > warps) slices >>= 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp & (slices - 1);
    const int64_t stride = (int64_t)tree_part_floats(cols);
    for (int64_t first = (int64_t)blockIdx.x * (kMergeWarps / slices); first < tasks; first += warps / slices) {
        const int64_t task = first + warp / slices;
        float4 acc[kQuarters];
#pragma unroll
        for (int t = 0; t < kQuarters; ++t) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        float inv = 0.f;
        int64_t at = -1;
        if (task < tasks) {
            const TreeJob job = a.sched->job[task / (kPer * cols)];
            const int c = (int)(task / kPer) % cols, d = (int)(task % kPer) * 128 + lane * 4;
            if (c < job.cols) {
                at = (job.col0 + c) * kKL + d;
                // part p: the first CTA's second set, every other CTA's first
                const float *base = a.part + (int64_t)job.first * 2 * stride;
                auto part = [&](int p) { return base + (2 * p + (p == 0 ? 1 : 0)) * stride; };
                float m = -INFINITY;
                for (int p = lane; p < job.count; p += 32) m = fmaxf(m, part(p)[cols * kKL + c]);
                m = warp_max(m);
                float z = 0.f, n0 = 0.f;
                for (int p0 = 0; p0 < job.count; p0 += 32) {
                    float w = 0.f;
                    if (p0 + lane < job.count) {
                        const float *mine = part(p0 + lane);
                        const float mp = mine[cols * kKL + c], zp = mine[cols * (kKL + 1) + c];
                        n0 += mine[cols * (kKL + 2) + c];
                        if (mp != -INFINITY) w = exp2f(mp - m);
                        if (w != 0.f) z = fmaf(w, zp, z);
                    }
                    const int n = min(32, job.count - p0);
                    constexpr int kAhead = kQuarters == 1 ? 4 : 2;
                    for (int i = slice; i < n; i += kAhead * slices) {
                        float4 v[kAhead][kQuarters];
                        float wi[kAhead];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const int j = i + k * slices;
                            wi[k] = __shfl_sync(0xffffffffu, w, j & 31);
                            if (j >= n) wi[k] = 0.f;
                            const float4 *src = reinterpret_cast<const float4 *>(part(p0 + j) + c * kKL + d);
#pragma unroll
                            for (int t = 0; t < kQuarters; ++t)  // (a part that attended nothing may hold anything)
                                v[k][t] = wi[k] != 0.f ? src[32 * t] : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int k = 0; k < kAhead; ++k)
#pragma unroll
                            for (int t = 0; t < kQuarters; ++t) {
                                acc[t].x = fmaf(wi[k], v[k][t].x, acc[t].x);
                                acc[t].y = fmaf(wi[k], v[k][t].y, acc[t].y);
                                acc[t].z = fmaf(wi[k], v[k][t].z, acc[t].z);
                                acc[t].w = fmaf(wi[k], v[k][t].w, acc[t].w);
                            }
                    }
                }
                z = warp_sum(z);
                n0 = warp_sum(n0);
                if (n0 != 0.f && m != -INFINITY) z = fmaf(n0, exp2f(-m), z);
                inv = z == 0.f ? 0.f : 1.f / z;
            }
        }
        if (slices > 1) {  // (one quarter, and every task has its warps: the loop runs once)
            other[warp][lane] = acc[0];
            __syncthreads();
            for (int k = 1; k < slices; ++k) {
                const float4 o = other[(warp & ~(slices - 1)) + k][lane];
                acc[0].x += o.x;
                acc[0].y += o.y;
                acc[0].z += o.z;
                acc[0].w += o.w;
            }
        }
        if (slice != 0 || at < 0) continue;
#pragma unroll
        for (int t = 0; t < kQuarters; ++t) {
            const float4 o = make_float4(acc[t].x * inv, acc[t].y * inv, acc[t].z * inv, acc[t].w * inv);
            if (a.out_bf16) {
                __nv_bfloat162 v[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at + 128 * t) = *reinterpret_cast<uint2 *>(v);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at + 128 * t) = o;
            }
        }
    }
}

}  // namespace

int tree_ctas() {
    const int n = device_sm_count();
    return n < kMaxShares ? n : kMaxShares;
}

TreeWorkspace tree_workspace(int R, int H, int B, bool q_bf16) {
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    TreeWorkspace w;
    w.part = up(sizeof(TreeSched));
    w.images = w.part + up(q_bf16 ? tree_tc_part_bytes(tree_ctas()) : (size_t)tree_ctas() * 2 * tree_part_floats(kCols) * sizeof(float));
    w.total = w.images + (q_bf16 ? up(tree_tc_images(R, H, B)) : 0);
    return w;
}

// A launch whose prologue may overlap the end of the kernel before it; the kernel waits for that kernel's results.
template <class... Args>
static cudaError_t launch_behind(void (*kernel)(Args...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_merge(const TreeArgs &a, int cols, cudaStream_t st) {
    // Whole columns where the step may cut more of them than there are warps for quarters (known is only how many there are
    // at most): 32 x 13 tokens of 16 heads 78.4 us against 84.8, one token of 128 heads 25.1 against 19.7.
    const unsigned grid = (unsigned)a.ctas * kMergeBlocksPerSm;
    const int64_t columns = std::min((int64_t)a.R * a.H, (int64_t)a.ctas * cols);
    return launch_behind(4 * columns > (int64_t)grid * kMergeWarps ? tree_merge_kernel<4> : tree_merge_kernel<1>, grid, kMergeWarps * 32u, 0, st, a, cols);
}

cudaError_t launch_tree_f32(const TreeArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attn_tree_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    if ((e = launch_behind(tree_sched_kernel, 1, 288, 0, st, a)) != cudaSuccess) return e;
    if ((e = launch_behind(attn_tree_f32_kernel, (unsigned)a.ctas, kThreads, sizeof(Smem), st, a)) != cudaSuccess) return e;
    return launch_tree_merge(a, kCols, st);
}

}  // namespace kv8
