// attn_tree.cu -- attention of drafted tokens over a paged latent cache: the CUDA-core kernel for f32
// queries, and the merge of the groups that a share boundary cuts.
//
// For column (token i, head h) of a sequence and row t:  s_t = sm_scale * scale_t * q.e4m3(row_t),
// out = sum_t 2^((s_t - m) log2 e) scale_t e4m3(Lc_t) / sum_t 2^((s_t - m) log2 e), one pass over the rows with
// the running maximum m.  All columns of a sequence read the same rows.
#include "sm100.cuh"
#include "tree.cuh"

#include <math.h>

namespace kv8 {
namespace {

using namespace sm100;

constexpr int kCols = 32;      // (token, head) columns per block
constexpr int kUnit = 32;      // rows that the shares count
constexpr int kRows = 64;      // rows per step: two units where there are two
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTileStride = 592;           // bytes: 16-byte copies, and 148 words put eight consecutive rows into eight banks
constexpr int kQStride = kCols + 4;        // words: 16-byte loads, four-way instead of 32-way conflicts where it is filled
constexpr int kSlice = kRow / 4 / kWarps;  // words of a row that a warp's part of the scores covers
static_assert(kSlice * 4 * kWarps == kRow, "a row's words by warp");

struct Smem {
    float q[kRow][kQStride];               // the columns' queries, transposed
    uint8_t tile[2][kRows][kTileStride];   // this step's cache rows and the next's; rows that are left out are zero
    union {
        float s[kWarps][kRows][kCols];     // the warps' parts of the dot products
        float2 p[kRows][kCols];            // weights p * scale, twice each
    };
    int64_t row[kRows];                    // of the next step: cache row, or -1
    float scale[2][kRows];
    uint8_t there[2][kRows];
    float m_part[kWarps][kCols];
    float corr[kCols];
};

__global__ void __launch_bounds__(288) tree_sched_kernel(TreeArgs a) {
    __shared__ TreeScan scan;
    grid_dependency_wait();
    grid_launch_dependents();
    tree_schedule<kCols, kUnit, 1, 1>(a, scan);  // (two units a share instead of one: 46 -> 54 us for 4 x 5 tokens of 16 heads)
}

// 16 bytes global -> shared, zeros where `there` is false (the address must be valid all the same).
__device__ __forceinline__ void copy_16(void *dst, const void *src, bool there) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Dot products: warp w takes words 18 w .. 18 w + 17 of every row, so that a thread's 8 rows (rg + 8 j) by 8 columns
// (8 cg + ..) use a loaded value eight times; the parts are summed through shared memory.  kGroups groups of 8 rows.
template <int kGroups>
__device__ __forceinline__ void partial_scores(Smem &sm, const uint8_t (*tile)[kTileStride], int warp, int lane) {
    const int rg = lane & 7, cg = lane >> 3;
    uint64_t acc[kGroups][4];
#pragma unroll
    for (int j = 0; j < kGroups; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[j][c] = 0;
#pragma unroll 6
    for (int k = 0; k < kSlice; ++k) {
        const int w = warp * kSlice + k;
        ulonglong2 q[4][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[e][0] = *reinterpret_cast<const ulonglong2 *>(&sm.q[4 * w + e][8 * cg]);
            q[e][1] = *reinterpret_cast<const ulonglong2 *>(&sm.q[4 * w + e][8 * cg + 4]);
        }
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            float v[4];
            e4m3x4_to_f32(*reinterpret_cast<const uint32_t *>(&tile[rg + 8 * j][4 * w]), v[0], v[1], v[2], v[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t vv = f2_pack(v[e], v[e]);
                acc[j][0] = f2_fma(q[e][0].x, vv, acc[j][0]);
                acc[j][1] = f2_fma(q[e][0].y, vv, acc[j][1]);
                acc[j][2] = f2_fma(q[e][1].x, vv, acc[j][2]);
                acc[j][3] = f2_fma(q[e][1].y, vv, acc[j][3]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
        ulonglong2 *dst = reinterpret_cast<ulonglong2 *>(&sm.s[warp][rg + 8 * j][8 * cg]);
        dst[0] = make_ulonglong2(acc[j][0], acc[j][1]);
        dst[1] = make_ulonglong2(acc[j][2], acc[j][3]);
    }
}

// acc += weights x rows: a thread holds 8 columns (8 (warp % 4) + ..) by 8 latent dims, a row's weights are the same for
// a warp.  kDraft: a drafted row may hold NaN codes where a column does not attend it (weight 0).
template <bool kDraft>
__device__ __forceinline__ void context(const Smem &sm, const uint8_t (*tile)[kTileStride], int rows, int c0, int d0, uint64_t (*acc)[4]) {
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
        const uint2 b = *reinterpret_cast<const uint2 *>(&tile[r][d0]);
        float f[8];
        e4m3x4_to_f32(b.x, f[0], f[1], f[2], f[3]);
        e4m3x4_to_f32(b.y, f[4], f[5], f[6], f[7]);
        uint64_t v[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) v[d] = f2_pack(f[2 * d], f[2 * d + 1]);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sm.p[r][c0 + c]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint64_t wt = u ? w.y : w.x;
                if (kDraft && (uint32_t)wt << 1 == 0u) continue;  // (uniform: all lanes hold the same weight)
#pragma unroll
                for (int d = 0; d < 4; ++d) acc[c + u][d] = f2_fma(wt, v[d], acc[c + u][d]);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) attn_tree_simt_kernel(TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c0 = 8 * (warp & 3), d0 = 256 * (warp >> 2) + 8 * lane;  // this thread's part of the context
    bool bad_page = false;
    grid_dependency_wait();
    grid_launch_dependents();
    TreeWalk walk;
    walk.begin(a, blockIdx.x);
    TreeSegment seg;
    while (walk.next<kCols, kUnit>(a, seg)) {
        const int g0 = seg.g * kCols, nc = min(kCols, seg.q.n * a.H - g0);
        const int64_t q_base = (int64_t)seg.q.q0 * a.H + g0, rows_end = seg.q.len + seg.q.n;
        const int64_t p_begin = (int64_t)seg.t0 * kUnit, p_end = min((int64_t)seg.t1 * kUnit, rows_end);
        // the step's cache rows from position p0 on, of which the first 64 threads hold one each
        int64_t row = -1;
        float scale = 0.f;
        auto fetch_row = [&](int64_t p0) {
            row = -1;
            if (tid < kRows && p0 + tid < p_end) {
                row = tree_row(a, seg.b, p0 + tid);
                bad_page |= row < 0;
            }
            scale = row >= 0 ? __ldg(a.kv_scale + row) : 0.f;
        };
        auto store_row = [&](int buf) {
            if (tid < kRows) {
                sm.row[tid] = row;
                sm.scale[buf][tid] = scale;
                sm.there[buf][tid] = row >= 0;
            }
        };
        auto copy_rows = [&](int buf) {
            for (int i = tid; i < kRows * (kRow / 16); i += kThreads) {
                const int r = i / (kRow / 16), ch = i - r * (kRow / 16);
                const int64_t at = sm.row[r];
                copy_16(&sm.tile[buf][r][ch * 16], a.kv8 + (at >= 0 ? at : 0) * kRow + ch * 16, at >= 0);
            }
        };
        __syncthreads();  // the segment before is done with all of this
        fetch_row(p_begin);
        store_row(0);
        __syncthreads();
        copy_rows(0);
        for (int i = tid; i < kCols * (kRow / 4); i += kThreads) {
            // eight threads read 128 bytes of a column
            const int k4 = (i & 7) + 8 * (i / (8 * kCols)), c = (i >> 3) % kCols;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < nc)
                v = k4 < kKL / 4 ? __ldg(static_cast<const float4 *>(a.q_lat) + (q_base + c) * (kKL / 4) + k4)
                                 : __ldg(static_cast<const float4 *>(a.q_rope) + (q_base + c) * (kKR / 4) + (k4 - kKL / 4));
            sm.q[4 * k4][c] = tree_query(v.x);
            sm.q[4 * k4 + 1][c] = tree_query(v.y);
            sm.q[4 * k4 + 2][c] = tree_query(v.z);
            sm.q[4 * k4 + 3][c] = tree_query(v.w);
        }
        uint64_t acc[8][4];
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) acc[c][d] = 0;
        const int node = (g0 + lane) / a.H;      // of column `lane`
        float m_run = -INFINITY, z_run = 0.f;    // of column `lane`: the maximum so far, and the sum over this warp's rows

        int buf = 0;
        for (int64_t p0 = p_begin; p0 < p_end; p0 += kRows, buf ^= 1) {
            const int nr = (int)min((int64_t)kRows, p_end - p0);
            const bool more = p0 + kRows < p_end;
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();  // the rows are there; the step before is done with its weights and its rows
            if (more) fetch_row(p0 + kRows);
            if (nr > kUnit) partial_scores<kRows / 8>(sm, sm.tile[buf], warp, lane);
            else partial_scores<kUnit / 8>(sm, sm.tile[buf], warp, lane);
            if (more) store_row(buf ^ 1);
            __syncthreads();
            if (more) copy_rows(buf ^ 1);
            // ---- softmax: warp w has rows w + 8 j, lane = column
            float s[kRows / kWarps];
            float m_new = -INFINITY;
#pragma unroll
            for (int j = 0; j < kRows / kWarps; ++j) {
                const int r = warp + kWarps * j;
                s[j] = -INFINITY;
                if (r >= nr || !sm.there[buf][r] || lane >= nc) continue;
                const int64_t draft = p0 + r - seg.q.len;  // the row's index in the draft
                if (draft >= 0 && !tree_sees(a, seg.q.q0, node, (int)draft)) continue;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += sm.s[w][r][lane];
                s[j] = v * (sm.scale[buf][r] * a.sm_scale_log2);
                m_new = fmaxf(m_new, s[j]);
            }
            sm.m_part[warp][lane] = m_new;
            __syncthreads();  // (and the parts are read: the weights take their place)
            m_new = m_run;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m_new = fmaxf(m_new, sm.m_part[w][lane]);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            const float corr = exp2f(m_run - ref);  // 0 before any row
            m_run = m_new;
            if (warp == 0) sm.corr[lane] = corr;
            z_run *= corr;
#pragma unroll
            for (int j = 0; j < kRows / kWarps; ++j) {
                const int r = warp + kWarps * j;
                // a row that the column does not attend weighs 0 whatever its scale holds
                const float pr = s[j] == -INFINITY ? 0.f : exp2f(s[j] - ref);
                z_run += pr;
                const float w = s[j] == -INFINITY ? 0.f : pr * sm.scale[buf][r];
                sm.p[r][lane] = make_float2(w, w);
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float f = sm.corr[c0 + c];
                const uint64_t ff = f2_pack(f, f);
#pragma unroll
                for (int d = 0; d < 4; ++d) acc[c][d] = f2_mul(acc[c][d], ff);
            }
            if (p0 + nr > seg.q.len) context<true>(sm, sm.tile[buf], nr, c0, d0, acc);
            else context<false>(sm, sm.tile[buf], nr, c0, d0, acc);
        }
        __syncthreads();
        sm.m_part[warp][lane] = z_run;
        __syncthreads();
        float z = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) z += sm.m_part[w][lane];
        const bool whole = seg.first && seg.last;
        float *part = a.part + ((int64_t)blockIdx.x * 2 + (seg.first ? 1 : 0)) * tree_part_floats(kCols);
        if (!whole && warp == 0 && lane < nc) {
            part[kCols * kKL + lane] = tree_part_exponent(m_run, z);
            part[kCols * (kKL + 1) + lane] = z;
            part[kCols * (kKL + 2) + lane] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float zc = __shfl_sync(0xffffffffu, z, c0 + c);
            if (c0 + c >= nc) continue;
            const float inv = !whole ? 1.f : zc == 0.f ? 0.f : 1.f / zc;
            float o[8];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                f2_unpack(acc[c][d], o[2 * d], o[2 * d + 1]);
                o[2 * d] *= inv;
                o[2 * d + 1] *= inv;
            }
            if (whole && a.out_bf16) {
                __nv_bfloat162 h[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) h[d] = __floats2bfloat162_rn(o[2 * d], o[2 * d + 1]);
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (q_base + c0 + c) * kKL + d0) = *reinterpret_cast<uint4 *>(h);
            } else {
                float4 *dst = reinterpret_cast<float4 *>((whole ? static_cast<float *>(a.out) + (q_base + c0 + c) * kKL : part + (c0 + c) * kKL) + d0);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
            }
        }
    }
    if (bad_page && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
}

// Joins the parts of the cut groups: out = sum_p 2^(m_p - M) cl_p / (sum_p 2^(m_p - M) z_p + 2^-M sum_p n0_p) with
// M = max_p m_p.
// A warp takes one column of one cut group and reads its parts in order: four dims a lane, 128 or all of them.  Where the
// warps outnumber the columns (few columns, so many parts each), up to eight warps of a block share a quarter's parts.
constexpr int kMergeWarps = 8;

template <int kQuarters>
__device__ __forceinline__ void merge_columns(const TreeArgs &a, int cols, int slices, float4 (*other)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp & (slices - 1);
    constexpr int kPer = 4 / kQuarters;  // tasks a column
    const int64_t tasks = (int64_t)a.sched->jobs * cols * kPer, warps = (int64_t)gridDim.x * kMergeWarps;
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

__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(TreeArgs a, int cols) {
    __shared__ float4 other[kMergeWarps][32];
    grid_dependency_wait();
    const int64_t columns = (int64_t)a.sched->jobs * cols, warps = (int64_t)gridDim.x * kMergeWarps;
    int slices = kMergeWarps;
    while (slices > 1 && 4 * columns * slices > warps) slices >>= 1;
    if (4 * columns > warps) merge_columns<4>(a, cols, 1, other);
    else merge_columns<1>(a, cols, slices, other);
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
    return launch_behind(tree_merge_kernel, (unsigned)a.ctas * 4u, kMergeWarps * 32u, 0, st, a, cols);
}

cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attn_tree_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    if ((e = launch_behind(tree_sched_kernel, 1, 288, 0, st, a)) != cudaSuccess) return e;
    if ((e = launch_behind(attn_tree_simt_kernel, (unsigned)a.ctas, kThreads, sizeof(Smem), st, a)) != cudaSuccess) return e;
    return launch_tree_merge(a, kCols, st);
}

}  // namespace kv8
