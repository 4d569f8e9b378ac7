// attn_tree.cu -- attention of drafted tokens over a paged latent cache: the CUDA-core kernel for f32
// queries, and the merge of the groups that a share boundary cuts.
//
// For column (token i, head h) of a sequence and row t:  s_t = sm_scale * scale_t * q.e4m3(row_t),
// out = sum_t 2^((s_t - m) log2 e) scale_t e4m3(Lc_t) / sum_t 2^((s_t - m) log2 e), one pass over the rows with
// the running maximum m.  All columns of a sequence read the same rows.
#include "tree.cuh"

#include <math.h>

namespace kv8 {
namespace {

constexpr int kCols = 32;      // (token, head) columns per block
constexpr int kRows = 64;      // rows per tile
constexpr int kThreads = 256;  // 8 warps
constexpr int kTileStride = kRow + 4;  // 145 words: odd, so row-per-lane reads are conflict-free
constexpr int kSStride = kCols + 1;

struct Smem {
    float q[kCols][kRow];             // the columns' queries (f32)
    uint8_t tile[kRows][kTileStride]; // current cache tile; rows that are left out are zero
    float s[kRows][kSStride];         // scores (log2 domain)
    float p[kRows][kCols];            // weights p * scale, row-major for broadcast reads
    float rscale[kRows];
    int64_t row[kRows];               // cache row, or -1
    float m_run[kCols], z_run[kCols], corr[kCols];
    int node[kCols];                  // the column's token
};

__global__ void __launch_bounds__(288) tree_sched_kernel(TreeArgs a) {
    __shared__ TreeScan scan;
    tree_schedule<kCols, kRows, 1>(a, scan);
}

__global__ void __launch_bounds__(kThreads, 1) attn_tree_simt_kernel(TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad_page = false;
    TreeWalk walk;
    walk.begin(a, blockIdx.x);
    TreeSegment seg;
    while (walk.next<kCols, kRows>(a, seg)) {
        const int c0 = seg.g * kCols, nc = min(kCols, seg.q.n * a.H - c0);
        const int64_t q_base = (int64_t)seg.q.q0 * a.H + c0, rows_end = seg.q.len + seg.q.n;
        __syncthreads();
        for (int i = tid; i < kCols * kRow; i += kThreads) {
            const int c = i / kRow, k = i - c * kRow;
            float v = 0.f;
            if (c < nc) {
                const int64_t at = k < kKL ? (q_base + c) * kKL + k : (q_base + c) * kKR + (k - kKL);
                const void *base = k < kKL ? a.q_lat : a.q_rope;
                v = static_cast<const float *>(base)[at];
            }
            sm.q[c][k] = v;
        }
        if (tid < kCols) {
            sm.m_run[tid] = -INFINITY;
            sm.z_run[tid] = 0.f;
            sm.node[tid] = (c0 + tid) / a.H;
        }
        float acc[kCols][2];
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c][0] = acc[c][1] = 0.f;

        for (int t = seg.t0; t < seg.t1; ++t) {
            const int64_t p0 = (int64_t)t * kRows;
            __syncthreads();  // the previous tile is consumed
            if (tid < kRows) {
                const int64_t pos = p0 + tid;
                int64_t row = -1;
                if (pos < rows_end) {
                    row = tree_row(a, seg.b, pos);
                    bad_page |= row < 0;
                }
                sm.row[tid] = row;
                sm.rscale[tid] = row >= 0 ? __ldg(a.kv_scale + row) : 0.f;
            }
            __syncthreads();
            for (int c = tid; c < kRows * (kRow / 16); c += kThreads) {
                const int r = c / (kRow / 16), col = c - r * (kRow / 16);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (sm.row[r] >= 0) v = __ldg(reinterpret_cast<const uint4 *>(a.kv8 + sm.row[r] * kRow) + col);
                uint32_t *dst = reinterpret_cast<uint32_t *>(&sm.tile[r][col * 16]);
                dst[0] = v.x;
                dst[1] = v.y;
                dst[2] = v.z;
                dst[3] = v.w;
            }
            __syncthreads();
            // ---- scores: warp w -> columns (w&3)*8..+7, rows (w>>2)*32 + lane
            {
                const int g = warp & 3, r = (warp >> 2) * 32 + lane;
                float s8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) s8[j] = 0.f;
                const uint32_t *rw = reinterpret_cast<const uint32_t *>(&sm.tile[r][0]);
#pragma unroll 4
                for (int k4 = 0; k4 < kRow / 4; ++k4) {
                    float e0, e1, e2, e3;
                    e4m3x4_to_f32(rw[k4], e0, e1, e2, e3);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 q4 = *reinterpret_cast<const float4 *>(&sm.q[g * 8 + j][k4 * 4]);
                        s8[j] = fmaf(q4.x, e0, s8[j]);
                        s8[j] = fmaf(q4.y, e1, s8[j]);
                        s8[j] = fmaf(q4.z, e2, s8[j]);
                        s8[j] = fmaf(q4.w, e3, s8[j]);
                    }
                }
                const float f = sm.rscale[r] * a.sm_scale_log2;
                const bool ok = sm.row[r] >= 0;
                const int64_t draft = p0 + r - seg.q.len;  // the row's index in the draft
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = g * 8 + j;
                    const bool sees = ok && c < nc && (draft < 0 || tree_sees(a, seg.q.q0, sm.node[c], (int)draft));
                    sm.s[r][c] = sees ? s8[j] * f : -INFINITY;
                }
            }
            __syncthreads();
            // ---- online softmax: thread -> column tid/8, rows (tid%8)*8..+7
            {
                const int c = tid >> 3, sub = tid & 7;
                float mloc = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; ++i) mloc = fmaxf(mloc, sm.s[sub * 8 + i][c]);
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) mloc = fmaxf(mloc, __shfl_xor_sync(0xffffffffu, mloc, o));
                const float m_old = sm.m_run[c], m_new = fmaxf(m_old, mloc);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                const float corr = exp2f(m_old - ref);  // 0 before any row
                float zloc = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = sub * 8 + i;
                    const float s = sm.s[r][c];
                    // a row that the column does not attend weighs 0 whatever its scale holds
                    const float pr = s == -INFINITY ? 0.f : exp2f(s - ref);
                    zloc += pr;
                    sm.p[r][c] = s == -INFINITY ? 0.f : pr * sm.rscale[r];
                }
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) zloc += __shfl_xor_sync(0xffffffffu, zloc, o);
                __syncwarp();
                if (sub == 0) {
                    sm.m_run[c] = m_new;
                    sm.z_run[c] = sm.z_run[c] * corr + zloc;
                    sm.corr[c] = corr;
                }
            }
            __syncthreads();
            // ---- context: thread -> latent dims 2*tid, 2*tid+1
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                acc[c][0] *= sm.corr[c];
                acc[c][1] *= sm.corr[c];
            }
            const int nr = (int)min((int64_t)kRows, rows_end - p0);
            const bool drafted = p0 + kRows > seg.q.len;
            for (int r = 0; r < nr; ++r) {
                float v0, v1;
                e4m3x2_to_f32(*reinterpret_cast<const uint16_t *>(&sm.tile[r][2 * tid]), v0, v1);
#pragma unroll
                for (int c4 = 0; c4 < kCols / 4; ++c4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(&sm.p[r][c4 * 4]);
                    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        // a drafted row may hold NaN codes where this column does not attend it
                        const bool skip = drafted && w[u] == 0.f;
                        acc[c4 * 4 + u][0] = skip ? acc[c4 * 4 + u][0] : fmaf(w[u], v0, acc[c4 * 4 + u][0]);
                        acc[c4 * 4 + u][1] = skip ? acc[c4 * 4 + u][1] : fmaf(w[u], v1, acc[c4 * 4 + u][1]);
                    }
                }
            }
        }
        __syncthreads();
        if (seg.first && seg.last) {
            for (int c = 0; c < nc; ++c) {
                const float z = sm.z_run[c], inv = z == 0.f ? 0.f : 1.f / z;
                const int64_t at = (q_base + c) * kKL + 2 * tid;
                if (a.out_bf16)
                    *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
                        __floats2bfloat162_rn(acc[c][0] * inv, acc[c][1] * inv);
                else
                    *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) =
                        make_float2(acc[c][0] * inv, acc[c][1] * inv);
            }
        } else {
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (seg.first ? 1 : 0)) * tree_part_floats(kCols);
            for (int c = 0; c < nc; ++c)
                *reinterpret_cast<float2 *>(part + c * kKL + 2 * tid) = make_float2(acc[c][0], acc[c][1]);
            if (tid < nc) {
                part[kCols * kKL + tid] = sm.m_run[tid];
                part[kCols * (kKL + 1) + tid] = sm.z_run[tid];
                part[kCols * (kKL + 2) + tid] = 0.f;
            }
        }
    }
    if (bad_page && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
}

// Joins the parts of the cut groups: out = sum_p 2^(m_p - M) cl_p / (sum_p 2^(m_p - M) z_p + 2^-M sum_p n0_p) with
// M = max_p m_p.
// A warp takes 128 dims of one column of one cut group, four dims a lane, and reads its parts in order.  Where the warps
// outnumber these (few columns, so many parts each), up to eight warps of a block share the parts.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(TreeArgs a, int cols) {
    __shared__ float4 other[kMergeWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t tasks = (int64_t)a.sched->jobs * cols * 4, warps = (int64_t)gridDim.x * kMergeWarps;
    int slices = kMergeWarps;
    while (slices > 1 && tasks * slices > warps) slices >>= 1;
    const int slice = warp & (slices - 1);
    const int64_t stride = (int64_t)tree_part_floats(cols), positions = tree_positions(a.max_pages, a.page_shift);
    for (int64_t first = (int64_t)blockIdx.x * (kMergeWarps / slices); first < tasks; first += warps / slices) {
        const int64_t task = first + warp / slices;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float inv = 0.f;
        int64_t at = -1;
        if (task < tasks) {
            const TreeJob job = a.sched->job[task / (4 * cols)];
            const int c = (int)(task >> 2) % cols, d = ((int)task & 3) * 128 + lane * 4;
            const TreeSeq q = tree_seq(a.q_start, a.lens, job.b, a.R, positions);
            const int64_t col = (int64_t)job.g * cols + c;
            if (col < (int64_t)q.n * a.H) {
                at = ((int64_t)q.q0 * a.H + col) * kKL + d;
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
                        n0 += mine[cols * (kKL + 2) + c];
                        const float mp = mine[cols * kKL + c];
                        if (mp != -INFINITY) w = exp2f(mp - m);
                        if (w != 0.f) z = fmaf(w, mine[cols * (kKL + 1) + c], z);
                    }
                    const int n = min(32, job.count - p0);
                    for (int i = slice; i < n; i += 4 * slices) {
                        float4 v[4];
                        float wi[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int j = i + k * slices;
                            wi[k] = __shfl_sync(0xffffffffu, w, j & 31);
                            if (j >= n) wi[k] = 0.f;
                            // (a part that attended nothing may hold anything)
                            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (wi[k] != 0.f) v[k] = *reinterpret_cast<const float4 *>(part(p0 + j) + c * kKL + d);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            acc.x = fmaf(wi[k], v[k].x, acc.x);
                            acc.y = fmaf(wi[k], v[k].y, acc.y);
                            acc.z = fmaf(wi[k], v[k].z, acc.z);
                            acc.w = fmaf(wi[k], v[k].w, acc.w);
                        }
                    }
                }
                z = warp_sum(z);
                n0 = warp_sum(n0);
                if (n0 != 0.f && m != -INFINITY) z = fmaf(n0, exp2f(-m), z);
                inv = z == 0.f ? 0.f : 1.f / z;
            }
        }
        if (slices > 1) {  // (then every task has its warps: the loop runs once)
            other[warp][lane] = acc;
            __syncthreads();
            for (int k = 1; k < slices; ++k) {
                const float4 o = other[(warp & ~(slices - 1)) + k][lane];
                acc.x += o.x;
                acc.y += o.y;
                acc.z += o.z;
                acc.w += o.w;
            }
        }
        if (slice == 0 && at >= 0) {
            acc.x *= inv;
            acc.y *= inv;
            acc.z *= inv;
            acc.w *= inv;
            if (a.out_bf16) {
                __nv_bfloat162 v[2] = {__floats2bfloat162_rn(acc.x, acc.y), __floats2bfloat162_rn(acc.z, acc.w)};
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = *reinterpret_cast<uint2 *>(v);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = acc;
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

cudaError_t launch_tree_merge(const TreeArgs &a, int cols, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas * 4u);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_merge_kernel, a, cols);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attn_tree_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    tree_sched_kernel<<<1, 288, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    attn_tree_simt_kernel<<<(unsigned)a.ctas, kThreads, sizeof(Smem), st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_tree_merge(a, kCols, st);
}

}  // namespace kv8
