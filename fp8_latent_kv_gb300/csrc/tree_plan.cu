// tree_plan.cu -- the bookkeeping around a step of drafted tokens over a paged cache: page lists and slot
// maps (kv8_page_plan), tree bits and positions (kv8_tree_mask), and the move of the accepted branch's rows
// (kv8_tree_commit).
#include "tree.cuh"

namespace kv8 {
namespace {

// ------------------------------------------------------------------------------------------------------------
// kv8_page_plan.  want_b = ceil((len_b + n_b) / page); surplus_b = max(0, have_b - want_b) pages go back,
// need_b = max(0, want_b - have_b) are taken; the places are exclusive prefix sums over the sequences, so the
// result does not depend on the order in which warps run.
// One thread-block cluster: every CTA computes all prefix sums for itself (a few words per sequence), returned
// pages are written, the cluster meets, pages are taken from the list and the slots written.  A second launch in place of the cluster's barrier would cost more than all of it.
// ------------------------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;  // (one CTA: 4.0 us as well for 4 sequences, 6.2 against 4.8 for 256, 40 against 10 for 4096)
constexpr int kPlanPer = KV8_MAX_SEQS / kPlanThreads;  // sequences per thread in the scans
// All of the kernel's shared memory is the launch's, so that its size alone says which launches need the larger limit: the
// warps' sums, then four words a sequence.
constexpr size_t kPlanSums = 32 * 2 * sizeof(int64_t);
constexpr size_t plan_smem_bytes(int B) { return kPlanSums + (size_t)B * 4 * sizeof(int32_t); }
constexpr size_t kDefaultSmem = 48 * 1024;  // what a launch may have without asking

struct PlanArgs {
    int B, R, page_shift, max_pages, free_cap;
    const int32_t *lens, *q_start;
    int32_t *n_pages, *table, *free_list, *n_free;
    int64_t *slots;
    int *err_word;
};

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PlanArgs a) {
    extern __shared__ __align__(16) unsigned char plan_smem[];
    int64_t(*const wsum)[2] = reinterpret_cast<int64_t(*)[2]>(plan_smem);
    int32_t *have = reinterpret_cast<int32_t *>(plan_smem + kPlanSums), *want = have + a.B, *spre = want + a.B, *npre = spre + a.B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t positions = 0x7fffffff;  // a table that is too narrow is a page error, not a bad number
    int err = 0;
    // ---- wants, and their prefix sums (64 bits: 4096 sequences of up to 2^27 pages)
    int64_t s_mine = 0, n_mine = 0;
    int32_t s_loc[kPlanPer], n_loc[kPlanPer];
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * per;
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        s_loc[k] = n_loc[k] = 0;
        const int b = b0 + k;
        if (k < per && b < a.B) {
            const TreeSeq q = tree_seq(a.q_start, a.lens, b, a.R, positions);
            const int h = a.n_pages[b];
            int w = -1;  // -1: not possible, -2: more pages than the table holds
            if (q.n < 0 || h < 0 || h > a.max_pages) err |= KV8_ERR_INDEX;
            else {
                const int64_t p = (q.len + q.n + ((int64_t)1 << a.page_shift) - 1) >> a.page_shift;
                if (p > a.max_pages) {
                    err |= KV8_ERR_PAGES;
                    w = -2;
                } else {
                    w = (int)p;
                    s_loc[k] = max(0, h - w);
                    n_loc[k] = max(0, w - h);
                }
            }
            have[b] = h;
            want[b] = w;
            s_mine += s_loc[k];
            n_mine += n_loc[k];
        }
    }
    int64_t si = s_mine, ni = n_mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, si, o), y = __shfl_up_sync(0xffffffffu, ni, o);
        if (lane >= o) {
            si += x;
            ni += y;
        }
    }
    if (lane == 31) {
        wsum[warp][0] = si;
        wsum[warp][1] = ni;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t x = wsum[lane][0], y = wsum[lane][1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        wsum[lane][0] = x;
        wsum[lane][1] = y;
    }
    const bool back = __syncthreads_or(err & KV8_ERR_INDEX) &&
                      tree_goes_back(a.q_start, a.lens, min(b0, a.B), min(b0 + per, a.B), a.R, positions);
    const int64_t S = wsum[31][0];
    const int F0 = *a.n_free;
    // the list itself is not possible, or rows would have two slots
    const bool broken = back || F0 < 0 || F0 > a.free_cap || F0 + S > a.free_cap;
    const int64_t top = F0 + S;
    int64_t sp = si - s_mine + (warp ? wsum[warp - 1][0] : 0), np = ni - n_mine + (warp ? wsum[warp - 1][1] : 0);
#pragma unroll
    for (int k = 0; k < kPlanPer; ++k) {
        const int b = b0 + k;
        if (k < per && b < a.B) {
            spre[b] = (int32_t)min(sp, (int64_t)0x7fffffff);
            npre[b] = (int32_t)min(np, (int64_t)0x7fffffff);
            sp += s_loc[k];
            np += n_loc[k];
        }
    }
    if (broken) err |= KV8_ERR_INDEX;
    __syncthreads();
    // Eight lanes for each sequence: what a sequence needs is a chain of loads, so that a warp's four take the time of one
    // (2048 sequences: 6.7 us; a warp each: 11.8).
    const int sub = lane & 7;
    const uint32_t group = 0xffu << (lane & ~7);
    const int w0 = (blockIdx.x * kPlanThreads + tid) >> 3, w_all = kPlanCtas * kPlanThreads >> 3;
    // ---- returned pages: the k-th of sequence b stands spre + k places below the new top
    if (!broken)
        for (int b = w0; b < a.B; b += w_all) {
            const int w = want[b];
            const int surplus = w < 0 ? 0 : have[b] - w;
            for (int k = sub; k < surplus; k += 8)
                a.free_list[top - 1 - ((int64_t)spre[b] + k)] = a.table[(int64_t)b * a.max_pages + w + k];
        }
    cluster_sync_all();  // every count has been read and every returned page written
    // ---- taken pages, the new counts, the slots
    int64_t took = 0;
    if (!broken)
        for (int b = w0; b < a.B; b += w_all) {
            const int w = want[b];
            if (w == -1) continue;
            const int h = have[b], need = w < 0 ? 0 : max(0, w - h);
            const bool ok = w >= 0 && (need == 0 || (int64_t)npre[b] + need <= top);
            int32_t *row = a.table + (int64_t)b * a.max_pages;
            if (ok) {
                for (int k = sub; k < need; k += 8)
                    row[h + k] = *(volatile int32_t *)(a.free_list + (top - 1 - ((int64_t)npre[b] + k)));
                if (sub == 0) a.n_pages[b] = w;
            } else if (sub == 0 && w >= 0) {
                err |= KV8_ERR_PAGES;
            }
            __syncwarp(group);
            const int q0 = a.q_start[b], n = a.q_start[b + 1] - q0;
            const int64_t len = a.lens[b];
            for (int i = sub; i < n; i += 8) {
                int64_t slot = -1;
                if (ok) {
                    const int64_t pos = len + i;
                    const int64_t page = *(volatile int32_t *)(row + (pos >> a.page_shift));
                    slot = (page << a.page_shift) + (pos & (((int64_t)1 << a.page_shift) - 1));
                }
                a.slots[q0 + i] = slot;
            }
        }
    // ---- what is left of the list: the wants that were met are a prefix of the sequences that want any
    if (blockIdx.x == 0 && !broken) {
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const int b = b0 + k;
            if (k < per && b < a.B && n_loc[k] > 0 && (int64_t)npre[b] + n_loc[k] <= top) took += n_loc[k];
        }
        __syncthreads();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) took += __shfl_xor_sync(0xffffffffu, took, o);
        if (lane == 0) wsum[warp][0] = took;
        __syncthreads();
        if (tid == 0) {
            int64_t t = 0;
            for (int w = 0; w < 32; ++w) t += wsum[w][0];
            *a.n_free = (int32_t)(top - t);
        }
    }
    if (err && a.err_word) atomicOr(a.err_word, err);
}

// ------------------------------------------------------------------------------------------------------------
// kv8_tree_mask.  Pointer doubling: after k rounds token i's bits hold its 2^k nearest ancestors (itself
// included) and ptr[i] the next one above them.  One block per sequence, one thread per token, W words each.
// 1024 sequences of 64 tokens take 2.4 us, eight of 16 1.8: a launch, and a few loads' latency.
// ------------------------------------------------------------------------------------------------------------
template <int W>
__global__ void __launch_bounds__(32 * W) tree_mask_kernel(const int32_t *q_start, const int32_t *lens, int R,
                                                           const int32_t *parent, uint32_t *mask, int32_t *position,
                                                           int *err_word) {
    __shared__ uint32_t bits[32 * W][W];
    __shared__ int ptr[32 * W];
    const int b = blockIdx.x, i = threadIdx.x;
    const TreeSeq q = tree_seq(q_start, lens, b, R, 0x7fffffff);
    if (q.n < 0 || q.n > 32 * W) {
        if (i == 0 && err_word) atomicOr(err_word, (int)KV8_ERR_INDEX);
        return;
    }
    uint32_t mine[W];
#pragma unroll
    for (int w = 0; w < W; ++w) mine[w] = (i >> 5) == w ? 1u << (i & 31) : 0u;
    int up = -1;
    if (i < q.n) {
        up = __ldg(parent + q.q0 + i);
        if (up < -1 || up >= i) {
            up = -1;
            if (err_word) atomicOr(err_word, (int)KV8_ERR_INDEX);
        }
    }
    for (int s = 1; s < q.n; s <<= 1) {
#pragma unroll
        for (int w = 0; w < W; ++w) bits[i][w] = mine[w];
        ptr[i] = up;
        __syncthreads();
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < W; ++w) mine[w] |= bits[up][w];
            up = ptr[up];
        }
        __syncthreads();
    }
    if (i < q.n) {
        int depth = -1;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            mask[(int64_t)(q.q0 + i) * W + w] = mine[w];
            depth += __popc(mine[w]);
        }
        if (position) position[q.q0 + i] = (lens ? __ldg(lens + b) : 0) + depth;
    }
}

// ------------------------------------------------------------------------------------------------------------
// kv8_tree_commit.  A source row stands at accept[k] >= k, so a row that is written by one round of the loop
// (destinations k of the round) is never a source of a later one; within a round all rows are read before
// any is written.  Six rows of 256 sequences in 61 layers (54 MB read and as many written, which stay in L2 between
// the measured calls) take 14.6 us, one launch and five loads in a chain 2.4.
// ------------------------------------------------------------------------------------------------------------
constexpr int kCommitThreads = 288;  // 36 16-byte pieces of a row, eight rows at once
constexpr int kCommitRows = 8;
constexpr int kCommitLayers = 4;  // that a block moves at once

struct CommitArgs {
    int B, max_accept, layers, per_block, max_pages, page_shift;
    const int32_t *q_start, *lens, *accept, *n_accept, *table;
    uint8_t *kv8;
    float *kv_scale;
    int64_t cache_rows;
    int32_t *new_lens;
    int *err_word;
};

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(CommitArgs a) {
    __shared__ int64_t src[KV8_MAX_TREE], dst[KV8_MAX_TREE];
    const int b = blockIdx.x, first = blockIdx.y * a.per_block, tid = threadIdx.x;
    const TreeSeq q = tree_seq(a.q_start, a.lens, b, 0x7fffffff, tree_positions(a.max_pages, a.page_shift));
    const int m = __ldg(a.n_accept + b);
    bool ok = q.n >= 0 && m >= 0 && m <= a.max_accept && m <= q.n;
    if (ok && tid < m) {
        const int32_t *acc = a.accept + (int64_t)b * a.max_accept;
        const int x = __ldg(acc + tid), before = tid ? __ldg(acc + tid - 1) : -1;
        auto row = [&](int64_t t) -> int64_t {
            const int64_t page = __ldg(a.table + (int64_t)b * a.max_pages + (t >> a.page_shift));
            const int64_t r = (page << a.page_shift) + (t & (((int64_t)1 << a.page_shift) - 1));
            return page >= 0 && r < a.cache_rows ? r : -1;
        };
        if (x <= before || x >= q.n) ok = false;
        else {
            src[tid] = row(q.len + x);
            dst[tid] = row(q.len + tid);
            ok = src[tid] >= 0 && dst[tid] >= 0;
        }
    }
    ok = __syncthreads_and(ok);
    if (first == 0 && tid == 0) {
        a.new_lens[b] = __ldg(a.lens + b) + (ok ? m : 0);
        if (!ok && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
    }
    if (!ok) return;
    const int piece = tid % 36, sub = tid / 36, end = min(first + a.per_block, a.layers);
    for (int k0 = 0; k0 < m; k0 += kCommitRows) {
        const int k = k0 + sub;
        const bool moves = k < m && src[k] != dst[k];
        for (int l0 = first; l0 < end; l0 += kCommitLayers) {
            uint4 v[kCommitLayers];
            float s[kCommitLayers];
#pragma unroll
            for (int l = 0; l < kCommitLayers; ++l) {
                v[l] = make_uint4(0u, 0u, 0u, 0u);
                s[l] = 0.f;
                if (!moves || l0 + l >= end) continue;
                const int64_t at = (int64_t)(l0 + l) * a.cache_rows + src[k];
                v[l] = *(reinterpret_cast<const uint4 *>(a.kv8 + at * kRow) + piece);
                if (piece == 0) s[l] = a.kv_scale[at];
            }
            __syncthreads();  // a row may be another's place
#pragma unroll
            for (int l = 0; l < kCommitLayers; ++l) {
                if (!moves || l0 + l >= end) continue;
                const int64_t at = (int64_t)(l0 + l) * a.cache_rows + dst[k];
                *(reinterpret_cast<uint4 *>(a.kv8 + at * kRow) + piece) = v[l];
                if (piece == 0) a.kv_scale[at] = s[l];
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_page_plan(int B, const int32_t *lens, const int32_t *q_start, int R, int page_shift, int max_pages,
                             int32_t *n_pages, int32_t *table, int32_t *free_list, int free_cap, int32_t *n_free,
                             int64_t *slots, int *err_word, cudaStream_t st) {
    PlanArgs a{B, R, page_shift, max_pages, free_cap, lens, q_start, n_pages, table, free_list, n_free, slots, err_word};
    const size_t smem = plan_smem_bytes(B);
    cudaError_t e;
    if (smem > kDefaultSmem && (e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                         (int)plan_smem_bytes(KV8_MAX_SEQS))) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPlanCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, page_plan_kernel, a)) != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t launch_tree_mask(int B, const int32_t *q_start, const int32_t *lens, int R, const int32_t *parent,
                             uint32_t *mask, int W, int32_t *position, int *err_word, cudaStream_t st) {
    const dim3 grid((unsigned)B);
#define KV8_MASK_CASE(w) \
    case w: tree_mask_kernel<w><<<grid, 32 * w, 0, st>>>(q_start, lens, R, parent, mask, position, err_word); break
    switch (W) {
        KV8_MASK_CASE(1);
        KV8_MASK_CASE(2);
        KV8_MASK_CASE(3);
        KV8_MASK_CASE(4);
        KV8_MASK_CASE(5);
        KV8_MASK_CASE(6);
        KV8_MASK_CASE(7);
        KV8_MASK_CASE(8);
        default: return cudaErrorInvalidValue;
    }
#undef KV8_MASK_CASE
    return cudaGetLastError();
}

cudaError_t launch_tree_commit(int B, const int32_t *q_start, const int32_t *lens, const int32_t *accept,
                               const int32_t *n_accept, int max_accept, int layers, uint8_t *kv8, float *kv_scale,
                               int64_t cache_rows, const int32_t *table, int max_pages, int page_shift,
                               int32_t *new_lens, int *err_word, cudaStream_t st) {
    // One wave of blocks, each with the same number of layers: 64 sequences in 64 layers 5.9 us, with a layer each 11.7.
    const int64_t wave = (int64_t)device_sm_count() * (2048 / kCommitThreads);
    const int per = (int)(((int64_t)B * layers + wave - 1) / wave), blocks = (layers + per - 1) / per;
    CommitArgs a{B,     max_accept, layers,   per,        max_pages, page_shift, q_start, lens, accept, n_accept, table,
                 kv8, kv_scale,   cache_rows, new_lens, err_word};
    tree_commit_kernel<<<dim3((unsigned)B, (unsigned)blocks), kCommitThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kv8
