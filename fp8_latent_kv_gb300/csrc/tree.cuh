// tree.cuh -- drafted tokens over a paged cache: the argument block, the ragged batch's bookkeeping and the
// work shares that the tree attention's kernels use.
#pragma once

#include "internal.h"

namespace kv8 {

// A sequence's step, checked: n < 0 means that its numbers are not possible and it is skipped.
struct TreeSeq {
    int q0, n;      // its drafted tokens are the step's rows q0 .. q0 + n - 1
    int64_t len;    // rows of its context
};

__device__ __forceinline__ TreeSeq tree_seq(const int32_t *q_start, const int32_t *lens, int b, int R, int64_t positions) {
    TreeSeq s;
    const int q0 = __ldg(q_start + b), q1 = __ldg(q_start + b + 1);
    s.q0 = q0;
    s.len = lens ? __ldg(lens + b) : 0;
    const int64_t n = (int64_t)q1 - q0;
    const bool ok = q0 >= 0 && n >= 0 && n <= KV8_MAX_TREE && q1 <= R && s.len >= 0 && s.len + n <= positions;
    s.n = ok ? (int)n : -1;
    return s;
}

// Positions that a table row of max_pages pages holds, as far as 32-bit lengths reach.
__host__ __device__ __forceinline__ int64_t tree_positions(int max_pages, int page_shift) {
    const int64_t p = (int64_t)max_pages << page_shift;
    return p < 0x7fffffff ? p : 0x7fffffff;
}

// Work shares.  A group is kCols consecutive (token, head) columns of one sequence (column = token * H +
// head); its work is the ceil(rows / kRows) row tiles of the sequence.  All groups' tiles in order (sequence,
// group, tile) are one line of W units, cut into `shares` equal pieces, one for each CTA: whatever the
// lengths, no CTA has more than one tile more than another.  A group that one CTA walks from its first tile
// to its last is finished there; one that a cut falls into leaves one partial set for each CTA that walks a
// part of it, and the merge joins them.
struct TreeShare {
    int64_t unit;  // first unit of the share
    int b, g, t;   // where that is
    int pad;
};
struct TreeJob {  // a group that was cut
    int b, g;
    int first, count;  // the CTAs first .. first + count - 1 hold its parts
};
constexpr int kMaxShares = 512;
struct TreeSched {
    int shares;  // CTAs that have work
    int jobs;
    int pad[2];
    TreeShare share[kMaxShares + 1];  // [shares] ends the last one
    TreeJob job[kMaxShares];
    int64_t unit0[KV8_MAX_SEQS + 1];  // units before sequence b
};

struct TreeArgs {
    const void *q_lat, *q_rope;  // [R][H][512], [R][H][64]
    int q_bf16;
    int R, H, B;
    const int32_t *q_start, *lens;
    const uint32_t *mask;        // [R][mask_words], or null: a chain
    int mask_words;
    const uint8_t *kv8;
    const float *kv_scale;
    int64_t cache_rows;
    const int32_t *table;        // [B][max_pages]
    int max_pages, page_shift;
    float sm_scale_log2;
    void *out;
    int out_bf16;
    int *err_word;
    int ctas;                    // shares asked for
    TreeSched *sched;
    float *part;                 // partial sets: [ctas][2] x { cl [cols][512], m [cols], z [cols], n0 [cols] }
};

// A partial set: cl and z relative to 2^m, and n0, the weight (relative to 2^0) of rows that only count in the sum.
__host__ __device__ constexpr size_t tree_part_floats(int cols) { return (size_t)cols * (kKL + 3); }

// Cache row of position t of sequence b, or -1 where its page is outside the cache.
__device__ __forceinline__ int64_t tree_row(const TreeArgs &a, int b, int64_t t) {
    const int64_t page = __ldg(a.table + (int64_t)b * a.max_pages + (t >> a.page_shift));
    const int64_t row = (page << a.page_shift) + (t & (((int64_t)1 << a.page_shift) - 1));
    return page >= 0 && row < a.cache_rows ? row : -1;
}

// Whether drafted token i of a sequence whose rows begin at q0 attends drafted token j.
__device__ __forceinline__ bool tree_sees(const TreeArgs &a, int q0, int i, int j) {
    if (!a.mask) return j <= i;
    if ((j >> 5) >= a.mask_words) return false;
    return (__ldg(a.mask + (int64_t)(q0 + i) * a.mask_words + (j >> 5)) >> (j & 31)) & 1u;
}

// One block: the shares and the cut groups.  `scan`: 33 * 8 bytes of shared memory.
template <int kCols, int kRows>
__device__ void tree_schedule(const TreeArgs &a, int64_t *scan) {
    TreeSched &s = *a.sched;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = (blockDim.x + 31) >> 5;
    const int64_t positions = tree_positions(a.max_pages, a.page_shift);
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    auto units = [&](int b, bool &bad) -> int64_t {
        const TreeSeq q = tree_seq(a.q_start, a.lens, b, a.R, positions);
        bad |= q.n < 0;
        if (q.n <= 0) return 0;
        return (int64_t)((q.n * a.H + kCols - 1) / kCols) * ((q.len + q.n + kRows - 1) / kRows);
    };
    bool bad = false;
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += units(b, bad);
    if (bad && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int64_t v = lane < n_warps ? scan[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        scan[lane] = v;
    }
    __syncthreads();
    int64_t at = inc - mine + (warp > 0 ? scan[warp - 1] : 0);
    for (int b = b0; b < b1; ++b) {
        s.unit0[b] = at;
        bool ignored = false;
        at += units(b, ignored);
    }
    const int64_t W = scan[n_warps - 1];
    if (tid == 0) {
        s.unit0[a.B] = W;
        s.jobs = 0;
        s.shares = (int)min((int64_t)a.ctas, W);
    }
    __syncthreads();
    const int C = (int)min((int64_t)a.ctas, W);
    // the last sequence whose first unit is <= u (it has work: the next one's first unit is larger)
    auto locate = [&](int64_t u, TreeShare &sh) {
        int lo = 0, hi = a.B;  // unit0[lo] <= u < unit0[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.unit0[mid] <= u) lo = mid;
            else hi = mid;
        }
        const TreeSeq q = tree_seq(a.q_start, a.lens, lo, a.R, positions);
        const int64_t tiles = (q.len + q.n + kRows - 1) / kRows, r = u - s.unit0[lo];
        sh.unit = u;
        sh.b = lo;
        sh.g = (int)(r / tiles);
        sh.t = (int)(r - sh.g * tiles);
        return tiles;
    };
    for (int c = tid; c <= C; c += blockDim.x) {
        TreeShare sh{};
        const int64_t u = C ? W / C * c + W % C * c / C : 0;  // floor(W * c / C) without the product
        if (c == C) {
            sh.unit = W;
            sh.b = a.B;
        } else {
            const int64_t tiles = locate(u, sh);
            // a share that begins inside a group whose first tile the share before it walks: that group is cut
            if (sh.t > 0) {
                const int64_t g0 = u - sh.t, g1 = g0 + tiles;
                const int64_t before = W / C * (c - 1) + W % C * (c - 1) / C;
                if (g0 >= before) {
                    int last = c;  // the share that holds the group's last unit
                    while (last + 1 < C && W / C * (last + 1) + W % C * (last + 1) / C < g1) ++last;
                    const int j = atomicAdd(&s.jobs, 1);
                    s.job[j] = TreeJob{sh.b, sh.g, c - 1, last - c + 2};
                }
            }
        }
        s.share[c] = sh;
    }
}

// The next segment of a CTA's share: tiles [t0, t1) of group g of sequence b.
struct TreeSegment {
    TreeSeq q;
    int b, g, t0, t1;
    bool first, last;  // it holds the group's first / last tile
};

struct TreeWalk {
    int64_t unit, end;
    int b, g, t;
    __device__ void begin(const TreeArgs &a, int cta) {
        const TreeSched &s = *a.sched;
        if (cta >= s.shares) {
            unit = end = 0;
            b = g = t = 0;
            return;
        }
        const TreeShare sh = s.share[cta];
        unit = sh.unit;
        b = sh.b;
        g = sh.g;
        t = sh.t;
        end = s.share[cta + 1].unit;
    }
    template <int kCols, int kRows>
    __device__ bool next(const TreeArgs &a, TreeSegment &seg) {
        if (unit >= end) return false;
        const int64_t positions = tree_positions(a.max_pages, a.page_shift);
        for (;;) {
            seg.q = tree_seq(a.q_start, a.lens, b, a.R, positions);
            if (seg.q.n > 0 && g < (seg.q.n * a.H + kCols - 1) / kCols) break;
            ++b;
            g = 0;
        }
        const int tiles = (int)((seg.q.len + seg.q.n + kRows - 1) / kRows);
        seg.b = b;
        seg.g = g;
        seg.t0 = t;
        seg.t1 = (int)min((int64_t)tiles, t + (end - unit));
        seg.first = t == 0;
        seg.last = seg.t1 == tiles;
        unit += seg.t1 - seg.t0;
        ++g;
        t = 0;
        return true;
    }
};

struct TreeWorkspace {
    size_t part, images, total;  // the shares come first
};
TreeWorkspace tree_workspace(int R, int H, int B, bool q_bf16);

cudaError_t launch_tree_merge(const TreeArgs &a, int cols, cudaStream_t st);
cudaError_t launch_tree_simt(const TreeArgs &a, cudaStream_t st);
cudaError_t launch_tree_tc(const TreeArgs &a, void *images, cudaStream_t st);
size_t tree_tc_images(int R, int H, int B);
size_t tree_tc_part_bytes(int ctas);
int tree_ctas();

}  // namespace kv8
