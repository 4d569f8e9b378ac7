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

// Whether some possible sequence with rows begins before the end of an earlier one; all threads of a block, each with its sequences
// [b0, b1).  That takes an impossible one between them, each start being the end before it, so that a batch without any need not
// be asked, and a start that falls: this is short rather than fast.  (With prefix maxima over the block: 2 us more for every
// call of eight sequences over 32768 rows, which do not run it.)
__device__ __forceinline__ bool tree_goes_back(const int32_t *q_start, const int32_t *lens, int b0, int b1, int R, int64_t positions) {
    bool back = false;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) back |= __ldg(q_start + b + 1) < __ldg(q_start + b);
    if (!__syncthreads_or(back)) return false;
    back = false;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const TreeSeq q = tree_seq(q_start, lens, b, R, positions);
#pragma unroll 1
        for (int e = 0; e < b; ++e) {
            const TreeSeq t = tree_seq(q_start, lens, e, R, positions);
            back |= q.n > 0 && t.n > 0 && t.q0 + t.n > q.q0;
        }
    }
    return __syncthreads_or(back);
}

// Positions that a table row of max_pages pages holds, as far as 32-bit lengths reach.
__host__ __device__ __forceinline__ int64_t tree_positions(int max_pages, int page_shift) {
    const int64_t p = (int64_t)max_pages << page_shift;
    return p < 0x7fffffff ? p : 0x7fffffff;
}

// Work shares.  A group is kCols consecutive (token, head) columns of one sequence (column = token * H +
// head); its work is the ceil(rows / kRows) row tiles of the sequence, and kSegment tiles' worth for its start
// and end.  All groups' work in order (sequence, group, tile) is one line, cut into `shares` equal pieces, one
// for each CTA, whatever the lengths.  A group that one CTA walks from its first tile to its last is finished
// there; one that a cut falls into leaves one partial set for each CTA that walks a part of it, and the merge
// joins them.
struct TreeShare {
    int64_t unit;  // tiles on the line before the share
    int b, g, t;   // where it begins
    int pad;
};
struct TreeJob {  // a group that was cut
    int64_t col0;      // its first column's place among the step's rows times heads
    int cols;
    int first, count;  // the CTAs first .. first + count - 1 hold its parts
    int pad;
};
constexpr int kMaxShares = 512;
struct TreeSched {
    int shares;  // CTAs that may have work
    int jobs;
    int pad[2];
    TreeShare share[kMaxShares + 1];  // [shares] ends the last one
    TreeJob job[kMaxShares];
    int64_t unit0[KV8_MAX_SEQS + 1];  // tiles and groups before sequence b, where they are more than shared memory takes
    int group0[KV8_MAX_SEQS + 1];
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

// The exponent that a partial set is stored with: a set of NaN sums has the largest, so that no other's makes it count as nothing.
__device__ __forceinline__ float tree_part_exponent(float m, float z) { return z == z ? m : INFINITY; }

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

// e4m3 NaN codes (0x7F, 0xFF) of four bytes -> 0
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
    const uint32_t hit = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    return w & ~hit;
}

// The rows of a 64-row tile that drafted token i attends (bit r: row r), where the tile's first row is the draft's
// row j0 (negative: a row of the context; all of those count).
__device__ __forceinline__ uint64_t tree_attended(const TreeArgs &a, int q0, int i, int64_t j0) {
    if (j0 <= -64) return ~(uint64_t)0;
    if (j0 >= KV8_MAX_TREE) return 0;
    const int skip = j0 < 0 ? (int)-j0 : 0, j = j0 < 0 ? 0 : (int)j0;  // rows of context, then draft from j on
    uint64_t bits;
    if (!a.mask) {
        const int n = i - j + 1;
        bits = n <= 0 ? 0 : n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1;
    } else {
        const uint32_t *m = a.mask + (int64_t)(q0 + i) * a.mask_words;
        uint32_t w[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) w[k] = (j >> 5) + k < a.mask_words ? __ldg(m + (j >> 5) + k) : 0u;
        bits = __funnelshift_r(w[0], w[1], j & 31) | (uint64_t)__funnelshift_r(w[1], w[2], j & 31) << 32;
    }
    return skip ? bits << skip | (((uint64_t)1 << skip) - 1) : bits;
}

// One block of 256 threads or more: the shares and the cut groups.
constexpr int kScanSeqs = 1024;
struct TreeScan {  // in shared memory
    int64_t unit0[kScanSeqs + 1];  // as in TreeSched
    int64_t unit[kMaxShares + 1];  // the shares' `unit`
    int64_t units[32];             // by warp
    int groups[32];
    int group0[kScanSeqs + 1];
    int jobs;
};
template <int kCols, int kRows, int kSegment, int kLeast>
__device__ void tree_schedule(const TreeArgs &a, TreeScan &sm) {
    TreeSched &s = *a.sched;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = (blockDim.x + 31) >> 5;
    const int64_t positions = tree_positions(a.max_pages, a.page_shift);
    int64_t *const unit0 = a.B <= kScanSeqs ? sm.unit0 : s.unit0;
    int *const group0 = a.B <= kScanSeqs ? sm.group0 : s.group0;
    const int per = (a.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    auto size_of = [&](int b, int &groups, int &tiles) -> TreeSeq {
        const TreeSeq q = tree_seq(a.q_start, a.lens, b, a.R, positions);
        groups = q.n > 0 ? (q.n * a.H + kCols - 1) / kCols : 0;
        tiles = q.n > 0 ? (int)((q.len + q.n + kRows - 1) / kRows) : 0;
        return q;
    };
    bool bad = false;
    int groups = 0, tiles = 0, gs = 0;
    int64_t us = 0;
    for (int b = b0; b < b1; ++b) {
        bad |= size_of(b, groups, tiles).n < 0;
        us += (int64_t)groups * tiles;
        gs += groups;
    }
    if (bad && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
    int64_t ui = us;
    int gi = gs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, ui, o);
        const int g = __shfl_up_sync(0xffffffffu, gi, o);
        if (lane >= o) {
            ui += u;
            gi += g;
        }
    }
    if (lane == 31) {
        sm.units[warp] = ui;
        sm.groups[warp] = gi;
    }
    if (__syncthreads_or(bad) && tree_goes_back(a.q_start, a.lens, b0, b1, a.R, positions)) {
        if (tid == 0) s.shares = s.jobs = 0;
        return;
    }
    int64_t U = 0, u_at = ui - us;
    int G = 0, g_at = gi - gs;
    for (int w = 0; w < n_warps; ++w) {
        if (w == warp) {
            u_at += U;
            g_at += G;
        }
        U += sm.units[w];
        G += sm.groups[w];
    }
    for (int b = b0; b < b1; ++b) {
        unit0[b] = u_at;
        group0[b] = g_at;
        if (per > 1) size_of(b, groups, tiles);
        u_at += (int64_t)groups * tiles;
        g_at += groups;
    }
    const int64_t W = U + (int64_t)kSegment * G;
    const int C = (int)min((int64_t)a.ctas, (U + kLeast - 1) / kLeast);
    if (tid == 0) {
        sm.jobs = 0;
        s.shares = C;
    }
    __syncthreads();
    // (most numbers have 32 bits, whose divisions are a fraction of the longer ones' time)
    constexpr int kPer = kMaxShares / 256 + 1;
    TreeShare sh[kPer];
    TreeSeq q[kPer];
    int its[kPer];  // tiles of the share's first group
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * (int)blockDim.x;
        if (c > C) break;
        sh[i] = TreeShare{U, a.B, 0, 0, 0};
        if (c < C) {
            const bool narrow = W <= 0x7fffffff;
            const int64_t w = narrow ? (int64_t)((uint32_t)W / C * c + (uint32_t)W % C * c / C) : W / C * c + W % C * c / C;  // floor(W c / C)
            int lo = 0, hi = a.B;  // work before lo <= w < work before hi: the last such sequence, so it has work
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (unit0[mid] + (int64_t)kSegment * group0[mid] <= w) lo = mid;
                else hi = mid;
            }
            q[i] = size_of(lo, groups, its[i]);
            const int64_t r = w - unit0[lo] - (int64_t)kSegment * group0[lo];
            const int each = its[i] + kSegment;
            const int g = narrow ? (int)((uint32_t)r / (uint32_t)each) : (int)(r / each);
            // (a cut in a group's start and end cost is one before its first tile)
            const int t = max((int)(r - (int64_t)g * each) - kSegment, 0);
            sh[i] = TreeShare{unit0[lo] + (int64_t)g * its[i] + t, lo, g, t, 0};
        }
        s.share[c] = sh[i];
        sm.unit[c] = sh[i].unit;
    }
    __syncthreads();
    // a share that begins inside a group whose first tile the share before it walks: that group is cut
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int c = tid + i * (int)blockDim.x;
        if (c >= C) break;
        const int64_t begin = sh[i].unit - sh[i].t, end = begin + its[i];
        if (c == 0 || sh[i].t == 0 || begin < sm.unit[c - 1]) continue;
        int lo = c, hi = C;  // the share that holds the group's last tile: unit[lo] < end <= unit[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.unit[mid] < end) lo = mid;
            else hi = mid;
        }
        const int64_t at = (int64_t)sh[i].g * kCols;
        s.job[atomicAdd(&sm.jobs, 1)] = TreeJob{(int64_t)q[i].q0 * a.H + at, (int)min((int64_t)kCols, (int64_t)q[i].n * a.H - at),
                                                c - 1, lo - c + 2, 0};
    }
    __syncthreads();
    if (tid == 0) s.jobs = sm.jobs;
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
cudaError_t launch_tree_f32(const TreeArgs &a, cudaStream_t st);
cudaError_t launch_tree_tc(const TreeArgs &a, void *images, cudaStream_t st);
size_t tree_tc_images(int R, int H, int B);
size_t tree_tc_part_bytes(int ctas);
int tree_ctas();

}  // namespace kv8
