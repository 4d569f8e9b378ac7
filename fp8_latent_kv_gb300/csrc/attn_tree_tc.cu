// attn_tree_tc.cu -- attention of drafted tokens over a paged latent cache on the tensor cores (tcgen05, sm_103a),
// for bf16 queries.
//
// All (token, head) columns of a sequence read the same rows, so a group of 64 columns against a tile of 128 rows
// is two contractions:
//   score    S^T[t][n]  = sum_k K8[t][k] Qs[n][k]      M = 128 rows, N = 128, K = 576 (e4m3 x e4m3)
//            Qs = [Q_hi; Q_lo]: a bf16 query element, scaled by its column's power of two, is the sum of two e4m3
//            values, so the two halves of S^T add up to the bf16 dot product.
//   context  O^T[d][n] += sum_t V8[t][d] W^T[t][n]     M = 128 dims (x4), K = 128 rows; V8 = the same bytes read
//            MN-major, W the softmax weights as two pieces, hi in e4m3 and lo, what hi leaves, in e5m2: 2^-7 of a
//            weight at most, and terms down to 2^-22 of the column's largest still count (two e4m3 pieces would
//            round everything below 2^-16 to nothing, which a long context's many small terms add up to).
// Weights: with e_t = score_t log2(e) + log2(scale_t) and a running reference m >= max e - 2 for each column,
// w_t = 2^(e_t - m + 6) <= 256 holds the row scale already, O = sum w_t v_t and z = sum w_t / scale_t; the factor
// 2^6 cancels.  A weight's share of e4m3's range then follows its own column's largest term whatever rows, drafted
// or not, other columns attend.  A row whose scale is below 2^-100 (zeros, subnormal maxima) has score 0 and adds
// nothing to O: such rows are only counted, and the count enters z as n0 2^-m at the end.
//
// Work: equal shares of (group, tile) units (tree.cuh), one CTA per SM.
// Warps: 0 = loads, 1 = MMA issue and TMEM, 2..17 = softmax and output in four sets of four warps (a warp per TMEM
// lane quadrant), 16 columns each; a thread holds one row of the tile.
// Shared memory: query image 72 KB, eight 16 KB latent blocks (two tiles; a block is refilled as soon as the context
// product has read it, and the score starts on a block when it lands), one 8 KB RoPE block (free again after the
// score), weights hi and lo 8 KB each.  TMEM: two score buffers of 128 columns, context accumulators 4 x 64.
// Every wait is bounded in time; one that gives up sets KV8_ERR_TIMEOUT and the CTA winds down.
#include "sm100.cuh"
#include "tree.cuh"

#include <math.h>
#include <stddef.h>

namespace kv8 {
namespace {

using namespace sm100;

constexpr int kCols = 64;
constexpr int kRows = 128;
constexpr int kHG = 16;                    // columns per softmax set
constexpr int kNG = kCols / kHG;
constexpr int kSoftmaxThreads = 128 * kNG;
constexpr int kThreads = 64 + kSoftmaxThreads;
constexpr uint32_t kBlk = 16384;           // 128 rows x 128 latent bytes (SW128)
constexpr uint32_t kRope = 8192;           // 128 rows x 64 RoPE bytes (SW64)
constexpr uint32_t kImg = 4 * kBlk + kRope;
constexpr uint32_t OFF_Q = 0, OFF_RING = kImg, OFF_ROPE = OFF_RING + 8 * kBlk, OFF_WHI = OFF_ROPE + kRope,
                   OFF_WLO = OFF_WHI + 8192, OFF_MISC = OFF_WLO + 8192;
constexpr float kTau = 2.0f;               // the reference moves when a term exceeds it by more than 2^kTau
constexpr float kUp = 6.0f;                // weights are held times 2^kUp: at most 2^8 < 448
constexpr float kTiny = 7.888609e-31f;     // 2^-100
constexpr uint32_t TM_S = 0, TM_O = 256;  // two score buffers of 128 columns, four accumulators of 64

struct Misc {
    alignas(16) float m_run[2][kCols];     // reference per column (log2 units), -inf before any attended row
    alignas(16) float red[4][kCols];       // per-quadrant maxima / row sums
    alignas(16) float c_head[kCols];       // sm_scale * log2(e) * 2^-e of the column's query
    alignas(16) float alpha[kNG][kHG];     // rescale factors, and the reference shifts; at the end 1 / z
    alignas(16) float delta[kNG][kHG];
    uint64_t blk_full[8], blk_free[8], rope_full, rope_free, q_full, q_free, s_full[2], s_free[2], w_full, lo_free, done[2],
        final_bar;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr uint32_t kSmemBytes = OFF_MISC + sizeof(Misc);
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(offsetof(Misc, blk_full) % 8 == 0 && OFF_MISC % 1024 == 0, "alignment");

struct TcArgs {
    TreeArgs t;
    const uint8_t *img;    // query images, one kImg for each group
    const float *c_head;   // [images][64]
};

// A sequence's groups' images begin at slot q0 * H / 64 + b: never past the next sequence's first.
__host__ __device__ __forceinline__ int64_t tree_slot(int64_t q0, int H, int b) { return q0 * H / kCols + b; }

__device__ __forceinline__ uint32_t enc_pair(float a, float b) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(b), "f"(a));
    return v;
}
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = enc_pair(a, b);
    float x, y;
    e4m3x2_to_f32((uint16_t)hi, x, y);
    lo = enc_pair(a - x, b - y);
}
// Two softmax weights (at most 2^8) -> e4m3 pieces and e5m2 pieces of what those leave.  By way of f16, whose 11
// bits are finer than the 7 that the pieces keep; the residual is exact there.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t &hi, uint32_t &lo) {
    uint32_t w16, h16, r16;
    uint16_t h8, l8;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w16) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h8) : "r"(w16));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(h8));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r16) : "r"(w16), "r"(h16));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(l8) : "r"(r16));
    hi = h8;
    lo = l8;
}
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e4m3 NaN codes (0x7F, 0xFF) of four bytes -> 0
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
    const uint32_t hit = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    return w & ~hit;
}

// ------------------------------------------------------------------------------------------------------------
// Query images, column factors, and (block 0) the work shares.  A block splits eight consecutive (row, head)
// columns, 36 threads each.
// ------------------------------------------------------------------------------------------------------------
constexpr int kPrepCols = 8, kPrepThreads = kPrepCols * 36;

__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(TreeArgs a, uint8_t *img, float *c_head) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int64_t scan[33];
    __shared__ int qmax_bits[kPrepCols];
    __shared__ int64_t pad_slot[kPrepCols];
    __shared__ int pad_from[kPrepCols];
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        tree_schedule<kCols, kRows>(a, scan);
        return;
    }
    const int64_t col0 = (int64_t)(blockIdx.x - 1) * kPrepCols;
    const int cl = tid / 36, ch = tid - cl * 36;
    const int64_t gc = col0 + cl;
    const int row = (int)(gc / a.H), head = (int)(gc - (int64_t)row * a.H);
    if (tid < kPrepCols) {
        qmax_bits[tid] = 0;
        pad_from[tid] = kCols;
    }
    // the sequence of the block's first column: how many sequences end at or before its row
    int b = 0;
    {
        const int row0 = (int)(col0 / a.H);
        for (int k0 = 0; k0 < a.B; k0 += kPrepThreads) {
            const int k = k0 + tid;
            b += __syncthreads_count(k < a.B && __ldg(a.q_start + k + 1) <= row0);
        }
    }
    while (b < a.B && __ldg(a.q_start + b + 1) <= row) ++b;
    bool mine = row < a.R && b < a.B;
    TreeSeq q{};
    if (mine) {
        q = tree_seq(a.q_start, a.lens, b, a.R, tree_positions(a.max_pages, a.page_shift));
        mine = q.n > 0 && row >= q.q0 && row < q.q0 + q.n;
    }
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (mine) {
        const __nv_bfloat16 *src = ch < 32 ? static_cast<const __nv_bfloat16 *>(a.q_lat) + gc * kKL + ch * 16
                                           : static_cast<const __nv_bfloat16 *>(a.q_rope) + gc * kKR + (ch - 32) * 16;
        const uint4 u0 = __ldg(reinterpret_cast<const uint4 *>(src)), u1 = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
        w[0] = u0.x; w[1] = u0.y; w[2] = u0.z; w[3] = u0.w;
        w[4] = u1.x; w[5] = u1.y; w[6] = u1.z; w[7] = u1.w;
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        atomicMax(&qmax_bits[cl], __float_as_int(mx));  // non-negative floats order like ints
    }
    __syncthreads();
    if (mine) {
        const float mx = __int_as_float(qmax_bits[cl]);
        int E = 0;
        if (mx > 0.f) frexpf(mx, &E);
        const int sh = mx > 0.f ? 8 - E : 0;  // max |q| 2^sh in [128, 256); values are scaled: 2^sh may overflow
        uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
            uint32_t ph, pl;
            split_pair(ldexpf(f.x, sh), ldexpf(f.y, sh), ph, pl);
            hi[e >> 1] |= ph << ((e & 1) * 16);
            lo[e >> 1] |= pl << ((e & 1) * 16);
        }
        const int col = (row - q.q0) * a.H + head, n = col % kCols;
        const int64_t slot = tree_slot(q.q0, a.H, b) + col / kCols;
        uint8_t *dst = img + slot * kImg;
        uint32_t off_hi, off_lo;
        if (ch < 32) {
            off_hi = (ch >> 3) * kBlk + sw128_offset(n, (ch & 7) * 16);
            off_lo = (ch >> 3) * kBlk + sw128_offset(n + 64, (ch & 7) * 16);
        } else {
            off_hi = 4 * kBlk + sw64_offset(n, (ch - 32) * 16);
            off_lo = 4 * kBlk + sw64_offset(n + 64, (ch - 32) * 16);
        }
        *reinterpret_cast<uint4 *>(dst + off_hi) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + off_lo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (ch == 0) {
            c_head[slot * kCols + n] = mx > 0.f ? ldexpf(a.sm_scale_log2, E - 8) : a.sm_scale_log2;
            if (col == q.n * a.H - 1) {  // the sequence's last column: the rest of its group is zeros
                pad_slot[cl] = slot;
                pad_from[cl] = n + 1;
            }
        }
    }
    __syncthreads();
    for (int c = 0; c < kPrepCols; ++c) {
        const int from = pad_from[c], cols = kCols - from;
        if (cols <= 0) continue;
        uint8_t *dst = img + pad_slot[c] * kImg;
        for (int i = tid; i < cols * 72; i += kPrepThreads) {
            const int n = from + i / 72, p = i % 72, lo = p / 36 * 64, k = p % 36;
            const uint32_t off = k < 32 ? (k >> 3) * kBlk + sw128_offset(n + lo, (k & 7) * 16)
                                        : 4 * kBlk + sw64_offset(n + lo, (k - 32) * 16);
            *reinterpret_cast<uint4 *>(dst + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int n = from + tid; n < kCols; n += kPrepThreads) c_head[pad_slot[c] * kCols + n] = 0.f;
    }
}

// ------------------------------------------------------------------------------------------------------------
// 18 warps: a sub-partition holding 5 warps caps a thread at 96 registers.
__global__ void __launch_bounds__(kThreads, 1)
    attn_tree_tc_kernel(const __grid_constant__ CUtensorMap map_lc, const __grid_constant__ CUtensorMap map_rc, TcArgs x) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const TreeArgs &a = x.t;
    Misc &ms = *reinterpret_cast<Misc *>(smem + OFF_MISC);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((smem_u32(smem) & 1023u) != 0) {  // swizzled operands need 1024-byte alignment
        if (tid == 0 && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_TIMEOUT);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < 8; ++s) {
            mbar_init(&ms.blk_full[s], 1);
            mbar_init(&ms.blk_free[s], 1);
        }
        mbar_init(&ms.rope_full, 1);
        mbar_init(&ms.rope_free, 1);
        mbar_init(&ms.q_full, 1);
        mbar_init(&ms.q_free, 1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(&ms.s_full[k], 1);
            mbar_init(&ms.s_free[k], kSoftmaxThreads);
        }
        mbar_init(&ms.w_full, kSoftmaxThreads);
        mbar_init(&ms.lo_free, 1);
        mbar_init(&ms.done[0], 1);
        mbar_init(&ms.done[1], 1);
        mbar_init(&ms.final_bar, 1);
        ms.abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&map_lc);
        prefetch_tensormap(&map_rc);
    }
    if (warp == 1) {
        tmem_alloc(&ms.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = ms.tmem_base;
    const uint32_t sbase = smem_u32(smem);
    grid_dependency_wait();  // the shares and images, and whatever wrote the cache before them

    TreeWalk walk;
    walk.begin(a, blockIdx.x);
    TreeSegment seg;

    if (warp == 0) {
        // ================================ loads ================================
        // A block's barrier is armed after its release, which implies that its previous phase is complete.
        const int sub_rows = min(kRows, 1 << a.page_shift), subs = kRows / sub_rows;
        int it = 0, sg = 0;
        uint32_t armed = 0;  // per slot: loads in flight since its last arming (bits), 8 = RoPE, 9 = image
        bool ok = true;
        while (ok && walk.next<kCols, kRows>(a, seg)) {
            const int64_t end = seg.q.len + seg.q.n;
            for (int t = seg.t0; ok && t < seg.t1; ++t, ++it) {
                // lane l < subs holds the cache row where the tile's l-th piece begins, or -1
                const int64_t pos = (int64_t)t * kRows + (int64_t)lane * sub_rows;
                int64_t row = -1;
                if (lane < subs && pos < end) row = tree_row(a, seg.b, pos);
                const int pieces = __popc(__ballot_sync(0xffffffffu, row >= 0));
                const uint32_t ph = ((it >> 1) - 1) & 1;
#pragma unroll 1
                for (int kb = 0; kb < 4 && ok; ++kb) {
                    const int s = (it & 1) * 4 + kb;
                    if (it >= 2) ok = mbar_wait(&ms.blk_free[s], ph, &ms.abort_flag, a.err_word);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&ms.blk_full[s], (uint32_t)pieces * sub_rows * 128u);
                    armed |= 1u << s;
                    __syncwarp();
                    if (row >= 0)
                        tma_load_2d(smem + OFF_RING + s * kBlk + lane * sub_rows * 128, &map_lc, kb * 128, (int)row,
                                    &ms.blk_full[s]);
                }
                if (ok && it >= 1) ok = mbar_wait(&ms.rope_free, (it - 1) & 1, &ms.abort_flag, a.err_word);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&ms.rope_full, (uint32_t)pieces * sub_rows * 64u);
                armed |= 1u << 8;
                __syncwarp();
                if (row >= 0) tma_load_2d(smem + OFF_ROPE + lane * sub_rows * 64, &map_rc, 512, (int)row, &ms.rope_full);
                if (t == seg.t0) {
                    // the segment's query image, once the last score of the segment before it has read the old one
                    if (sg >= 1) ok = mbar_wait(&ms.q_free, (sg - 1) & 1, &ms.abort_flag, a.err_word);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ms.q_full, kImg);
                        const uint8_t *src = x.img + (tree_slot(seg.q.q0, a.H, seg.b) + seg.g) * kImg;
                        for (int kb = 0; kb < 4; ++kb) bulk_load(smem + OFF_Q + kb * kBlk, src + kb * kBlk, kBlk, &ms.q_full);
                        bulk_load(smem + OFF_Q + 4 * kBlk, src + 4 * kBlk, kRope, &ms.q_full);
                    }
                    armed |= 1u << 9;
                    ++sg;
                }
            }
        }
        // every load in flight lands before the CTA ends: the last phase of each armed barrier
        if (lane == 0) {
            const int last = ok ? it - 1 : it;  // after a timeout tile `it` is partly armed: waiting for it too
            for (int kb = 0; kb < 8; ++kb)
                if (armed >> kb & 1) {
                    // the newest tile of this parity whose block was armed
                    int i = last - ((last ^ (kb >> 2)) & 1);
                    if (i >= 0) mbar_wait(&ms.blk_full[kb], (i >> 1) & 1, nullptr, a.err_word, ok ? 200000000ull : 20000000ull);
                }
            if (armed >> 8 & 1) mbar_wait(&ms.rope_full, last & 1, nullptr, a.err_word, ok ? 200000000ull : 20000000ull);
            if (armed >> 9 & 1) mbar_wait(&ms.q_full, (sg - 1) & 1, nullptr, a.err_word, 200000000ull);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================ MMA issue ================================
        if (lane == 0) {
            const uint32_t id_s = idesc_e4m3_f32(128, 128, false, false);
            const uint32_t id_hi = idesc_e4m3_f32(128, 64, true, true), id_lo = id_hi | (1u << 10);  // B in e5m2
            const uint32_t qb = sbase + OFF_Q, rope = sbase + OFF_ROPE, phi = sbase + OFF_WHI, plo = sbase + OFF_WLO;
            const int64_t n_tiles = walk.end - walk.unit;
            auto issue_pv = [&](int j, bool first) {
                const int s = (j & 1) * 4;
                const uint32_t st = sbase + OFF_RING + s * kBlk;
                const uint32_t keep = first ? 0u : 1u;
                // the lo pieces first: the next tile's may then be written while the hi pieces run
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8f6f4(tmem + TM_O + 64u * ch, smem_desc(st + ch * kBlk + kk * 4096, 0, 1024, kSw128),
                                   smem_desc(plo + kk * 2048, 0, 512, kSw64), id_lo, kk ? 1u : keep);
                mma_commit(&ms.lo_free);
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8f6f4(tmem + TM_O + 64u * ch, smem_desc(st + ch * kBlk + kk * 4096, 0, 1024, kSw128),
                                   smem_desc(phi + kk * 2048, 0, 512, kSw64), id_hi, 1u);
                    mma_commit(&ms.blk_free[s + ch]);
                }
                mma_commit(&ms.done[j & 1]);
            };
            // whichever is ready: the next context product (its weights written), else the next part of the next
            // score (part kb needs latent block kb, part 4 the RoPE block)
            int ns = 0, part = 0, np = 0, sg = 0;
            int seg_end = 0;          // first tile after the score side's segment
            uint32_t firsts = 0;      // bit i % 32: tile i begins a segment
            uint64_t t_last = globaltimer_ns();
            uint32_t spins = 0;
            while (np < n_tiles) {
                bool did = false;
                if (np < ns && mbar_test_wait(&ms.w_full, np & 1)) {
                    tc_fence_after_sync();
                    issue_pv(np, firsts >> (np & 31) & 1);
                    ++np;
                    did = true;
                } else if (ns < n_tiles) {
                    bool ready = true;
                    if (part == 0) {
                        if (ns == seg_end) {  // a new segment
                            walk.next<kCols, kRows>(a, seg);
                            seg_end = ns + (seg.t1 - seg.t0);
                            ++sg;
                            firsts |= 1u << (ns & 31);
                        } else if (ns != seg_end - (seg.t1 - seg.t0)) {
                            firsts &= ~(1u << (ns & 31));
                        }
                        ready = mbar_test_wait(&ms.q_full, (sg - 1) & 1) && (ns < 2 || mbar_test_wait(&ms.s_free[ns & 1], ((ns >> 1) - 1) & 1));
                    }
                    const int s = (ns & 1) * 4;
                    if (ready) ready = part < 4 ? mbar_test_wait(&ms.blk_full[s + part], (ns >> 1) & 1)
                                                : mbar_test_wait(&ms.rope_full, ns & 1);
                    if (ready) {
                        tc_fence_after_sync();
                        if (part < 4) {
                            const uint32_t kblk = sbase + OFF_RING + (s + part) * kBlk, qblk = qb + part * kBlk;
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_f8f6f4(tmem + TM_S + 128u * (ns & 1), smem_desc(kblk + kk * 32, 0, 1024, kSw128),
                                           smem_desc(qblk + kk * 32, 0, 1024, kSw128), id_s, (part | kk) != 0);
                            ++part;
                        } else {
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                mma_f8f6f4(tmem + TM_S + 128u * (ns & 1), smem_desc(rope + kk * 32, 0, 512, kSw64),
                                           smem_desc(qb + 4 * kBlk + kk * 32, 0, 512, kSw64), id_s, 1u);
                            mma_commit(&ms.s_full[ns & 1]);
                            mma_commit(&ms.rope_free);
                            if (ns + 1 == seg_end) mma_commit(&ms.q_free);
                            ++ns;
                            part = 0;
                        }
                        did = true;
                    }
                }
                if (did) {
                    spins = 0;
                } else if ((++spins & 255u) == 0) {
                    const uint64_t now = globaltimer_ns();
                    if (*(volatile int *)&ms.abort_flag) break;
                    if (spins > 256u && now - t_last > 2000000000ull) {  // no progress for 2 s
                        ms.abort_flag = 1;
                        if (a.err_word) atomicOr(a.err_word, (int)KV8_ERR_TIMEOUT);
                        break;
                    }
                } else if (spins == 1) {
                    t_last = globaltimer_ns();
                }
            }
            mma_commit(&ms.final_bar);  // all issued MMAs complete before the CTA tears down
            mbar_wait(&ms.final_bar, 0, nullptr, a.err_word, 200000000ull);
        }
        __syncwarp();
    } else {
        // ============================ softmax and output ============================
        // A wait that gives up clears `ok`; the thread then skips its remaining waits but still reaches every named
        // barrier, so that no other warp waits for it.
        constexpr int kV4 = kHG / 4, kP = kHG / 2;
        const int q = warp & 3, grp = (warp - 2) >> 2, h0 = kHG * grp, r = q * 32 + lane;
        const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
        const int bar_id = 2 + grp;
        const int pshift = a.page_shift;
        const int64_t pmask = ((int64_t)1 << pshift) - 1;
        bool ok = true, bad_page = false;  // ok is the same in a warp's lanes: TMEM loads need all of them
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &ms.abort_flag, a.err_word));
        };
        grid_launch_dependents();
        int it = 0;
        while (walk.next<kCols, kRows>(a, seg)) {
            const int64_t end = seg.q.len + seg.q.n;
            const int32_t *table = a.table + (int64_t)seg.b * a.max_pages;
            const int64_t slot = tree_slot(seg.q.q0, a.H, seg.b) + seg.g;
            named_sync(bar_id, 128);  // the set's arrays: every warp is done with the segment before
            if (q == 0 && lane < kHG) {
                ms.c_head[h0 + lane] = x.c_head[slot * kCols + h0 + lane];
                ms.m_run[0][h0 + lane] = -INFINITY;
            }
            named_sync(bar_id, 128);
            uint64_t z2[kP];
#pragma unroll
            for (int j = 0; j < kP; ++j) z2[j] = f2_pack(0.f, 0.f);
            // the row of position pos: page entries are fetched two tiles ahead, scales one
            auto page_of = [&](int64_t pos) -> int64_t { return pos < end ? (int64_t)__ldg(table + (pos >> pshift)) : -1; };
            auto scale_of = [&](int64_t pos, int64_t page, bool &in) -> float {
                const int64_t row = (page << pshift) + (pos & pmask);
                in = page >= 0 && row < a.cache_rows;
                bad_page |= pos < end && !in;
                return in ? __ldg(a.kv_scale + row) : 1.f;
            };
            bool in_next;
            const int64_t p_first = (int64_t)seg.t0 * kRows + r;
            int64_t page2 = page_of(p_first);
            float sc_next = scale_of(p_first, page2, in_next);
            page2 = seg.t0 + 1 < seg.t1 ? page_of(p_first + kRows) : -1;
            int n0 = 0;             // zero rows of the context that this thread has met
            uint32_t n0_draft = 0;  // and of the draft, column j's count in bits j and 16 + j
            bool seen = false;  // every column of the set has a finite reference
            int cur = 0;        // which copy of ms.m_run is current
            for (int t = seg.t0; t < seg.t1; ++t, ++it) {
                const int64_t pos = (int64_t)t * kRows + r;
                const float sc = sc_next;
                const bool in = in_next;
                if (t + 1 < seg.t1) {
                    sc_next = scale_of(pos + kRows, page2, in_next);
                    if (t + 2 < seg.t1) page2 = page_of(pos + 2 * kRows);
                }
                // which of the 16 columns attend the row: all of them in the context, by their bits in the draft
                uint32_t sees = in ? 0xFFFFu : 0u;
                const int64_t draft = pos - seg.q.len;
                const bool drafted = in && draft >= 0;
                if (drafted) {
                    sees = 0;
                    const int c0 = seg.g * kCols + h0, top = seg.q.n * a.H;
                    int node = c0 / a.H, left = a.H - (c0 - node * a.H);
#pragma unroll 1
                    for (int j = 0; j < kHG; ++j) {
                        if (c0 + j < top && tree_sees(a, seg.q.q0, node, (int)draft)) sees |= 1u << j;
                        if (--left == 0) {
                            ++node;
                            left = a.H;
                        }
                    }
                }
                if (sc < kTiny) {  // a zero row: counted, and left out of everything else
                    if (!drafted) n0 += sees ? 1 : 0;
                    else {  // two bits for each column: a thread has at most three of the draft's rows
                        const uint32_t both = n0_draft & 0xFFFFu & sees;
                        n0_draft = (n0_draft ^ sees) ^ (both << 16);
                    }
                    sees = 0;
                }
                const float lg = lg2_approx(sc) + kUp;
                // 0 for a zero row (its w is 0) and for a scale that is not finite (its w is NaN where it is attended)
                const float inv = sc >= kTiny && sc <= 3.402823466e38f ? __fdividef(1.f, sc) : 0.f;

                wait(&ms.s_full[it & 1], (it >> 1) & 1);
                tc_fence_after_sync();
                uint64_t s2[kP];  // hi + lo halves of the score, column pairs packed
                {
                    uint32_t shi[16], slo[16];
                    const uint32_t ta = tmem + lane_addr + TM_S + 128u * (it & 1) + (uint32_t)h0;
                    tmem_ld_32x32b_x16(ta, shi);
                    tmem_ld_32x32b_x16(ta + 64u, slo);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kP; ++j)
                        s2[j] = f2_add(f2_pack(__uint_as_float(shi[2 * j]), __uint_as_float(shi[2 * j + 1])),
                                       f2_pack(__uint_as_float(slo[2 * j]), __uint_as_float(slo[2 * j + 1])));
                }
                tc_fence_before_sync();
                mbar_arrive(&ms.s_free[it & 1]);
                // d = e + 6 - m (m counts as 0 while it is -inf)
                uint64_t d2[kP];
                float dmax = -INFINITY;
                {
                    const uint64_t st2 = f2_pack(sc, sc), lg2 = f2_pack(lg, lg);
#pragma unroll
                    for (int j4 = 0; j4 < kV4; ++j4) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(&ms.c_head[h0 + 4 * j4]);
                        float4 r4 = *reinterpret_cast<const float4 *>(&ms.m_run[cur][h0 + 4 * j4]);
                        if (!seen) {
                            r4.x = r4.x == -INFINITY ? 0.f : r4.x;
                            r4.y = r4.y == -INFINITY ? 0.f : r4.y;
                            r4.z = r4.z == -INFINITY ? 0.f : r4.z;
                            r4.w = r4.w == -INFINITY ? 0.f : r4.w;
                        }
                        d2[2 * j4] = f2_fma(s2[2 * j4], f2_mul(f2_pack(c4.x, c4.y), st2), f2_add(lg2, f2_pack(-r4.x, -r4.y)));
                        d2[2 * j4 + 1] =
                            f2_fma(s2[2 * j4 + 1], f2_mul(f2_pack(c4.z, c4.w), st2), f2_add(lg2, f2_pack(-r4.z, -r4.w)));
                    }
                    if (sees != 0xFFFFu) {
#pragma unroll
                        for (int j = 0; j < kP; ++j) {
                            float u, v;
                            f2_unpack(d2[j], u, v);
                            d2[j] = f2_pack(sees >> (2 * j) & 1 ? u : -INFINITY, sees >> (2 * j + 1) & 1 ? v : -INFINITY);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kP; ++j) {
                        float u, v;
                        f2_unpack(d2[j], u, v);
                        dmax = fmaxf(dmax, fmaxf(u, v));
                    }
                }
                // the set moves its references together when a term exceeds one by more than kTau, or while a column
                // has none
                const bool slow = bar_red_or(bar_id, 128, dmax > kTau + kUp || !seen);
                bool any_alpha = false;
                if (slow) {
                    float hm[kHG];
#pragma unroll
                    for (int j = 0; j < kP; ++j) {
                        float u, v;
                        f2_unpack(d2[j], u, v);
                        hm[2 * j] = warp_redux_max(u);
                        hm[2 * j + 1] = warp_redux_max(v);
                    }
                    if (lane == 0) {
#pragma unroll
                        for (int j4 = 0; j4 < kV4; ++j4)
                            *reinterpret_cast<float4 *>(&ms.red[q][h0 + 4 * j4]) =
                                make_float4(hm[4 * j4], hm[4 * j4 + 1], hm[4 * j4 + 2], hm[4 * j4 + 3]);
                    }
                    const int hl = lane & (kHG - 1), hj = h0 + hl;
                    named_sync(bar_id, 128);
                    const float mo = ms.m_run[cur][hj], ref_o = mo == -INFINITY ? 0.f : mo;
                    const float tmax = fmaxf(fmaxf(ms.red[0][hj], ms.red[1][hj]), fmaxf(ms.red[2][hj], ms.red[3][hj])) + (ref_o - kUp);
                    const float mn = mo == -INFINITY ? tmax : (tmax > mo + kTau ? tmax : mo);
                    const float al = (mo == -INFINITY || mn == mo) ? 1.f : ex2_approx(mo - mn);
                    const float ref_n = mn == -INFINITY ? 0.f : mn;
                    if (lane < kHG) {  // the four quadrant warps write the same values
                        ms.m_run[cur ^ 1][hj] = mn;
                        ms.alpha[grp][hl] = al;
                        ms.delta[grp][hl] = ref_o - ref_n;
                    }
                    seen = __all_sync(0xffffffffu, mn != -INFINITY);
                    any_alpha = __any_sync(0xffffffffu, al != 1.f);
                    __syncwarp();
#pragma unroll
                    for (int j4 = 0; j4 < kV4; ++j4) {
                        const float4 a4 = *reinterpret_cast<const float4 *>(&ms.alpha[grp][4 * j4]);
                        const float4 e4 = *reinterpret_cast<const float4 *>(&ms.delta[grp][4 * j4]);
                        d2[2 * j4] = f2_add(d2[2 * j4], f2_pack(e4.x, e4.y));
                        d2[2 * j4 + 1] = f2_add(d2[2 * j4 + 1], f2_pack(e4.z, e4.w));
                        z2[2 * j4] = f2_mul(z2[2 * j4], f2_pack(a4.x, a4.y));
                        z2[2 * j4 + 1] = f2_mul(z2[2 * j4 + 1], f2_pack(a4.z, a4.w));
                    }
                    cur ^= 1;
                }
                const uint64_t inv2 = f2_pack(inv, inv);
                uint32_t whi[kV4], wlo[kV4];
#pragma unroll
                for (int j4 = 0; j4 < kV4; ++j4) {
                    float d0, d1, e0, e1;
                    f2_unpack(d2[2 * j4], d0, d1);
                    f2_unpack(d2[2 * j4 + 1], e0, e1);
                    const float w0 = ex2_approx(d0), w1 = ex2_approx(d1), w3 = ex2_approx(e0), w4 = ex2_approx(e1);
                    z2[2 * j4] = f2_fma(f2_pack(w0, w1), inv2, z2[2 * j4]);
                    z2[2 * j4 + 1] = f2_fma(f2_pack(w3, w4), inv2, z2[2 * j4 + 1]);
                    uint32_t h01, l01, h23, l23;
                    split_weights(w0, w1, h01, l01);
                    split_weights(w3, w4, h23, l23);
                    whi[j4] = h01 | (h23 << 16);
                    wlo[j4] = l01 | (l23 << 16);
                }
                // rows that were not loaded, and NaN codes of drafted rows (attended columns have NaN weights
                // already): a weight of 0 must not meet them.  Thread (row, set) owns the row's bytes in block `grp`.
                if (!in || drafted) {
                    // (complete since before the score: this makes the copy's bytes visible here too)
                    (void)mbar_wait(&ms.blk_full[(it & 1) * 4 + grp], (it >> 1) & 1, &ms.abort_flag, a.err_word);
                    uint4 *p = reinterpret_cast<uint4 *>(smem + OFF_RING + ((it & 1) * 4 + grp) * kBlk + r * 128);
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (in) {
                            v = p[k];
                            v.x = without_nan(v.x);
                            v.y = without_nan(v.y);
                            v.z = without_nan(v.z);
                            v.w = without_nan(v.w);
                        }
                        p[k] = v;
                    }
                }
                if (it >= 1) {
                    // the context product before has read its lo weights
                    wait(&ms.lo_free, (it - 1) & 1);
                }
                *reinterpret_cast<uint4 *>(smem + OFF_WLO + sw64_offset(r, h0)) = make_uint4(wlo[0], wlo[1], wlo[2], wlo[3]);
                auto rescale_trip = [&](int c0) {
                    uint32_t o[2][kHG];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x16(tmem + lane_addr + TM_O + 64u * (c0 + c) + (uint32_t)h0, o[c]);
                    tmem_wait_ld();
                    const float *al = ms.alpha[grp];
#pragma unroll
                    for (int j4 = 0; j4 < kV4; ++j4) {
                        const float4 a4 = *reinterpret_cast<const float4 *>(al + 4 * j4);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t *oc = &o[c][4 * j4];
                            oc[0] = __float_as_uint(__uint_as_float(oc[0]) * a4.x);
                            oc[1] = __float_as_uint(__uint_as_float(oc[1]) * a4.y);
                            oc[2] = __float_as_uint(__uint_as_float(oc[2]) * a4.z);
                            oc[3] = __float_as_uint(__uint_as_float(oc[3]) * a4.w);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_st_32x32b_x16(tmem + lane_addr + TM_O + 64u * (c0 + c) + (uint32_t)h0, o[c]);
                };
                const bool rescale = any_alpha && t > seg.t0;
                if (it >= 1) wait(&ms.done[(it - 1) & 1], ((it - 1) >> 1) & 1);
                *reinterpret_cast<uint4 *>(smem + OFF_WHI + sw64_offset(r, h0)) = make_uint4(whi[0], whi[1], whi[2], whi[3]);
                if (rescale) {
                    tc_fence_after_sync();
                    rescale_trip(0);
                    rescale_trip(2);
                    tmem_wait_st();
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                mbar_arrive(&ms.w_full);
            }

            // ---- output: sums over the warp's rows (lane l ends up with column l % 16), then over the quadrants
            auto over_rows = [&](float (&v)[kHG]) -> float {
#pragma unroll
                for (int k = kHG / 2; k >= 1; k >>= 1) {
                    const bool upper = (lane & k) != 0;
#pragma unroll
                    for (int j = 0; j < k; ++j) {
                        const float send = upper ? v[j] : v[j + k], keep = upper ? v[j + k] : v[j];
                        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, k);
                    }
                }
                return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
            };
            const int hcol = h0 + (lane & (kHG - 1));
            auto over_quadrants = [&]() -> float { return ms.red[0][hcol] + ms.red[1][hcol] + ms.red[2][hcol] + ms.red[3][hcol]; };
            float nn = 0.f;
            float z[kHG];
            // (the barrier also says that a last slow path's readers of red are done)
            if (bar_red_or(bar_id, 128, n0 != 0 || n0_draft != 0)) {
#pragma unroll
                for (int j = 0; j < kHG; ++j) z[j] = (float)(n0 + (n0_draft >> j & 1) + 2 * (n0_draft >> (16 + j) & 1));
                const float nw = over_rows(z);
                if (lane < kHG) ms.red[q][hcol] = nw;
                named_sync(bar_id, 128);
                nn = over_quadrants() * exp2f(kUp);
                named_sync(bar_id, 128);
            }
#pragma unroll
            for (int j = 0; j < kP; ++j) f2_unpack(z2[j], z[2 * j], z[2 * j + 1]);
            const float zw = over_rows(z);
            if (lane < kHG) ms.red[q][hcol] = zw;
            wait(&ms.done[(it - 1) & 1], ((it - 1) >> 1) & 1);
            tc_fence_after_sync();
            named_sync(bar_id, 128);
            const bool whole = seg.first && seg.last;
            const float zz = over_quadrants();
            const int c0 = seg.g * kCols, nc = min(kCols, seg.q.n * a.H - c0);
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (seg.first ? 1 : 0)) * tree_part_floats(kCols);
            const float mm = ms.m_run[cur][hcol];
            if (lane < kHG) {  // the same from all four warps
                // nothing but zero rows: the accumulators are 0 and stay so
                const float all = nn == 0.f ? zz : zz + nn * exp2f(mm == -INFINITY ? 0.f : -mm);
                ms.alpha[grp][lane] = !whole ? 1.f : all == 0.f ? 0.f : 1.f / all;
            }
            if (!whole && q == 0 && lane < kHG) {
                part[kCols * kKL + hcol] = mm;
                part[kCols * (kKL + 1) + hcol] = zz;
                part[kCols * (kKL + 2) + hcol] = nn;
            }
            __syncwarp();
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    // thread: dim 128 c + r of 16 columns
                    uint32_t o[kHG];
                    tmem_ld_32x32b_x16(tmem + lane_addr + TM_O + 64u * c + (uint32_t)h0, o);
                    tmem_wait_ld();
                    float v[kHG];
#pragma unroll
                    for (int j4 = 0; j4 < kV4; ++j4) {
                        const float4 a4 = *reinterpret_cast<const float4 *>(&ms.alpha[grp][4 * j4]);
                        v[4 * j4] = __uint_as_float(o[4 * j4]) * a4.x;
                        v[4 * j4 + 1] = __uint_as_float(o[4 * j4 + 1]) * a4.y;
                        v[4 * j4 + 2] = __uint_as_float(o[4 * j4 + 2]) * a4.z;
                        v[4 * j4 + 3] = __uint_as_float(o[4 * j4 + 3]) * a4.w;
                    }
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < kHG; ++j)
                            if (h0 + j < nc) part[(h0 + j) * kKL + 128 * c + r] = v[j];
                    } else if (a.out_bf16) {
                        // even lanes store column j, odd lanes column j + 1: two dims each
                        const bool odd = lane & 1;
#pragma unroll
                        for (int j = 0; j < kHG; j += 2) {
                            const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                            const __nv_bfloat162 pk = odd ? __floats2bfloat162_rn(other, v[j + 1]) : __floats2bfloat162_rn(v[j], other);
                            const int col = h0 + j + (odd ? 1 : 0);
                            if (col < nc)
                                *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                                    ((int64_t)seg.q.q0 * a.H + c0 + col) * kKL + 128 * c + (r & ~1)) = pk;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kHG; ++j)
                            if (h0 + j < nc)
                                static_cast<float *>(a.out)[((int64_t)seg.q.q0 * a.H + c0 + h0 + j) * kKL + 128 * c + r] = v[j];
                    }
                }
            }
            tc_fence_before_sync();  // the accumulators' reads come before the next segment's first weights
        }
        if (bad_page && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

size_t tree_tc_images(int R, int H, int B) { return (size_t)(tree_slot(R, H, B)) * (kImg + kCols * sizeof(float)); }
size_t tree_tc_part_bytes(int ctas) { return (size_t)ctas * 2 * tree_part_floats(kCols) * sizeof(float); }

cudaError_t launch_tree_tc(const TreeArgs &a, void *images, cudaStream_t st) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    CUtensorMap m_lc, m_rc;
    const cuuint64_t dims[2] = {(cuuint64_t)kRow, (cuuint64_t)a.cache_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)kRow};
    const cuuint32_t rows = (cuuint32_t)(a.page_shift < 7 ? 1 << a.page_shift : kRows);
    const cuuint32_t box_lc[2] = {128, rows}, box_rc[2] = {64, rows}, es[2] = {1, 1};
    void *base = const_cast<uint8_t *>(a.kv8);
    if (encode(&m_lc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box_lc, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
            CUDA_SUCCESS ||
        encode(&m_rc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box_rc, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
            CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const size_t slots = (size_t)tree_slot(a.R, a.H, a.B);
    TcArgs x{};
    x.t = a;
    x.img = static_cast<uint8_t *>(images);
    x.c_head = reinterpret_cast<float *>(static_cast<uint8_t *>(images) + slots * kImg);
    cudaError_t e = cudaFuncSetAttribute(attn_tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(1 + ((int64_t)a.R * a.H + kPrepCols - 1) / kPrepCols));
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, tree_prep_kernel, a, const_cast<uint8_t *>(x.img), const_cast<float *>(x.c_head))) !=
        cudaSuccess)
        return e;
    cfg.gridDim = dim3((unsigned)a.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    if ((e = cudaLaunchKernelEx(&cfg, attn_tree_tc_kernel, m_lc, m_rc, x)) != cudaSuccess) return e;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_tree_merge(a, kCols, st);
}

}  // namespace kv8
