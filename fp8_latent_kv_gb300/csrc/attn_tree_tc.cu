// attn_tree_tc.cu -- attention of drafted tokens over a paged latent cache on the tensor cores (tcgen05, sm_103a),
// for bf16 queries.
//
// All (token, head) columns of a sequence read the same rows, so a group of 64 columns against a tile of 128 rows is
// two contractions:
//   score    S[x][t]    = sum_k Qs[x][k] K8[t][k]      M = 128, N = 2 x 64 rows, K = 576 (e4m3 x e4m3)
//            Qs: a bf16 query element, scaled by its column's power of two, is the sum of two e4m3 values; each
//            TMEM lane quadrant holds 16 columns' hi pieces on lanes 0..15 and their lo pieces on lanes 16..31, so
//            that one shuffle adds the halves of the dot product.
//   context  O^T[d][n] += sum_t V8[t][d] W[n][t]       M = 128 dims (x4), N = 64 columns, K = 128 rows; V8 = the same
//            bytes read MN-major, W the softmax weights as two pieces, hi in e4m3 and lo, what hi leaves, in e5m2:
//            2^-7 of a weight at most, and terms down to 2^-21 of the column's largest still count (two e4m3 pieces
//            would round everything below 2^-16 to nothing, which a long context's many small terms add up to).
// Weights: with e_t = score_t log2(e) + log2(scale_t) and a running reference m >= max e - 3.75 for each column,
// w_t = 2^(e_t - m + 5) <= 2^8.75 holds the row scale already, O = sum w_t v_t and z = sum w_t / scale_t; the factor
// 2^5 cancels.  A weight's share of e4m3's range then follows its own column's largest term whatever rows, drafted
// or not, other columns attend.  A row whose scale is below 2^-100 (zeros, subnormal maxima) has score 0 and adds
// nothing to O: such rows are only counted, and the count enters z as n0 2^-m at the end.
//
// Work: equal shares of (group, tile) units (tree.cuh), one CTA per SM.
// Warps: 0 = row loads, 1 = scores and TMEM, 2 = the rows' scales, 3 = context products, 4..19 = softmax and output; warp % 4 is a
// warp's TMEM lane quadrant, its set (0..3) picks 32 of the tile's rows, and a thread holds 16 rows of one column.
// The query pieces are the score's A operand in TMEM, so shared memory holds rows: five stages of 64 rows (36 KB),
// two 16 KB weight buffers, the queries' RoPE part (8 KB).  A stage is held from its load through score, softmax and
// context product; with two stages of 128 rows beside a 72 KB query image that chain set the pace.
// TMEM: query 128 columns, score 128, context accumulators 4 x 64.
// Every wait is bounded in time; one that gives up sets KV8_ERR_TIMEOUT and the CTA winds down.
#include "sm100.cuh"
#include "tree.cuh"

#include <math.h>
#include <stddef.h>

namespace kv8 {
namespace {

using namespace sm100;

constexpr int kCols = 64;
constexpr int kRows = 64;
constexpr int kStages = 5;
constexpr int kSegment = 8;                // a segment's start and end cost about as much as this many tiles
constexpr int kTeam = 256;                 // threads of a softmax team
constexpr int kThreads = 128 + 2 * kTeam;
constexpr uint32_t kBlk = 8192;            // 64 rows x 128 latent bytes (SW128)
constexpr uint32_t kRope = 4096;           // 64 rows x 64 RoPE bytes (SW64)
constexpr uint32_t kStage = 4 * kBlk + kRope;
constexpr uint32_t kQLat = 128 * 512;      // a group's query image: 128 lanes x 512 latent bytes, row-major,
constexpr uint32_t kQRope = 128 * 64;      // then 128 x 64 RoPE bytes (SW64)
constexpr uint32_t kImg = kQLat + kQRope;
constexpr uint32_t kW = 8192;              // hi [64 columns][64 rows] (SW64), then lo
constexpr uint32_t OFF_ST = 0, OFF_W = kStages * kStage, OFF_Q = OFF_W + 2 * kW, OFF_MISC = OFF_Q + kQRope;
constexpr float kTau = 3.75f;              // the reference moves when a term exceeds it by more than 2^kTau
constexpr float kUp = 5.0f;                // weights are held times 2^kUp: at most 2^8.75 < 448
constexpr float kTiny = 7.888609e-31f;     // 2^-100
constexpr uint32_t TM_Q = 0, TM_S = 128, TM_O = 256;

struct RowInfo {
    alignas(16) float scale[kRows];        // 0 for rows that are not there
    alignas(16) float lg[kRows];           // log2(scale) + kUp
    alignas(16) float inv[kRows];          // 1 / scale
    uint64_t in, zero;                     // rows that are there / whose scale is below 2^-100
};
struct Misc {
    RowInfo rows[kStages];
    alignas(16) float m[kCols];            // running references (log2 units), -inf before any attended row
    alignas(16) float red[4][kCols];       // maxima of a team's two sets of rows, team by team; at the end sums
    alignas(16) float zinv[kCols];         // at the end: 1 / z
    uint64_t kv_full[kStages], kv_free[kStages], row_full[kStages], s_full[2], s_free[2], w_full[2], pv_done[2], q_ready,
        final_bar[2];
    uint32_t tmem_base;
    int abort_flag;
};
constexpr uint32_t kSmemBytes = OFF_MISC + sizeof(Misc);
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(offsetof(Misc, kv_full) % 8 == 0 && OFF_MISC % 1024 == 0 && OFF_W % 1024 == 0 && kStage % 1024 == 0, "alignment");

struct TcArgs {
    TreeArgs t;
    const uint8_t *img;    // query images, one kImg for each group
    const float *c_head;   // [images][64]: sm_scale * log2(e) * 2^-e of the column's query
};

// A sequence's groups' images begin at slot q0 * H / 64 + b: never past the next sequence's first.
__host__ __device__ __forceinline__ int64_t tree_slot(int64_t q0, int H, int b) { return q0 * H / kCols + b; }

// Lane of column n's piece (0 = hi, 1 = lo).
__device__ __forceinline__ int query_lane(int n, int piece) { return (n >> 4) * 32 + piece * 16 + (n & 15); }

// Arrive at a named barrier that other threads wait at; what this thread wrote before is theirs to read after it.
__device__ __forceinline__ void named_arrive(int id, int count) {
    __threadfence_block();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// 16 lanes x 32 consecutive 32-bit columns: register 4 i + k of lane l holds lane l / 4 + 8 (k / 2), column
// 8 i + 2 (l % 4) + k % 2.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// Score MMA with A in tensor memory.
__device__ __forceinline__ void mma_f8f6f4_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Bounded wait on the SM's own clock: reading the global timer takes about a microsecond, which a wait that is not
// ready at once would pay every time.  2^32 cycles are two seconds; drains give a shorter limit.
constexpr long long kLimit = 1ll << 32;

__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *err,
                                         long long limit = kLimit) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 31u) == 0) {
            if (abort_flag && *abort_flag) return false;
            if (clock64() - t0 > limit) {
                if (abort_flag) *abort_flag = 1;
                if (err) atomicOr(err, (int)KV8_ERR_TIMEOUT);
                return false;
            }
        }
    }
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(p));
    return p != 0;
}

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
// Two softmax weights (at most 2^8.75) -> e4m3 pieces and e5m2 pieces of what those leave.  By way of f16, whose 11
// bits are finer than the 7 that the pieces keep; the residual is exact there.
__device__ __forceinline__ void split_weights(float a, float b, uint16_t &hi, uint16_t &lo) {
    uint32_t w16, h16, r16;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w16) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(w16));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r16) : "r"(w16), "r"(h16));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r16));
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
// Byte offset of 16-byte chunk ch (32 latent, 4 RoPE) of a lane's query pieces.
__device__ __forceinline__ uint32_t image_offset(int lane, int ch) {
    return ch < 32 ? (uint32_t)lane * 512u + ch * 16u : kQLat + sw64_offset(lane, (ch - 32) * 16);
}

constexpr int kPrepCols = 8, kPrepThreads = kPrepCols * 36;

__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(TreeArgs a, uint8_t *img, float *c_head) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ int64_t scan[66];
    __shared__ int qmax_bits[kPrepCols];
    __shared__ int64_t pad_slot[kPrepCols];
    __shared__ int pad_from[kPrepCols];
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        tree_schedule<kCols, kRows, kSegment>(a, scan);
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
        const uint32_t off_hi = image_offset(query_lane(n, 0), ch), off_lo = image_offset(query_lane(n, 1), ch);
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
            const int n = from + i / 72, p = i % 72;
            const uint32_t off = image_offset(query_lane(n, p / 36), p % 36);
            *reinterpret_cast<uint4 *>(dst + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        for (int n = from + tid; n < kCols; n += kPrepThreads) c_head[pad_slot[c] * kCols + n] = 0.f;
    }
}

// ------------------------------------------------------------------------------------------------------------
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
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ms.kv_full[s], 1);
            mbar_init(&ms.kv_free[s], 1);
            mbar_init(&ms.row_full[s], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&ms.s_full[k], 1);
            mbar_init(&ms.s_free[k], kTeam / 32);  // one arrival for each warp
            mbar_init(&ms.w_full[k], kTeam / 32);
            mbar_init(&ms.pv_done[k], 1);
        }
        mbar_init(&ms.q_ready, 2 * kTeam / 32);
        mbar_init(&ms.final_bar[0], 1);
        mbar_init(&ms.final_bar[1], 1);
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
        // ================================ row loads ================================
        // Lane l fetches the tile's l-th piece (a page, or the tile where pages are larger); pieces past the
        // sequence's rows or outside the cache are not loaded.  A stage's barrier is armed after its release, which
        // implies that its previous phase is complete.
        const int sub_rows = min(kRows, 1 << a.page_shift), subs = kRows / sub_rows;
        int it = 0, s = 0;
        uint32_t ph = 1;  // parity of the release that stage s waits for
        bool ok = true;
        while (ok && walk.next<kCols, kRows>(a, seg)) {
            const int64_t end = seg.q.len + seg.q.n;
            auto piece = [&](int t) -> int64_t {
                const int64_t pos = (int64_t)t * kRows + (int64_t)lane * sub_rows;
                return lane < subs && pos < end ? tree_row(a, seg.b, pos) : -1;
            };
            int64_t next = piece(seg.t0);
            for (int t = seg.t0; t < seg.t1; ++t, ++it) {
                const int64_t row = next;
                next = t + 1 < seg.t1 ? piece(t + 1) : -1;  // a page entry's latency ahead
                const int pieces = __popc(__ballot_sync(0xffffffffu, row >= 0));
                if (it >= kStages) ok = __all_sync(0xffffffffu, bar_wait(&ms.kv_free[s], ph, &ms.abort_flag, a.err_word));
                if (!ok) break;
                uint8_t *st = smem + OFF_ST + s * kStage;
                if (lane == 0) mbar_arrive_expect_tx(&ms.kv_full[s], (uint32_t)pieces * sub_rows * (uint32_t)kRow);
                __syncwarp();
                if (row >= 0) {
                    if (subs == 1) {  // one copy for the four latent blocks
                        tma_load_3d(st, &map_lc, 0, (int)row, 0, &ms.kv_full[s]);
                    } else {
#pragma unroll
                        for (int kb = 0; kb < 4; ++kb)
                            tma_load_3d(st + kb * kBlk + lane * sub_rows * 128, &map_lc, 0, (int)row, kb, &ms.kv_full[s]);
                    }
                    tma_load_2d(st + 4 * kBlk + lane * sub_rows * 64, &map_rc, 512, (int)row, &ms.kv_full[s]);
                }
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        // every load in flight lands before the CTA ends
        if (lane == 0)
            for (int i = max(0, it - kStages); i < it; ++i)
                bar_wait(&ms.kv_full[i % kStages], (i / kStages) & 1, nullptr, a.err_word, kLimit / 8);
        __syncwarp();
    } else if (warp == 1) {
        // ================================ scores ================================
        // The whole warp runs the loop and one elected lane issues: operands stay in uniform registers.  (Issued from
        // `if (lane == 0)` the same MMAs took 46 cycles each instead of 32 alone, and 85 beside the softmax warps.)
        // Scores and context products have a warp each: the tensor core's queue takes a few MMAs only, so the hundreds
        // of cycles that an issuer spends on its waits are the core's idle time unless another one issues meanwhile.
        const uint32_t id_s = idesc_e4m3_f32(128, kRows, false, false);
        // descriptors of stage 0 and of the query's RoPE part: an offset adds to the address field
        const uint64_t k_desc = smem_desc(sbase + OFF_ST, 0, 1024, kSw128);
        const uint64_t kr_desc = smem_desc(sbase + OFF_ST + 4 * kBlk, 0, 512, kSw64);
        const uint64_t qr_desc = smem_desc(sbase + OFF_Q, 0, 512, kSw64);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = bar_wait(bar, parity, &ms.abort_flag, a.err_word);
            ok = __all_sync(0xffffffffu, ok);
        };
        int j = 0, sg = 0, s = 0;  // tiles, segments, the stage
        uint32_t s_ph = 0;
        while (ok && walk.next<kCols, kRows>(a, seg)) {
            wait(&ms.q_ready, sg & 1);
            ++sg;
            for (int t = seg.t0; ok && t < seg.t1; ++t, ++j) {
                wait(&ms.kv_full[s], s_ph);
                if (j >= 2) wait(&ms.s_free[j & 1], ((j >> 1) - 1) & 1);
                tc_fence_after_sync();
                if (ok && elect_one()) {
                    const uint32_t d = tmem + TM_S + 64u * (j & 1);
                    const uint64_t k = k_desc + (uint64_t)(s * (kStage >> 4)), kr = kr_desc + (uint64_t)(s * (kStage >> 4));
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f8f6f4_ts(d, tmem + TM_Q + kb * 32 + kk * 8, k + (uint64_t)((kb * kBlk + kk * 32) >> 4), id_s, (kb | kk) != 0);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) mma_f8f6f4(d, qr_desc + (uint64_t)(kk * 2), kr + (uint64_t)(kk * 2), id_s, 1u);
                    mma_commit(&ms.s_full[j & 1]);
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    s_ph ^= 1;
                }
            }
        }
        if (elect_one()) mma_commit(&ms.final_bar[0]);  // all issued MMAs complete before the CTA tears down
        __syncwarp();
        bar_wait(&ms.final_bar[0], 0, nullptr, a.err_word, kLimit / 8);
        __syncwarp();
    } else if (warp == 3) {
        // ================================ context products ================================
        const uint32_t id_hi = idesc_e4m3_f32(128, kCols, true, false), id_lo = id_hi | (1u << 10);  // B in e5m2
        const uint64_t v_desc = smem_desc(sbase + OFF_ST, 0, 1024, kSw128);  // (the score's bytes, MN-major)
        const uint64_t w_desc = smem_desc(sbase + OFF_W, 0, 512, kSw64);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = bar_wait(bar, parity, &ms.abort_flag, a.err_word);
            ok = __all_sync(0xffffffffu, ok);
        };
        int i = 0, s = 0;
        uint32_t s_ph = 0;
        while (ok && walk.next<kCols, kRows>(a, seg)) {
            for (int t = seg.t0; ok && t < seg.t1; ++t, ++i) {
                wait(&ms.kv_full[s], s_ph);  // (complete since before the score)
                wait(&ms.w_full[i & 1], (i >> 1) & 1);
                tc_fence_after_sync();
                if (ok && elect_one()) {
                    const uint64_t v = v_desc + (uint64_t)(s * (kStage >> 4));
                    const uint64_t w = w_desc + (uint64_t)((i & 1) * (kW >> 4));
                    const uint32_t keep = t > seg.t0;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            const uint64_t av = v + (uint64_t)((ch * kBlk + kk * 4096) >> 4);
                            mma_f8f6f4(tmem + TM_O + 64u * ch, av, w + (uint64_t)((kk * 32) >> 4), id_hi, kk ? 1u : keep);
                            mma_f8f6f4(tmem + TM_O + 64u * ch, av, w + (uint64_t)((kW / 2 + kk * 32) >> 4), id_lo, 1u);
                        }
                    mma_commit(&ms.kv_free[s]);
                    mma_commit(&ms.pv_done[i & 1]);
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    s_ph ^= 1;
                }
            }
        }
        if (elect_one()) mma_commit(&ms.final_bar[1]);
        __syncwarp();
        bar_wait(&ms.final_bar[1], 0, nullptr, a.err_word, kLimit / 8);
        __syncwarp();
    } else if (warp == 2) {
        // ================================ the rows' scales ================================
        // Four stages at a time, eight rows per lane: their page entries, then their scales, one latency each; the
        // stages' five sets of row figures keep this ahead of the softmax.
        constexpr int kBatch = 4;
        int is = 0;
        bool ok = true, bad_page = false;
        while (ok && walk.next<kCols, kRows>(a, seg)) {
            const int64_t end = seg.q.len + seg.q.n;
            for (int t = seg.t0; ok && t < seg.t1; t += kBatch) {
                int64_t row[2 * kBatch];
                float sc[2 * kBatch];
#pragma unroll
                for (int u = 0; u < 2 * kBatch; ++u) {
                    const int64_t pos = (int64_t)t * kRows + 32 * u + lane;
                    row[u] = -1;
                    if (t + u / 2 < seg.t1 && pos < end) {
                        row[u] = tree_row(a, seg.b, pos);
                        bad_page |= row[u] < 0;
                    }
                }
#pragma unroll
                for (int u = 0; u < 2 * kBatch; ++u) sc[u] = row[u] >= 0 ? __ldg(a.kv_scale + row[u]) : 0.f;
#pragma unroll
                for (int v = 0; v < kBatch; ++v) {
                    if (t + v >= seg.t1) break;
                    const int s = is % kStages;
                    if (is >= kStages)
                        ok = __all_sync(0xffffffffu, bar_wait(&ms.kv_free[s], (is / kStages - 1) & 1, &ms.abort_flag, a.err_word));
                    if (!ok) break;
                    RowInfo &ri = ms.rows[s];
                    uint32_t in[2], zero[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float c = sc[2 * v + k];
                        const bool there = row[2 * v + k] >= 0;
                        in[k] = __ballot_sync(0xffffffffu, there);
                        zero[k] = __ballot_sync(0xffffffffu, there && c < kTiny);
                        ri.scale[32 * k + lane] = c;
                        ri.lg[32 * k + lane] = lg2_approx(c) + kUp;
                        // 0 for a zero row (its weight is 0) and for a scale that is not finite (its weight is NaN
                        // where it is attended)
                        ri.inv[32 * k + lane] = c >= kTiny && c <= 3.402823466e38f ? __fdividef(1.f, c) : 0.f;
                    }
                    if (lane == 0) {
                        ri.in = in[0] | (uint64_t)in[1] << 32;
                        ri.zero = zero[0] | (uint64_t)zero[1] << 32;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.row_full[s]);
                    ++is;
                }
            }
        }
        if (bad_page && a.err_word) atomicOr(a.err_word, (int)KV8_ERR_INDEX);
    } else {
        // ============================ softmax and output ============================
        // A wait that gives up clears `ok` (the same in a warp's lanes: TMEM accesses need all of them); the warp
        // then skips its remaining waits but still reaches every named barrier, so that no other warp waits for it.
        const int st = tid - 128;                     // 0..511
        const int q = warp & 3, w16 = (warp - 4) >> 2;
        const int team = w16 >> 1, set = w16 & 1;     // tiles of the team's parity; rows 32 set .. 32 set + 31 of them
        // A 16-lane TMEM load of 8 columns hands lane l rows 2 (l % 4) and 2 (l % 4) + 1 of columns l / 4 and l / 4 + 8: the
        // hi and lo pieces' loads match register by register.  So a thread holds, for two columns, rows 8 i + 2 (l % 4)
        // and the next, i < 4, of its set's 32.
        const int n_a = 16 * q + (lane >> 2), n_b = n_a + 8;
        const int r0 = 32 * set + 2 * (lane & 3);     // its first row
        const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
        const int team_bar = 2 + team;                // the team's own barrier
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar, parity, &ms.abort_flag, a.err_word));
        };
        grid_launch_dependents();
        int it = 0, s = 0;  // tiles and stages, the other team's included
        uint32_t s_ph = 0;
        while (walk.next<kCols, kRows>(a, seg)) {
            const int64_t slot = tree_slot(seg.q.q0, a.H, seg.b) + seg.g;
            // ---- the group's queries: 128 latent bytes of this thread's lane to TMEM, one RoPE chunk to shared memory.
            // (The scores of the segment before are complete: its last one was read before the output's barriers.)
            {
                const uint8_t *img = x.img + slot * kImg;
                const uint4 *src = reinterpret_cast<const uint4 *>(img + (32 * q + lane) * 512 + w16 * 128);
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __ldg(src + k);
                const uint4 rp = __ldg(reinterpret_cast<const uint4 *>(img + kQLat) + st);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t w[16] = {v[4 * k].x,     v[4 * k].y,     v[4 * k].z,     v[4 * k].w,
                                            v[4 * k + 1].x, v[4 * k + 1].y, v[4 * k + 1].z, v[4 * k + 1].w,
                                            v[4 * k + 2].x, v[4 * k + 2].y, v[4 * k + 2].z, v[4 * k + 2].w,
                                            v[4 * k + 3].x, v[4 * k + 3].y, v[4 * k + 3].z, v[4 * k + 3].w};
                    tmem_st_32x32b_x16(tmem + lane_addr + TM_Q + w16 * 32 + 16 * k, w);
                }
                *reinterpret_cast<uint4 *>(smem + OFF_Q + st * 16) = rp;
                if (st < kCols) ms.m[st] = -INFINITY;
                tmem_wait_st();
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.q_ready);
            }
            named_sync(1, 2 * kTeam);
            const float c_a = __ldg(x.c_head + slot * kCols + n_a), c_b = __ldg(x.c_head + slot * kCols + n_b);
            const int top = seg.q.n * a.H;
            float m_a = -INFINITY, m_b = -INFINITY;             // the references that z is relative to: the team's last
            uint64_t z_a = f2_pack(0.f, 0.f), z_b = f2_pack(0.f, 0.f);
            int zero_a = 0, zero_b = 0;                         // zero rows that the columns attend among this thread's
            for (int t = seg.t0; t < seg.t1; ++t, ++it) {
                const bool mine = (it & 1) == team;
                const int s_now = s;
                const uint32_t ph_now = s_ph;
                if (++s == kStages) {
                    s = 0;
                    s_ph ^= 1;
                }
                if (!mine) continue;
                const int64_t p0 = (int64_t)t * kRows;
                // ---- scores
                wait(&ms.s_full[team], (it >> 1) & 1);
                tc_fence_after_sync();
                uint32_t hi[16], lo[16];
                tmem_ld_16x256b_x4(tmem + lane_addr + TM_S + 64u * team + 32u * set, hi);
                tmem_ld_16x256b_x4(tmem + lane_addr + (16u << 16) + TM_S + 64u * team + 32u * set, lo);
                // meanwhile the rows' figures, and which rows the columns attend (bit 2 i + k: row r0 + 8 i + k)
                wait(&ms.row_full[s_now], ph_now);
                const RowInfo &ri = ms.rows[s_now];
                const uint64_t in = ri.in;
                const bool drafted = p0 + kRows > seg.q.len;
                const bool plain = !drafted && in == ~(uint64_t)0 && ri.zero == 0;  // every column attends every row
                uint32_t on_a = 0xFFu, on_b = 0xFFu;
                if (!plain) {
                    on_a = on_b = 0;
                    const int c0 = seg.g * kCols, node_a = min(c0 + n_a, top - 1) / a.H, node_b = min(c0 + n_b, top - 1) / a.H;
#pragma unroll 1
                    for (int u = 0; u < 8; ++u) {
                        const int r = r0 + 8 * (u >> 1) + (u & 1);
                        if (!(in >> r & 1)) continue;
                        const int64_t draft = p0 + r - seg.q.len;  // the row's index in the draft
                        const bool sa = draft < 0 || tree_sees(a, seg.q.q0, node_a, (int)draft);
                        const bool sb = draft < 0 || tree_sees(a, seg.q.q0, node_b, (int)draft);
                        if (ri.zero >> r & 1) {
                            zero_a += sa;
                            zero_b += sb;
                        } else {
                            on_a |= (uint32_t)sa << u;
                            on_b |= (uint32_t)sb << u;
                        }
                    }
                }
                tmem_wait_ld();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.s_free[team]);
                // ---- e + 5, row pairs packed: 0..3 of column a, 4..7 of column b
                uint64_t d2[8];
                float max_a = -INFINITY, max_b = -INFINITY;
                {
                    const uint64_t ca = f2_pack(c_a, c_a), cb = f2_pack(c_b, c_b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 sc = *reinterpret_cast<const float2 *>(&ri.scale[r0 + 8 * i]);
                        const float2 lg = *reinterpret_cast<const float2 *>(&ri.lg[r0 + 8 * i]);
                        const uint64_t sc2 = f2_pack(sc.x, sc.y), lg2 = f2_pack(lg.x, lg.y);
                        const uint64_t sa = f2_add(f2_pack(__uint_as_float(hi[4 * i]), __uint_as_float(hi[4 * i + 1])),
                                                   f2_pack(__uint_as_float(lo[4 * i]), __uint_as_float(lo[4 * i + 1])));
                        const uint64_t sb = f2_add(f2_pack(__uint_as_float(hi[4 * i + 2]), __uint_as_float(hi[4 * i + 3])),
                                                   f2_pack(__uint_as_float(lo[4 * i + 2]), __uint_as_float(lo[4 * i + 3])));
                        d2[i] = f2_fma(sa, f2_mul(sc2, ca), lg2);
                        d2[4 + i] = f2_fma(sb, f2_mul(sc2, cb), lg2);
                    }
                    if (!plain) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float u, v;
                            f2_unpack(d2[i], u, v);
                            d2[i] = f2_pack(on_a >> (2 * i) & 1 ? u : -INFINITY, on_a >> (2 * i + 1) & 1 ? v : -INFINITY);
                            f2_unpack(d2[4 + i], u, v);
                            d2[4 + i] = f2_pack(on_b >> (2 * i) & 1 ? u : -INFINITY, on_b >> (2 * i + 1) & 1 ? v : -INFINITY);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float u, v;
                        f2_unpack(d2[i], u, v);
                        max_a = fmaxf(max_a, fmaxf(u, v));
                        f2_unpack(d2[4 + i], u, v);
                        max_b = fmaxf(max_b, fmaxf(u, v));
                    }
                }
                // ---- the references, tile after tile: the other team has decided on the tile before.  They move
                // together when a term exceeds one by more than kTau, or a column that has none meets its first row.
                if (t > seg.t0) named_sync(4 + (team ^ 1), 2 * kTeam);
                float na = ms.m[n_a], nb = ms.m[n_b];
                const float m_c = ms.m[32 * set + lane];  // of the accumulator columns that this warp rescales
                const bool slow = bar_red_or(team_bar, kTeam, max_a > na + (kTau + kUp) || max_b > nb + (kTau + kUp));
                float move = 1.f;                         // that column's factor
                if (slow) {
                    max_a = fmaxf(max_a, __shfl_xor_sync(0xffffffffu, max_a, 1));
                    max_b = fmaxf(max_b, __shfl_xor_sync(0xffffffffu, max_b, 1));
                    max_a = fmaxf(max_a, __shfl_xor_sync(0xffffffffu, max_a, 2));
                    max_b = fmaxf(max_b, __shfl_xor_sync(0xffffffffu, max_b, 2));
                    if ((lane & 3) == 0) {
                        ms.red[w16][n_a] = max_a;
                        ms.red[w16][n_b] = max_b;
                    }
                    named_sync(team_bar, kTeam);
                    auto moved = [&](int n, float m) -> float {
                        const float top_e = fmaxf(ms.red[2 * team][n], ms.red[2 * team + 1][n]) - kUp;
                        return top_e > m + kTau ? top_e : m;
                    };
                    na = moved(n_a, na);
                    nb = moved(n_b, nb);
                    const float nc = moved(32 * set + lane, m_c);
                    if (q == 0) ms.m[32 * set + lane] = nc;  // (all have read the old ones)
                    move = m_c == -INFINITY || nc == m_c ? 1.f : ex2_approx(m_c - nc);
                }
                if (t + 1 < seg.t1) named_arrive(4 + team, 2 * kTeam);
                if (m_a != na || m_b != nb) {  // z, relative to the team's last references, to these
                    const float fa = m_a == -INFINITY || m_a == na ? 1.f : ex2_approx(m_a - na);
                    const float fb = m_b == -INFINITY || m_b == nb ? 1.f : ex2_approx(m_b - nb);
                    z_a = f2_mul(z_a, f2_pack(fa, fa));
                    z_b = f2_mul(z_b, f2_pack(fb, fb));
                    m_a = na;
                    m_b = nb;
                }
                // the context product of the team's tile before has read this weight buffer
                if (it >= 2) wait(&ms.pv_done[team], ((it >> 1) - 1) & 1);
                // ---- weights 2^(e + 5 - m)
                {
                    const float ref_a = m_a == -INFINITY ? 0.f : -m_a, ref_b = m_b == -INFINITY ? 0.f : -m_b;
                    const uint64_t ra = f2_pack(ref_a, ref_a), rb = f2_pack(ref_b, ref_b);
                    uint8_t *const wb = smem + OFF_W + team * kW;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 inv = *reinterpret_cast<const float2 *>(&ri.inv[r0 + 8 * i]);
                        const uint64_t inv2 = f2_pack(inv.x, inv.y);
                        float u, v, x0, x1, y0, y1;
                        f2_unpack(f2_add(d2[i], ra), u, v);
                        x0 = ex2_approx(u);
                        x1 = ex2_approx(v);
                        f2_unpack(f2_add(d2[4 + i], rb), u, v);
                        y0 = ex2_approx(u);
                        y1 = ex2_approx(v);
                        z_a = f2_fma(f2_pack(x0, x1), inv2, z_a);
                        z_b = f2_fma(f2_pack(y0, y1), inv2, z_b);
                        uint16_t wh, wl;
                        split_weights(x0, x1, wh, wl);
                        uint8_t *p = wb + sw64_offset(n_a, r0 + 8 * i);
                        *reinterpret_cast<uint16_t *>(p) = wh;
                        *reinterpret_cast<uint16_t *>(p + kW / 2) = wl;
                        split_weights(y0, y1, wh, wl);
                        p = wb + sw64_offset(n_b, r0 + 8 * i);
                        *reinterpret_cast<uint16_t *>(p) = wh;
                        *reinterpret_cast<uint16_t *>(p + kW / 2) = wl;
                    }
                }
                // ---- rows that were not loaded, and NaN codes of drafted rows (attended columns have NaN weights
                // already): a weight of 0 must not meet them.  A thread owns a row's 128 bytes of a latent block.
                if (drafted || in != ~(uint64_t)0) {
                    const int r = st & 63;
                    const bool there = in >> r & 1;
                    if (!there || p0 + r >= seg.q.len) {
                        // (complete since before the score: this makes the copy's bytes visible here too)
                        (void)bar_wait(&ms.kv_full[s_now], ph_now, &ms.abort_flag, a.err_word);
                        uint4 *p = reinterpret_cast<uint4 *>(smem + OFF_ST + s_now * kStage + ((st >> 6) & 3) * kBlk + r * 128);
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) {
                            uint4 u = make_uint4(0u, 0u, 0u, 0u);
                            if (there) {
                                u = p[k];
                                u.x = without_nan(u.x);
                                u.y = without_nan(u.y);
                                u.z = without_nan(u.z);
                                u.w = without_nan(u.w);
                            }
                            p[k] = u;
                        }
                    }
                }
                if (slow && t > seg.t0 && __any_sync(0xffffffffu, move != 1.f)) {
                    // this warp's part of the accumulators, 32 columns by 32 dims of each block, where a column moved,
                    // once the context product before is complete.  (The one before that is: the wait above.)
                    wait(&ms.pv_done[team ^ 1], ((it - 1) >> 1) & 1);
                    tc_fence_after_sync();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!__any_sync(0xffffffffu, (lane >> 4) == h && move != 1.f)) continue;
                        const uint32_t at = tmem + lane_addr + TM_O + 32u * set + 16u * h;
#pragma unroll 1
                        for (int c = 0; c < 4; c += 2) {
                            uint32_t o[2][16];
                            tmem_ld_32x32b_x16(at + 64u * c, o[0]);
                            tmem_ld_32x32b_x16(at + 64u * (c + 1), o[1]);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float f = __shfl_sync(0xffffffffu, move, 16 * h + j);
                                o[0][j] = __float_as_uint(__uint_as_float(o[0][j]) * f);
                                o[1][j] = __float_as_uint(__uint_as_float(o[1][j]) * f);
                            }
                            tmem_st_32x32b_x16(at + 64u * c, o[0]);
                            tmem_st_32x32b_x16(at + 64u * (c + 1), o[1]);
                        }
                    }
                    tmem_wait_st();
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.w_full[team]);
            }

            // ---- output: sums over a column's threads, four lanes of each set
            const int c0 = seg.g * kCols, nc = min(kCols, top - c0);
            const bool whole = seg.first && seg.last;
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (seg.first ? 1 : 0)) * tree_part_floats(kCols);
            // returns the sum for column st (threads st < 64)
            auto over_sets = [&](float u, float v) -> float {
                u += __shfl_xor_sync(0xffffffffu, u, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                u += __shfl_xor_sync(0xffffffffu, u, 2);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                named_sync(1, 2 * kTeam);  // red's readers before this are done
                if ((lane & 3) == 0) {
                    ms.red[w16][n_a] = u;
                    ms.red[w16][n_b] = v;
                }
                named_sync(1, 2 * kTeam);
                const int n = st & (kCols - 1);
                return ms.red[0][n] + ms.red[1][n] + ms.red[2][n] + ms.red[3][n];
            };
            const float nn = over_sets((float)zero_a, (float)zero_b) * exp2f(kUp);
            float zz;
            {
                const float ea = ms.m[n_a], eb = ms.m[n_b];  // (the barriers above: both teams' last)
                float u, v, fa = m_a == -INFINITY ? 1.f : ex2_approx(m_a - ea), fb = m_b == -INFINITY ? 1.f : ex2_approx(m_b - eb);
                f2_unpack(z_a, u, v);
                fa *= u + v;
                f2_unpack(z_b, u, v);
                fb *= u + v;
                zz = over_sets(fa, fb);
            }
            if (st < kCols) {
                const float m_end = ms.m[st];
                // nothing but zero rows: the accumulators are 0 and stay so
                const float all = nn == 0.f ? zz : zz + nn * exp2f(m_end == -INFINITY ? 0.f : -m_end);
                ms.zinv[st] = !whole ? 1.f : all == 0.f ? 0.f : 1.f / all;
                if (!whole) {
                    part[kCols * kKL + st] = m_end;
                    part[kCols * (kKL + 1) + st] = zz;
                    part[kCols * (kKL + 2) + st] = nn;
                }
            }
            wait(&ms.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
            tc_fence_after_sync();
            named_sync(1, 2 * kTeam);
            const int h0 = 16 * w16;  // columns h0 .. h0 + 15
            if (ok) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    // thread: dim 128 c + 32 q + lane of columns h0 .. h0 + 15
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(tmem + lane_addr + TM_O + 64u * c + (uint32_t)h0, o);
                    tmem_wait_ld();
                    const int d = 128 * c + 32 * q + lane;
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 a4 = *reinterpret_cast<const float4 *>(&ms.zinv[h0 + 4 * k]);
                        v[4 * k] = __uint_as_float(o[4 * k]) * a4.x;
                        v[4 * k + 1] = __uint_as_float(o[4 * k + 1]) * a4.y;
                        v[4 * k + 2] = __uint_as_float(o[4 * k + 2]) * a4.z;
                        v[4 * k + 3] = __uint_as_float(o[4 * k + 3]) * a4.w;
                    }
                    if (!whole) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (h0 + j < nc) part[(h0 + j) * kKL + d] = v[j];
                    } else if (a.out_bf16) {
                        // even lanes store column j, odd lanes column j + 1: two dims each
                        const bool odd = lane & 1;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                            const __nv_bfloat162 pk = odd ? __floats2bfloat162_rn(other, v[j + 1]) : __floats2bfloat162_rn(v[j], other);
                            const int cj = h0 + j + (odd ? 1 : 0);
                            if (cj < nc)
                                *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                                    ((int64_t)seg.q.q0 * a.H + c0 + cj) * kKL + (d & ~1)) = pk;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (h0 + j < nc)
                                static_cast<float *>(a.out)[((int64_t)seg.q.q0 * a.H + c0 + h0 + j) * kKL + d] = v[j];
                    }
                }
            }
            tc_fence_before_sync();  // the accumulators' reads come before the next segment's first weights
        }
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
    // latent bytes as [4 blocks][rows][128 bytes], so that one copy lays four swizzled blocks down; RoPE bytes by row
    const bool whole = a.page_shift >= 6;  // a tile lies within a page
    const cuuint64_t dims_lc[3] = {128, (cuuint64_t)a.cache_rows, 4}, strides_lc[2] = {(cuuint64_t)kRow, 128};
    const cuuint64_t dims_rc[2] = {(cuuint64_t)kRow, (cuuint64_t)a.cache_rows}, strides_rc[1] = {(cuuint64_t)kRow};
    const cuuint32_t rows = (cuuint32_t)(whole ? kRows : 1 << a.page_shift);
    const cuuint32_t box_lc[3] = {128, rows, whole ? 4u : 1u}, box_rc[2] = {64, rows}, es[3] = {1, 1, 1};
    void *base = const_cast<uint8_t *>(a.kv8);
    if (encode(&m_lc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims_lc, strides_lc, box_lc, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) !=
            CUDA_SUCCESS ||
        encode(&m_rc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims_rc, strides_rc, box_rc, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
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
