// matmul8.cu -- product of e4m3 rows with an fmt=8 weight on the tensor cores (tcgen05, sm_103a).
//
//     out[m][n] = sum_kb  sa[kb][m] sw[n / 128][kb]  sum_{k in block kb} e4m3(a8[m][k]) e4m3(w8[n][k])
//
// The inner sums (128 exact products) run in kind::f8f6f4 MMAs with f32 accumulators; the scales change from one block of
// 128 to the next, so each block's sums leave TMEM, are multiplied by sa sw and added in f32 registers while the tensor
// cores work on the next block in other columns.
//
// Three arrangements of one kernel:
//   many rows, whole tiles (kSwap = kSplit = false): MMA rows are 128 rows of a8 (256 of a pair of blocks), columns kNT rows of
//     w8.  sa is one number a thread, sw one a warp.  Persistent blocks, one an SM, that take tile after tile.
//   many rows, shared tiles (kSwap = false, kSplit): tiles of 128 x 128, one for each cluster.
//   few rows (kSwap, kSplit): MMA rows are 128 rows of w8, columns kNT = 16 / 32 / 64 rows of a8, so that no MMA row is idle.  One
//     tile for each cluster, or block.  A tile reads its rows of the weight once; up to 16 tiles of kNT rows lie side by side,
//     and each of them reads the weight again (from the L2, where it holds them).  The columns' factors sa sw stand in shared memory.
// Where the tiles are fewer than the SMs, a cluster of up to 8 blocks shares a tile along K: each block owns some columns of
// the tile, the others store their sums for them into its shared memory, and it adds them in the order of their ranks (the
// result does not depend on timing, and no workspace is needed).
//
// What bounds it.  Many rows: a K block's 128 x 256 sums a block leave TMEM while the next one's are made, and with two
// accumulators of 256 columns filling TMEM the next but one waits for them: 512 cycles of products, about 550 until the end
// of the products has come to the adding warps and their end back to the issuing one, about 480 of loads and FMAs, for two
// blocks of K: 770 a block, tensor pipe 68 % active (8192 x 4096 x 16384: 363 us in bursts, 3.03 PFLOP/s; products alone 289 us).
// Taken and left, beside 357 us then: one block's 128 x 256 tile, which needs 48 KB a stage for the same work where a pair's needs 32 (452 us);
// sixteen adding warps (409), two MMAs of 128 columns a K block (398), loads of 32 columns at a time (403), or one ahead of the
// sums (406): TMEM loads in larger bursts hold up the products.  An output as large as the product's work
// is bound by its writes: 4096 x 32768 x 512 takes 78 us for 268 MB, which a plain fill writes in 71 us.
// Few rows: the weight's bytes (37 x 24576 x 2048: 14.8 us, 3.5 TB/s; 1 x 4096 x 16384: 14.3 us, 4.7 TB/s), of which about
// 3 us are a launch's way to its first bytes and 1 to 3 us the exchange of a split; where the tiles are not a multiple of the SMs,
// the SMs that hold two.
#include "elem.cuh"
#include "internal.h"
#include "sm100_more.cuh"

#include <math.h>

namespace kv8 {
namespace {

using namespace sm100;

constexpr int kMmBlk = KV8_KVB_BLOCK;  // K per scale block: 128 e4m3 bytes, one 128-byte swizzled row
constexpr int kMmRows = 128;           // MMA M
constexpr int kScaleBlocks = 4, kScaleSlots = 4;  // K blocks whose scales travel together, and slots of them
constexpr int kFirst = 4;              // the first warp that adds; warps 0 to 2 bring operands, issue products, bring scales
// Registers a thread of a pair's twelve warps: 4 x 40 + 8 x 232 = 12 x 168.  (One setmaxnreg for all four warps that hand some on, as
// the ISA has it: lowered in each warp's own part instead, 8192 x 4096 x 16384 took 2 % less in bursts and 4 % less at the power limit,
// 4096 x 32768 x 512 1 % more.  48 and 224: 2 % slower; no hand-over, 168 for all: 10 to 50 %, for sums that spill.)
constexpr int kRegsLoad = 40, kRegsAdd = 232;
constexpr int kGroupRows = 2048;       // rows of tiles that are walked together, for the L2's sake

struct MmArgs {
    const float *a_scale;
    int64_t a_scale_stride;  // between K blocks; 0: one scale a row
    const float *w_scale;
    void *out;
    int64_t out_stride;
    int M, N, kb;            // kb: blocks of 128 along K
    int p_tiles, q_tiles;    // tiles along the MMA rows' and columns' operand
    int split;               // blocks of a cluster, along K
    int tma_out;             // out can be written by tensor stores
    int *err_word;
};

// kNT: rows of the columns' operand.  With kNT = 256 two blocks are a pair: MMAs of 256 rows, half of both operands in each
// block.
template <bool kSwap, int kNT, int kStages>
struct MmShape {
    static constexpr bool kPair = kNT == 256;
    static constexpr int kEpi = kNT == 16 ? 4 : 8;             // warps that scale and add
    static constexpr int kThreads = 32 * (kFirst + kEpi);
    static constexpr int kCols = kNT / (kEpi / 4);             // accumulator columns of a thread
    static constexpr int kLoad = kPair ? kNT / 2 : kNT;        // rows of the columns' operand that a block loads
    static constexpr int kChunk = kNT >= 256 || kNT == 64 ? 16 : kCols < 32 ? kCols : 32;  // of which so many are loaded at a time,
    static constexpr int kBatch = kNT == 16 ? 4 : kNT == 32 ? 2 : 1;     // of so many K blocks together
    static constexpr int kAcc = kPair ? 2 : 4;                 // TMEM accumulators in turn
    static constexpr uint32_t kTmem = kNT * kAcc;
    static constexpr uint32_t kStage = (kMmRows + kLoad) * 128;
    static constexpr uint32_t kStaging = kEpi * 2 * 4096;
    static constexpr int kScales = (kSwap ? kNT : kMmRows) + 4;  // floats of a K block: those of a8's rows, then of w8's blocks
    static constexpr uint32_t kFac = kScaleSlots * kScaleBlocks * kScales * 4;
    // split (1, 2, 4 or 8): columns that a block owns, whose sums come from every rank; at least 4
    static constexpr __host__ __device__ int own(int split) {
        return kNT / split < 4 ? 4 : kNT / split;
    }
    static constexpr int kRedCols = kNT == 16 ? 32 : kNT;  // the most of split * own(split)
    static constexpr int kRedRow = kMmRows + 1;            // (rows of 16 bytes, so that neighbours in either direction lie in other banks)
    static constexpr uint32_t kRed = kRedCols / 4 * kRedRow * 16;
    static constexpr uint32_t bytes(bool split) {
        return 1024 + kStages * kStage + (split ? kRed : kStaging) + kFac + 256;
    }
};

// What is in flight when a warp ends its work.  A block whose shared memory a copy or a commit's arrival may still reach must
// not leave, and a barrier of all threads does not wait for either: of n K blocks the last ones' barriers are waited for.  (The
// phases before them have passed: a K block is loaded, or multiplied, when the one before it in its stage or accumulator has
// been used.)
template <int kBars>
__device__ __forceinline__ void phases_ended(uint64_t *bars, int n) {
#pragma unroll 1
    for (int i = n < kBars ? 0 : n - kBars; i < n; ++i) (void)bar_wait_inline(bars + i % kBars, (i / kBars) & 1, nullptr, nullptr, kDrainCycles);
}

// A wait gave up in one block of a pair.  The two may have loaded different numbers of K blocks, and block 0's barriers count both
// blocks' bytes.  The one that is behind loads as many (its stages are free: the other one saw them used), block 0 waits for the
// copies of both, block 1 for the commits that block 0 sent it.
template <typename S, int kStages>
__device__ __forceinline__ void even_out(const CUtensorMap &map_p, const CUtensorMap &map_q, uint8_t *smem, uint64_t *full, uint64_t *empty,
                                         uint64_t *t_full, const int *issued, const int *peer, uint32_t rank, int warp) {
    if (warp < 2 && elect_one()) cluster_store(of_rank(peer + 1 + warp, rank ^ 1), issued[warp]);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
        const int mine = issued[0], most = max(mine, *(const volatile int *)(peer + 1));
#pragma unroll 1
        for (int i = mine; i < most; ++i) {
            uint8_t *p = smem + i % kStages * S::kStage;
            if (elect_one()) {
                const uint32_t bar = of_rank(full + i % kStages, 0);
                if (rank == 0) mbar_arrive_expect_tx(full + i % kStages, 2 * S::kStage);
                tma_load_2d_pair(p, &map_p, 0, 0, bar);
                tma_load_2d_pair(p + kMmRows * 128, &map_q, 0, 0, bar);
            }
            __syncwarp();
        }
        if (rank == 0) phases_ended<kStages>(full, most);
    } else if (warp == 1 && rank == 1) {
        const int products = *(const volatile int *)(peer + 2);
        phases_ended<kStages>(empty, products);
        phases_ended<S::kAcc>(t_full, products);
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
}

// four values of a row, of which `left` exist
template <typename Out>
__device__ __forceinline__ void store_row(Out *p, const float (&v)[4], int left, bool wide) {
    if (wide && left >= 4) {
        store<4>(p, v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float one[1] = {v[j]};
            if (j < left) store<1>(p + j, one);
        }
    }
}

template <bool kSwap, int kNT, int kStages, int kBlocks, bool kBf16, bool kSplit>
__global__ void __launch_bounds__(MmShape<kSwap, kNT, kStages>::kThreads, kBlocks)
    matmul8_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                   const __grid_constant__ CUtensorMap map_out, const MmArgs a) {
    using S = MmShape<kSwap, kNT, kStages>;
    using Out = typename Elem<kBf16>::T;
    constexpr bool kPair = S::kPair;
    static_assert(!(kPair && kSplit) && (kSplit || !kSwap), "a cluster is a pair or a split");
    static_assert((S::bytes(kSplit) + 1024) * kBlocks <= 228 * 1024, "shared memory of an SM");
    constexpr uint32_t kOut = kSplit ? S::kRed : S::kStaging;  // staging of the output, or the sums of a split
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *staging = smem + kStages * S::kStage;
    float *fac = reinterpret_cast<float *>(staging + kOut);
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + kOut + S::kFac);
    uint64_t *full = bars, *empty = bars + kStages, *t_full = bars + 2 * kStages, *t_empty = t_full + S::kAcc;
    uint64_t *red_full = t_empty + S::kAcc, *s_full = red_full + 1, *s_empty = s_full + kScaleSlots;
    static_assert((2 * kStages + 2 * S::kAcc + 1 + 2 * kScaleSlots) * 8 + 28 <= 256, "barriers");
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(s_empty + kScaleSlots);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    int *issued = abort_flag + 1;  // (pair) K blocks loaded, K blocks multiplied
    int *peer = issued + 2;        // what the other block stores here: whether it gave up, and its `issued`

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (told to be the same in the whole warp: one row of 16384 10.2 -> 9.6 us)
    const int split = kSplit ? a.split : 1;
    const int rank = kSplit || kPair ? (int)cluster_rank() : 0;
    const int cluster = kPair ? 2 : split, first = (int)blockIdx.x / cluster, step = (int)gridDim.x / cluster;
    constexpr int kRows = kPair ? 2 * kMmRows : kMmRows;  // rows of a tile
    const int row0 = kPair ? rank * kMmRows : 0;          // this block's among them
    const int tiles = a.p_tiles * a.q_tiles;
    const int kb0 = kSplit ? (int)((int64_t)a.kb * rank / split) : 0, kb1 = kSplit ? (int)((int64_t)a.kb * (rank + 1) / split) : a.kb;

    // warp 0 makes the barriers and begins to load, warp 3 allocates the accumulators; the others wait for both
    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&map_p);
            prefetch_tensormap(&map_q);
            for (int i = 0; i < kStages; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, 1);
            }
            for (int i = 0; i < S::kAcc; ++i) {
                mbar_init(t_full + i, 1);
                mbar_init(t_empty + i, S::kEpi * (kPair ? 2 : 1));
            }
            for (int i = 0; i < kScaleSlots; ++i) {
                mbar_init(s_full + i, 32);
                mbar_init(s_empty + i, S::kEpi);
            }
            mbar_init(red_full, S::kEpi * split);
            *abort_flag = 0;
            issued[0] = issued[1] = peer[0] = peer[1] = peer[2] = 0;
            fence_barrier_init();
        }
        __syncwarp();
        named_arrive(1, S::kThreads);
    } else {
        if (warp == 3) {
            if constexpr (kPair) {
                tmem_alloc_pair(tmem_slot, S::kTmem);
            } else {
                tmem_alloc(tmem_slot, S::kTmem);
                tmem_relinquish();
            }
            tc_fence_before_sync();
        }
        named_sync(1, S::kThreads);
        tc_fence_after_sync();
    }
    if constexpr (kSplit) cluster_arrive_relaxed();
    if constexpr (kPair) {  // the other block's barriers stand, and its words are zero
        cluster_arrive();
        cluster_wait();
    }

    // tile -> (tile of the MMA rows' operand, tile of the columns'): kGroupRows rows at a time, the columns' outside
    auto place = [&](int tile, int &tp, int &tq) {
        constexpr int kGroup = kGroupRows / kRows;
        const int per = kGroup * a.q_tiles, g = tile / per, r = tile - g * per;
        const int rows = min(kGroup, a.p_tiles - g * kGroup);
        tq = r / rows;
        tp = g * kGroup + r - tq * rows;
    };

    if (warp < kFirst) {
        if constexpr (kPair) fewer_registers<kRegsLoad>();  // (one instruction for all four warps)
        if (warp == 0) {
            // ---- loads
            grid_dependency_wait();  // (what comes before needs nothing of the kernel before this one)
            grid_launch_dependents();
            int it = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tp, tq;
                place(tile, tp, tq);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % kStages;
                    if (it >= kStages) ok = __all_sync(0xffffffffu, bar_wait_inline(empty + s, (it / kStages - 1) & 1, abort_flag, a.err_word));
                    if (!ok) break;
                    uint8_t *p = smem + s * S::kStage;
                    if (elect_one()) {
                        if constexpr (kPair) {  // both blocks' bytes count on block 0's barrier
                            const uint32_t bar = of_rank(full + s, 0);
                            if (rank == 0) mbar_arrive_expect_tx(full + s, 2 * S::kStage);
                            tma_load_2d_pair(p, &map_p, kb * kMmBlk, tp * kRows + row0, bar);
                            tma_load_2d_pair(p + kMmRows * 128, &map_q, kb * kMmBlk, tq * kNT + rank * S::kLoad, bar);
                        } else {
                            mbar_arrive_expect_tx(full + s, S::kStage);
                            tma_load_2d(p, &map_p, kb * kMmBlk, tp * kRows, full + s);
                            tma_load_2d(p + kMmRows * 128, &map_q, kb * kMmBlk, tq * kNT, full + s);
                        }
                    }
                    __syncwarp();
                }
            }
            if constexpr (kPair) {  // used, in both blocks, and said so here: block 0's products do not end before both blocks' copies
#pragma unroll 1
                for (int i = it < kStages ? 0 : it - kStages; i < it && ok; ++i)
                    ok = __all_sync(0xffffffffu, bar_wait_inline(empty + i % kStages, (i / kStages) & 1, abort_flag, a.err_word));
                if (lane == 0) issued[0] = it;
            } else {
                phases_ended<kStages>(full, it);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---- products
            grid_dependency_wait();  // (so that the time limits of its waits do not count the kernel before)
            if (!kPair || rank == 0) {
                constexpr uint32_t idesc = idesc_e4m3_f32(kRows, kNT, false, false);
                const uint64_t desc0 = smem_desc(smem_u32(smem), 0, 1024, kSw128);
                const uint32_t d0 = __shfl_sync(0xffffffffu, *tmem_slot, 0);
                int it = 0;
                bool ok = true;
                for (int tile = first; tile < tiles && ok; tile += step) {
                    for (int kb = kb0; kb < kb1; ++kb, ++it) {
                        const int s = it % kStages, c = it % S::kAcc;
                        ok = bar_wait_inline(full + s, (it / kStages) & 1, abort_flag, a.err_word);
                        if (it >= S::kAcc && ok) ok = bar_wait_inline(t_empty + c, (it / S::kAcc - 1) & 1, abort_flag, a.err_word);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after_sync();
                        // (a descriptor's address counts 16 bytes; 32 bytes of K a step)
                        const uint64_t dp = desc0 + s * (S::kStage >> 4), dq = dp + (kMmRows * 128 >> 4);
                        const uint32_t d = d0 + (uint32_t)(c * kNT);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                if constexpr (kPair)
                                    mma_f8f6f4_pair(d, dp + 2 * kk, dq + 2 * kk, idesc, kk > 0);
                                else
                                    mma_f8f6f4(d, dp + 2 * kk, dq + 2 * kk, idesc, kk > 0);
                            }
                            if constexpr (kPair) {
                                mma_commit_pair(t_full + c);
                                mma_commit_pair(empty + s);
                            } else {
                                mma_commit(t_full + c);
                                mma_commit(empty + s);
                            }
                        }
                        __syncwarp();
                    }
                }
                phases_ended<kStages>(empty, it);
                phases_ended<S::kAcc>(t_full, it);
                if (kPair && lane == 0) issued[1] = it;
            }
            __syncwarp();
        } else if (warp == 2) {
            // ---- scales, kScaleBlocks K blocks at a time.  (Loaded by the warps that add, they held up each of their arrivals
            // until they were there: 8192 x 4096 x 16384 took 449 us so, 387 from here.)
            grid_dependency_wait();
            // a8's rows (kSwap: the tile's columns) and w8's blocks of 128; past the ends the last one's are repeated, for sums that are not written
            int g = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tp, tq;
                place(tile, tp, tq);
                const int m0 = kSwap ? tq * kNT : tp * kRows + row0, n0 = kSwap ? tp * kMmRows : tq * kNT;
                constexpr int kMs = kSwap ? kNT : kMmRows, kNs = kPair ? 2 : 1, kXs = (kMs + 31) / 32;
                float x[kScaleBlocks][kXs], w[kScaleBlocks];
                auto fetch = [&](int k) {
#pragma unroll
                    for (int u = 0; u < kScaleBlocks; ++u) {
                        const int kb = min(k + u, kb1 - 1);
                        w[u] = load_now(a.w_scale + (int64_t)tp * a.kb + kb);
#pragma unroll
                        for (int i = 0; i < kXs; ++i) x[u][i] = load_now(a.a_scale + kb * a.a_scale_stride + min(m0 + 32 * i + lane, a.M - 1));
                    }
                };
                for (int k = kb0; k < kb1; k += kScaleBlocks, ++g) {
                    const int s = g % kScaleSlots;
                    if constexpr (kSwap)
                        if (k == kb0) fetch(k);
                    if (g >= kScaleSlots) ok = __all_sync(0xffffffffu, bar_wait_inline(s_empty + s, (g / kScaleSlots - 1) & 1, abort_flag, a.err_word));
                    if (!ok) break;
                    if constexpr (kSwap) {  // the columns' factors are multiplied here, once; the next group's are on their way meanwhile
                        float y[kScaleBlocks][kXs];
#pragma unroll
                        for (int u = 0; u < kScaleBlocks; ++u)
#pragma unroll
                            for (int i = 0; i < kXs; ++i) y[u][i] = x[u][i] * w[u];
                        if (k + kScaleBlocks < kb1) fetch(k + kScaleBlocks);
#pragma unroll
                        for (int u = 0; u < kScaleBlocks; ++u)
#pragma unroll
                            for (int i = 0; i < kXs; ++i)
                                if (32 * i + lane < kMs) fac[(s * kScaleBlocks + u) * S::kScales + 32 * i + lane] = y[u][i];
                        mbar_arrive(s_full + s);
                    } else {
                        for (int u = 0; u < kScaleBlocks && k + u < kb1; ++u) {
                            float *to = fac + (s * kScaleBlocks + u) * S::kScales;
                            const float *from = a.a_scale + (k + u) * a.a_scale_stride;
#pragma unroll
                            for (int i = 0; i < kMs; i += 32)
                                if (i + lane < kMs) cp_async_4(to + i + lane, from + min(m0 + i + lane, a.M - 1));
                            if (lane < kNs) cp_async_4(to + kMs + lane, a.w_scale + (int64_t)min(n0 / kMmBlk + lane, (a.N - 1) / kMmBlk) * a.kb + k + u);
                        }
                        cp_async_mbar_arrive(s_full + s);
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");  // (none is in flight when the block ends)
            __syncwarp();
        }
    } else {
        // ---- sums
        if constexpr (kPair) more_registers<kRegsAdd>();
        grid_dependency_wait();  // (out may still be read by the kernel before)
        const int quad = warp & 3, half = (warp - kFirst) >> 2;  // (a warp reads TMEM lanes 32 (warp % 4) ..)
        const int row = quad * 32 + lane, col0 = half * S::kCols;
        const uint32_t tmem = *tmem_slot, lane_addr = (uint32_t)(quad * 32) << 16;
        Out *out = static_cast<Out *>(a.out);
        int it = 0, g = 0, parts = 0;  // K blocks, slots of scales, staging tiles
        bool ok = true;
        for (int tile = first; tile < tiles; tile += step) {
            int tp, tq;
            place(tile, tp, tq);
            uint64_t acc[S::kCols / 2];
#pragma unroll
            for (int i = 0; i < S::kCols / 2; ++i) acc[i] = 0;
            // adds n <= kBatch K blocks: acc += D * factor(block, pair of columns)
            auto add_blocks = [&](int n, auto factor) {
                const auto at = [&](int u) { return (it + u) % S::kAcc; };
                if (ok) {
#pragma unroll
                    for (int u = 0; u < S::kBatch; ++u)
                        if (u < n && ok) ok = bar_wait_inline(t_full + at(u), ((it + u) / S::kAcc) & 1, abort_flag, a.err_word);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after_sync();
#pragma unroll
                for (int j = 0; j < S::kCols; j += S::kChunk) {
                    uint32_t v[S::kBatch][S::kChunk / 16][16];
#pragma unroll
                    for (int u = 0; u < S::kBatch; ++u)
#pragma unroll
                        for (int i = 0; i < S::kChunk / 16; ++i)
                            if (u < n) tmem_ld_32x32b_x16(tmem + lane_addr + (uint32_t)(at(u) * kNT + col0 + j + 16 * i), v[u][i]);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < S::kBatch; ++u)
#pragma unroll
                        for (int i = 0; i < S::kChunk / 16; ++i) tmem_loaded(v[u][i]);
                    if (j + S::kChunk == S::kCols) {
                        tc_fence_before_sync();
                        if (lane == 0) {
#pragma unroll
                            for (int u = 0; u < S::kBatch; ++u) {
                                if (u < n) {
                                    if constexpr (kPair)
                                        mbar_arrive_cluster_relaxed(of_rank(t_empty + at(u), 0));
                                    else
                                        mbar_arrive(t_empty + at(u));
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < S::kBatch; ++u) {
                        if (u < n) {
#pragma unroll
                            for (int i = 0; i < S::kChunk / 2; ++i) {
                                const uint32_t x = v[u][i / 8][2 * (i % 8)], y = v[u][i / 8][2 * (i % 8) + 1];
                                uint64_t &sum = acc[j / 2 + i];
                                const uint64_t f = factor(u, j / 2 + i);
                                if constexpr (kSwap) {
                                    sum = f2_fma(f2_pack(__uint_as_float(x), __uint_as_float(y)), f, sum);
                                } else {  // (one factor: plain FMAs keep the tensor cores busier; 8192 x 4096 x 16384: 385 us packed, 364 plain)
                                    float lo, hi, f0, f1;
                                    f2_unpack(sum, lo, hi);
                                    f2_unpack(f, f0, f1);
                                    sum = f2_pack(fmaf(__uint_as_float(x), f0, lo), fmaf(__uint_as_float(y), f1, hi));
                                }
                            }
                        }
                    }
                }
                it += n;
            };
            for (int k = kb0; k < kb1; k += kScaleBlocks, ++g) {
                const int s = g % kScaleSlots;
                const float *sc = fac + s * kScaleBlocks * S::kScales;
                if (ok) ok = bar_wait_inline(s_full + s, (g / kScaleSlots) & 1, abort_flag, a.err_word);
                ok = __all_sync(0xffffffffu, ok);
                if constexpr (kSwap) {
#pragma unroll
                    for (int u = 0; u < kScaleBlocks; u += S::kBatch) {
                        if (k + u < kb1)
                            add_blocks(min(S::kBatch, kb1 - k - u), [&](int b, int i) {
                                const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sc + (u + b) * S::kScales + col0 + 4 * (i / 2));
                                return i % 2 ? f.y : f.x;
                            });
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty + s);
                } else {
                    float f[kScaleBlocks];
#pragma unroll
                    for (int u = 0; u < kScaleBlocks; ++u) f[u] = sc[u * S::kScales + row] * sc[u * S::kScales + kMmRows + col0 / kMmBlk];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty + s);
#pragma unroll
                    for (int u = 0; u < kScaleBlocks; ++u) {
                        if (k + u < kb1) {
                            const uint64_t ff = f2_pack(f[u], f[u]);
                            add_blocks(1, [&](int, int) { return ff; });
                        }
                    }
                }
            }
            if constexpr (kSplit) {
                // (rows of out that do not exist have no sums to hand over)
                __syncwarp();
                const int own = S::own(split);
                const int cols = kSwap ? min(kNT, a.M - tq * kNT) : min(kNT, a.N - tq * kNT);  // the tile's columns that exist
                if (kSwap && split == 1) {
                    const int n = tp * kMmRows + row, m = tq * kNT + col0;
#pragma unroll
                    for (int i = 0; i < S::kCols; ++i) {
                        float v[2];
                        f2_unpack(acc[i / 2], v[0], v[1]);
                        const float r[1] = {v[i & 1]};
                        if (ok && m + i < a.M && n < a.N) store<1>(out + (m + i) * a.out_stride + n, r);
                    }
                    cluster_wait();
                } else {
                    cluster_wait();  // every block's barriers stand
                    // sums of a tile lie as [rank][column / 4][row][4 columns] in the block that owns the columns
                    float4 *red = reinterpret_cast<float4 *>(staging);
                    if (ok) {
                        uint32_t to = 0;
#pragma unroll
                        for (int i = 0; i < S::kCols; i += 4) {
                            const int c = col0 + i;
                            if (i == 0 || c % own == 0) to = of_rank(red + (rank * own + c % own) / 4 * S::kRedRow + row, c / own);
                            float v[4];
                            f2_unpack(acc[i / 2], v[0], v[1]);
                            f2_unpack(acc[i / 2 + 1], v[2], v[3]);
                            if (c < cols) cluster_store(to, v[0], v[1], v[2], v[3]);
                            to += S::kRedRow * 16;
                        }
                        fence_cluster();
                        __syncwarp();
                        if (lane < split && lane * own < cols) mbar_arrive_cluster(of_rank(red_full, lane));
                    }
                    const int c0 = rank * own, mine = min(own, cols - c0);
                    if (mine > 0) {
                        ok = bar_wait_cluster(red_full, 0, abort_flag, a.err_word);
                        // four columns of a row a step; neighbours in a warp are neighbours in out: rows of the tile (kSwap), or its columns
                        const int quads = (mine + 3) / 4;
                        for (int i = tid - 32 * kFirst; ok && i < quads * kMmRows; i += 32 * S::kEpi) {
                            const int r = kSwap ? i % kMmRows : i / quads, c = 4 * (kSwap ? i / kMmRows : i - r * quads);
                            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int b = 0; b < 8; ++b) {
                                if (b < split) {
                                    const float4 x = red[(b * own + c) / 4 * S::kRedRow + r];
                                    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                                }
                            }
                            if constexpr (kSwap) {
                                const int m = tq * kNT + c0 + c, n = tp * kMmRows + r;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float one[1] = {v[j]};
                                    if (m + j < a.M && n < a.N) store<1>(out + (m + j) * a.out_stride + n, one);
                                }
                            } else {
                                const int m = tp * kMmRows + r, n = tq * kNT + c0 + c;
                                if (m < a.M) store_row(out + m * a.out_stride + n, v, a.N - n, a.tma_out);
                            }
                        }
                    }
                }
            } else if (!ok) {
            } else {
                // 32 rows x 128 bytes at a time through two swizzled staging tiles of the warp's own, in turn
                constexpr int kPart = kBf16 ? 64 : 32;
                const int m0 = tp * kRows + row0 + quad * 32;
#pragma unroll
                for (int c = 0; c < S::kCols; c += kPart) {
                    const int n0 = tq * kNT + col0 + c;
                    uint8_t *st = staging + ((warp - kFirst) * 2 + (parts++ & 1)) * 4096;
                    if (elect_one()) bulk_wait_read<1>();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint4 w;
                        if constexpr (kBf16) {
                            float v[8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) f2_unpack(acc[c / 2 + 4 * j + i], v[2 * i], v[2 * i + 1]);
                            w = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                        } else {
                            float v[4];
                            f2_unpack(acc[c / 2 + 2 * j], v[0], v[1]);
                            f2_unpack(acc[c / 2 + 2 * j + 1], v[2], v[3]);
                            w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                        }
                        *reinterpret_cast<uint4 *>(st + sw128_offset(lane, 16 * j)) = w;
                    }
                    if (a.tma_out) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (elect_one()) {
                            if (m0 < a.M && n0 < a.N) tma_store_2d(&map_out, st, n0, m0);
                            bulk_commit();  // (an empty group where nothing is stored: the count of groups goes by the parts)
                        }
                    } else {
                        __syncwarp();
                        for (int r = 0; r < 32 && m0 + r < a.M; ++r)
                            for (int e = lane; e < kPart && n0 + e < a.N; e += 32)
                                out[(int64_t)(m0 + r) * a.out_stride + n0 + e] =
                                    *reinterpret_cast<const Out *>(st + sw128_offset(r, e * (int)sizeof(Out)));
                        __syncwarp();
                    }
                }
            }
        }
        if constexpr (!kSplit && !kSwap) {
            if (elect_one()) bulk_wait();
            __syncwarp();
        }
    }
    if constexpr (kSplit) {
        __syncwarp();
        if (warp < kFirst) cluster_wait();
    }
    tc_fence_before_sync();
    __syncthreads();
    // no block leaves while another's products, sums or the arrivals of its threads may reach it
    if constexpr (kPair) {
        if (elect_one() && *(volatile int *)abort_flag) cluster_store(of_rank(peer, cluster_rank() ^ 1), 1);
        __syncwarp();
    }
    if constexpr (kPair || kSplit) {
        cluster_arrive();
        cluster_wait();
    }
    if constexpr (kPair) {
        if (*(volatile int *)abort_flag | *(volatile int *)peer) {  // (the same in all threads of both blocks)
            // all places anew: kept until here they would cost the warps of few registers some of theirs
            uint32_t base = smem_u32(smem_raw), thread = threadIdx.x;
            asm volatile("" : "+r"(base), "+r"(thread));
            uint8_t *again = smem_raw + ((1024u - (base & 1023u)) & 1023u);
            uint64_t *b = reinterpret_cast<uint64_t *>(again + (reinterpret_cast<uint8_t *>(bars) - smem));
            int *words = reinterpret_cast<int *>(again + (reinterpret_cast<uint8_t *>(issued) - smem));
            even_out<S, kStages>(map_p, map_q, again, b, b + kStages, b + 2 * kStages, words, words + 2, cluster_rank(), thread >> 5);
        }
    }
    if (warp == 3) {
        if constexpr (kPair)
            tmem_dealloc_pair(*tmem_slot, S::kTmem);
        else
            tmem_dealloc(*tmem_slot, S::kTmem);
    }
}

bool map_bytes(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *m, const uint8_t *p, int K, int64_t rows, int64_t stride, int box) {
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, es[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(p), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct MmCall {
    const uint8_t *a8, *w8;
    int64_t a_stride;
    int K;
    bool bf16;
    MmArgs a;
    cudaStream_t st;
};

template <bool kSwap, int kNT, int kStages, int kBlocks, bool kBf16, bool kSplit>
cudaError_t mm_launch(MmCall c, int blocks) {
    using S = MmShape<kSwap, kNT, kStages>;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    alignas(64) CUtensorMap map_a, map_w, map_out;
    const int w = kBf16 ? 2 : 4;
    if (!map_bytes(encode, &map_a, c.a8, c.K, c.a.M, c.a_stride, kSwap ? kNT : kMmRows) ||
        !map_bytes(encode, &map_w, c.w8, c.K, c.a.N, c.K, kSwap ? kMmRows : S::kLoad))
        return cudaErrorInvalidValue;
    map_out = map_a;  // (not read where out is not written by tensor stores)
    c.a.tma_out = reinterpret_cast<uintptr_t>(c.a.out) % 16 == 0 && c.a.out_stride * w % 16 == 0;
    if (!kSwap && !kSplit && c.a.tma_out) {
        const cuuint64_t dims[2] = {(cuuint64_t)c.a.N, (cuuint64_t)c.a.M}, strides[1] = {(cuuint64_t)c.a.out_stride * w};
        const cuuint32_t box[2] = {128u / w, 32}, es[2] = {1, 1};
        if (encode(&map_out, kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, c.a.out, dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    auto kernel = matmul8_kernel<kSwap, kNT, kStages, kBlocks, kBf16, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::bytes(kSplit));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::bytes(kSplit);
    cfg.stream = c.st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S::kPair ? 2u : (unsigned)c.a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kSplit || S::kPair ? 2 : 1;
    e = kSwap ? cudaLaunchKernelEx(&cfg, kernel, map_w, map_a, map_out, c.a) : cudaLaunchKernelEx(&cfg, kernel, map_a, map_w, map_out, c.a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <bool kSwap, int kNT, int kStages, int kBlocks, bool kSplit>
cudaError_t mm_typed(const MmCall &c, int blocks) {
    return c.bf16 ? mm_launch<kSwap, kNT, kStages, kBlocks, true, kSplit>(c, blocks)
                  : mm_launch<kSwap, kNT, kStages, kBlocks, false, kSplit>(c, blocks);
}

int tiles_of(int n, int t) { return (n + t - 1) / t; }

// The forms of the kernel, and what each takes: microseconds, fitted to 1100 of its times over M from 1 to 8192, N from 512 to
// 24576 and K from 512 to 16384 (each form within 5 % rms; the form of the least estimate took 0.6 % longer than the best one on
// average, 17 % at most).  A launch has a fixed part, its first round of tiles in it; a further round takes `round`, a K block
// `kb` (few rows: `shared` times that where two blocks share an SM), or `weight` for each block that streams weights beside it,
// whichever is more, rounded off between the two by a fourth-power mean.  A split adds its exchange.
// Both sides of the borders, in us: 64 x 24576 x 2048: tiles of 64 rows 14.4, of 32 19.2; 64 x 2048 x 2048: 7.1 and 5.7.
// 128 x 8192 x 8192: 128-wide tiles whole 25.6, in halves of K 20.4; 128 x 8192 x 2048: 8.2 and 9.5.
// 2048 x 8192 x 2048: pairs of 256 32.9, 128-wide 41.4; 128 x 24576 x 8192: 58.1 and 52.3.
enum MmForm { kFew16, kFew32, kFew64, kSplit128, kWhole128, kPair256, kForms };
struct MmTimes {
    double fixed, kb, round, shared, weight, split[4];  // split: by its log2
};
constexpr MmTimes kTimes[kForms] = {{3.07, 0.268, 2.55, 1.26, 0.0025, {0.0, 0.99, 1.11, 1.40}},
                                    {3.25, 0.287, 2.80, 1.34, 0.0026, {0.0, 1.18, 1.18, 1.58}},
                                    {4.20, 0.365, 4.31, 1.41, 0.0026, {0.0, 1.33, 1.46, 1.44}},
                                    {6.40, 0.308, 0.0, 1.0, 0.0031, {0.0, 0.0, 0.30, 0.80}},
                                    {3.07, 0.320, 0.56, 1.0, 0.0, {}},
                                    {4.19, 0.378, 1.62, 1.0, 0.0, {}}};

struct MmPlan {
    MmForm form;
    int p_tiles, q_tiles, split, blocks;
    double us;
};

MmPlan mm_plan(int M, int N, int kb, int sms) {
    MmPlan best{};
    best.us = 1e30;
    for (int f = 0; f < kForms; ++f) {
        MmPlan p{};
        p.form = (MmForm)f;
        const bool few = f <= kFew64;
        const int nt = f == kFew16 ? 16 : f == kFew32 ? 32 : 64;
        if (few && M > 16 * nt) continue;
        p.p_tiles = few ? tiles_of(N, kMmRows) : tiles_of(M, f == kPair256 ? 256 : kMmRows);
        p.q_tiles = few ? tiles_of(M, nt) : tiles_of(N, f == kPair256 ? 256 : 128);
        const int64_t tiles = (int64_t)p.p_tiles * p.q_tiles;
        const int slots = few ? 2 * sms : f == kPair256 ? sms / 2 : sms;  // tiles at a time
        for (int log = 0; log < (few || f == kSplit128 ? 4 : 1); ++log) {
            p.split = 1 << log;
            if (f == kSplit128 && log == 0) continue;
            // (clusters of 8 find room for 256 blocks of few rows; of the 128-wide ones 16 no longer fitted at once)
            if (log > 0 && (kb < 2 * p.split || tiles * p.split > (log < 3 ? slots : few ? 256 : 96))) break;
            if (tiles * p.split > 0x3fffffff) break;
            const int64_t at_once = tiles * p.split < slots ? tiles * p.split : slots, rounds = (tiles * p.split + slots - 1) / slots;
            const MmTimes &t = kTimes[f];
            const double own = t.kb * (tiles * p.split > sms ? t.shared : 1.0);
            const double stream = t.weight * (double)at_once / (few ? p.q_tiles : p.p_tiles);
            const double each = sqrt(sqrt(own * own * own * own + stream * stream * stream * stream));
            p.us = t.fixed + rounds * ((kb + p.split - 1) / p.split * each) + (rounds - 1) * t.round + t.split[log];
            if (p.us < best.us) {
                best = p;
                const int64_t launch = few || f == kSplit128 ? tiles * p.split : at_once;
                best.blocks = (int)(f == kPair256 ? 2 * launch : launch);
            }
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_matmul8(const uint8_t *a8, int64_t a_stride, const float *a_scale, int64_t a_scale_stride, int M, int N,
                           int K, const uint8_t *w8, const float *w_scale, void *out, int out_bf16, int64_t out_stride,
                           int *err_word, cudaStream_t st) {
    MmCall c{};
    c.a8 = a8, c.w8 = w8, c.a_stride = a_stride, c.K = K, c.bf16 = out_bf16 != 0, c.st = st;
    c.a.a_scale = a_scale, c.a.a_scale_stride = a_scale_stride, c.a.w_scale = w_scale;
    c.a.out = out, c.a.out_stride = out_stride, c.a.M = M, c.a.N = N, c.a.kb = tiles_of(K, kMmBlk), c.a.err_word = err_word;
    const MmPlan p = mm_plan(M, N, c.a.kb, device_sm_count());
    c.a.p_tiles = p.p_tiles, c.a.q_tiles = p.q_tiles, c.a.split = p.split;
    switch (p.form) {
        case kFew16: return mm_typed<true, 16, 5, 2, true>(c, p.blocks);
        case kFew32: return mm_typed<true, 32, 4, 2, true>(c, p.blocks);
        case kFew64: return mm_typed<true, 64, 3, 2, true>(c, p.blocks);
        case kSplit128: return mm_typed<false, 128, 4, 1, true>(c, p.blocks);
        case kWhole128: return mm_typed<false, 128, 4, 1, false>(c, p.blocks);
        default: return mm_typed<false, 256, 4, 1, false>(c, p.blocks);
    }
}

}  // namespace kv8
