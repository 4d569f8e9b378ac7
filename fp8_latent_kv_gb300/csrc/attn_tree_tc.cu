// attn_tree_tc.cu -- attention of drafted tokens over a paged latent cache on the tensor cores (tcgen05, sm_103a),
// for bf16 queries.
//
// All (token, head) columns of a sequence read the same rows, so a group of 64 columns against a tile of 64 rows is
// two contractions:
//   score    S[x][t]    = sum_k Qs[x][k] K8[t][k]      M = 128, N = 64 rows, K = 576 (e4m3 x e4m3)
//            Qs: a bf16 query element, scaled by its column's power of two, is the sum of two e4m3 values; each
//            TMEM lane quadrant holds 16 columns' hi pieces on lanes 0..15 and their lo pieces on lanes 16..31, so
//            that two 16-lane loads hand a thread both halves of its dot products.
//   context  O^T[d][n] += sum_t V8[t][d] W[n][t]       M = 128 dims (x4), N = 64 columns, K = 64 rows; V8 = the same
//            bytes read MN-major, W the softmax weights as the sum of two e4m3 values with a power of two for each
//            column and 32 rows (the block-scaled form of the MMA).
// Weights: with e_t = score_t log2(e) + log2(scale_t), X = floor(max e) over a block of 32 rows and R the column's
// reference, a weight is held as 2^(e_t - X + 7) < 256 and the block's power is 2^(X - R - 67).  So O and z are relative
// to 2^(R + 60) in 32-bit floats, each block's weights use all of e4m3's range whatever the others hold, and R, the
// exponent of the column's first tile, has to move (and O to be rescaled) only when a term exceeds it by 2^100, not
// whenever a larger one turns up: with one power for all rows, 64 columns' new maxima had every second tile of the
// first fifty wait for the context product before it and rescale.
// A tile of context rows alone, all there, with scales within 2^8 of one another, needs no masks and no logarithms: its
// blocks' powers are the largest scores' times the power of two above the scales, which costs a weight up to 8 of the
// binary orders below the block's largest (plain in the code; the others took 6.5 thousand cycles against 3.2).
// w_t holds the row scale already: O = sum w_t v_t, z = sum w_t / scale_t.  A row whose scale is below 2^-60 (zeros,
// subnormal maxima) has score 0 and adds nothing to O: such rows are only counted, and the count enters z at the end.
// A row whose scale is above 2^60 would have its term of z, 2^-60 / scale relative to its weight, fall out of 32 bits: its
// weight is NaN instead.
//
// Work: equal shares of (group, tile) units (tree.cuh), one CTA per SM.
// What bounds it: a tile's products take 1408 cycles (14 score MMAs with A in TMEM at 32, 4 from shared memory and 16 context MMAs at
// 48) of the 1570 that a tile takes where a share has hundreds of them.  An MMA with both operands in shared memory has 6 KB to read,
// 128 + 64 rows of 32 bytes, at 128 bytes a cycle; its 32 cycles of arithmetic are what the pipe's counter shows (69 %).
// The two teams' 3.9 thousand warp instructions a tile run beside that.  64 tokens of 128 heads over 32768 rows: 396 us, 1476
// TFLOP/s.  Three teams did not pay: of eight warps each they spilled (658 us against 522 then), of four they missed the
// instruction cache (557 against 497).
// Warps: 0 = row loads, 1 = scores and TMEM, 2 = the rows' scales, 3 = context products, 4..19 = softmax and output in
// two teams that take alternate tiles.  warp % 4 is a warp's TMEM lane quadrant, its set (0, 1) the block of 32 rows,
// and a thread holds 8 rows of two columns.
// The query pieces are the score's A operand in TMEM (448 latent bytes) and shared memory (the rest).  Shared memory:
// five stages of 64 rows (36 KB each), two weight buffers of 8 KB, the query's part 16 KB.
// TMEM: query 112 columns, scale factors 12, two score buffers of 64, context accumulators 4 x 64.
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
// A segment's start and end cost as much as eight tiles, its draft's tile included.  Ragged sequences are where it shows: 16
// sequences of 64 tokens took 1799 us with 4, 1646 with 6, 1573 with 8, 1582 with 12, 1597 with 16; 32 of 13 tokens and 16
// heads 80.5, 78.8, 79.6, 82.1, 84.4.
constexpr int kSegment = 8;
// A share is at least two tiles where there is less work than shares: the teams take one each at the same time, and
// half as many partial sets are written and joined (one token over 4096 rows: 22.0 us with one tile, 19.6 with two, 20.1
// with four).
constexpr int kLeast = 2;
constexpr int kTeams = 2;                  // softmax teams of 256 threads
constexpr int kTeam = 256;
constexpr int kSoftmax = kTeams * kTeam;
constexpr int kThreads = 128 + kSoftmax;
constexpr uint32_t kBlk = 8192;            // 64 rows x 128 latent bytes (SW128)
constexpr uint32_t kRope = 4096;           // 64 rows x 64 RoPE bytes (SW64)
constexpr uint32_t kStage = 4 * kBlk + kRope;
constexpr uint32_t kQLat = 28 * 128 * 16;  // a group's query image: 28 chunks of 16 latent bytes of 128 lanes,
constexpr uint32_t kQTail = 128 * 128;     // then 128 x (64 latent + 64 RoPE bytes) (SW128)
constexpr uint32_t kImg = kQLat + kQTail;
constexpr uint32_t kW = 8192;              // hi [64 columns][64 rows] (SW64), then lo
constexpr uint32_t OFF_ST = 0, OFF_W = kStages * kStage, OFF_Q = OFF_W + kTeams * kW, OFF_MISC = OFF_Q + kQTail;
constexpr float kRoom = 100.0f;            // the reference moves when a block's exponent exceeds it by more
// A reference is the sum of a score, a scale's logarithm and small whole numbers: from 2^24 on it would round those away, and the
// weights would no longer fit their pieces.  A column whose reference goes beyond 2^23 is NaN.
constexpr float kFar = 8388608.f;
constexpr int kBase = 60;                  // O and z are relative to 2^(reference + kBase)
constexpr float kTiny = 8.6736174e-19f;    // 2^-60
constexpr uint32_t TM_Q = 0, TM_SFA = 112, TM_SFB = 116, TM_S = 128, TM_O = 256;

struct RowInfo {
    alignas(16) float scale[kRows];        // 0 for rows that are not there
    uint64_t in, zero;                     // rows that are there / whose scale is below 2^-60
    float norm[2];                         // 2^-K of each block of 32 rows, K = ceil(log2 of its largest scale) ...
    uint32_t even;                         // ... where all are there and within 2^8 of one another; else 0
};
struct Misc {
    RowInfo rows[kStages];
    alignas(16) float ref[kCols];          // the columns' references R (whole numbers), -inf before any attended row
    alignas(16) float zinv[kCols];         // at the end: 1 / z
    union {
        float top[kTeams][2][kCols];       // X of a team's two blocks
        float red[2 * kTeams][kCols];      // at the end: sums
    };
    TreeWalk walk;                         // the softmax's: one thread's, kept out of the others' registers
    TreeSegment seg[3];                    // this segment and the next two
    int more[3];
    uint64_t kv_full[kStages], kv_free[kStages], row_full[kStages], s_free[2], s_full[kTeams], w_full[kTeams], pv_done[kTeams],
        q_ready, final_bar[2];
    uint32_t tmem_base;
    int abort_flag;
};
constexpr uint32_t kSmemBytes = OFF_MISC + sizeof(Misc);
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(offsetof(Misc, kv_full) % 8 == 0 && OFF_MISC % 1024 == 0 && OFF_W % 1024 == 0 && kStage % 1024 == 0, "alignment");

struct TcArgs {
    TreeArgs t;
    const uint8_t *img;    // query images, one kImg for each group
    const float *c_head;   // [images][64]: |sm_scale| * log2(e) * 2^-e of the column's query
};

// A sequence's groups' images begin at slot q0 * H / 64 + b: never past the next sequence's first.
__host__ __device__ __forceinline__ int64_t tree_slot(int64_t q0, int H, int b) { return q0 * H / kCols + b; }

// Arrive at a named barrier that other threads wait at.
__device__ __forceinline__ void named_arrive(int id, int count) {
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

// Block-scaled MMA (e4m3 x e4m3, 32 elements of K): each row of A and of B times a power of two, an exponent byte per
// row that the instruction descriptor's ids pick from the 32-bit words at `sfa` / `sfb` in TMEM (row r: lane r % 32 of
// every quadrant, column r / 32).
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// Its instruction descriptor: e4m3 A (MN-major) and B (K-major), scale bytes are exponents.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N, int sfb_id) {
    return ((uint32_t)sfb_id << 4) | (1u << 15) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_st_32x32b_x2(uint32_t taddr, uint32_t a, uint32_t b) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
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
// Two softmax weights (at most 2^8) -> e4m3 pieces and e4m3 pieces of what those leave.  By way of f16, whose 11 bits
// are finer than the 8 that the pieces keep; the residual is exact there.
__device__ __forceinline__ uint32_t split_weights(uint64_t w) {  // hi pieces in the low half, lo pieces in the high half
    uint32_t w16, h16, r16;
    uint16_t hi, lo;
    float a, b;
    f2_unpack(w, a, b);
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w16) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(w16));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h16) : "h"(hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r16) : "r"(w16), "r"(h16));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r16));
    return (uint32_t)hi | (uint32_t)lo << 16;
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// log2 of a power of two
__device__ __forceinline__ float log2_whole(float p) { return (float)((int)(__float_as_uint(p) >> 23) - 127); }
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// ------------------------------------------------------------------------------------------------------------
// Query images, column factors, and (block 0) the work shares.  A block splits 16 columns of a group, two by each warp:
// their pieces are 32 consecutive lanes of the image, so that by way of shared memory whole lines are written.
// ------------------------------------------------------------------------------------------------------------
constexpr int kPrepCols = 16, kPrepWarps = 8, kPrepThreads = 32 * kPrepWarps;
constexpr int kPieceStride = 33;  // 16-byte units of a chunk's 32 lanes, and one against bank conflicts

// 16 bf16 elements times 2^sh -> 16 bytes of hi pieces and of lo pieces
__device__ __forceinline__ void split_chunk(const uint4 (&u)[2], float f0, float f1, uint4 &hi, uint4 &lo) {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    uint32_t h[4] = {0u, 0u, 0u, 0u}, l[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = __uint_as_float(w[e] << 16) * f0 * f1, y = __uint_as_float(w[e] & 0xFFFF0000u) * f0 * f1;
        uint32_t ph, pl;
        split_pair(x, y, ph, pl);
        h[e >> 1] |= ph << ((e & 1) * 16);
        l[e >> 1] |= pl << ((e & 1) * 16);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// The largest magnitude of 16 bf16 elements, as its bits (NaN above infinity above numbers).
__device__ __forceinline__ uint32_t chunk_max(const uint4 (&u)[2]) {
    uint32_t m = 0;
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
    return max(m >> 16, m & 0xFFFFu);
}

// (Six blocks an SM: 48 warps' loads in flight, for which the compiler has 40 registers and spills 28 bytes of the shares' code.
// Four, as many as the shares' block would leave: 546 us against 537 for 16 x 64 tokens over 2048 rows.)
__global__ void __launch_bounds__(kPrepThreads, 6) tree_prep_kernel(TreeArgs a, uint8_t *img, float *c_head) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ union {
        TreeScan scan;
        struct {
            uint4 piece[28 * kPieceStride];  // 28 latent chunks of 32 lanes
            uint4 tail[32 * 8];              // the lanes' 128 bytes, swizzled
        };
    } sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0) {
        tree_schedule<kCols, kRows, kSegment, kLeast>(a, sm.scan);
        return;
    }
    const int64_t slot = (blockIdx.x - 1) / (kCols / kPrepCols);
    const int quarter = (blockIdx.x - 1) % (kCols / kPrepCols);
    // the slot's sequence: the last one with rows whose images begin at or before it (an impossible one's start says nothing)
    __shared__ int last;
    __shared__ TreeSeq found;
    if (tid == 0) last = -1;
    __syncthreads();
    int mine_b = -1;
    TreeSeq q{};
    for (int k = tid; k < a.B; k += kPrepThreads) {
        const TreeSeq t = tree_seq(a.q_start, a.lens, k, a.R, tree_positions(a.max_pages, a.page_shift));
        if (t.n <= 0 || tree_slot(t.q0, a.H, k) > slot) continue;
        mine_b = k;
        q = t;
    }
    int b = __reduce_max_sync(0xffffffffu, mine_b);
    if (lane == 0 && b >= 0) atomicMax(&last, b);
    __syncthreads();
    b = last;
    if (b < 0) return;
    if (mine_b == b) found = q;
    __syncthreads();
    q = found;
    const int64_t col0 = (slot - tree_slot(q.q0, a.H, b)) * kCols + quarter * kPrepCols, cols = (int64_t)q.n * a.H;
    // (a group's columns that the sequence does not have are zeros)
    if (col0 - quarter * kPrepCols >= cols) return;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // a warp's two columns: 32 chunks of latent elements by lane, four of RoPE elements by lanes 0..3 and 4..7
    uint4 u[3][2];
    const int64_t at = (int64_t)q.q0 * a.H + col0 + 2 * warp;
    const bool mine[2] = {col0 + 2 * warp < cols, col0 + 2 * warp + 1 < cols};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint4 *src = static_cast<const uint4 *>(a.q_lat) + (at + k) * (kKL / 8) + 2 * lane;
        u[k][0] = mine[k] ? __ldg(src) : zero;
        u[k][1] = mine[k] ? __ldg(src + 1) : zero;
    }
    const int rope = lane >> 2;
    const bool has = rope < 2 && mine[rope & 1];
    {
        const uint4 *src = static_cast<const uint4 *>(a.q_rope) + (at + (rope & 1)) * (kKR / 8) + 2 * (lane & 3);
        u[2][0] = has ? __ldg(src) : zero;
        u[2][1] = has ? __ldg(src + 1) : zero;
    }
    const uint32_t m_rope = chunk_max(u[2]);
    float f0[2], f1[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t bits = __reduce_max_sync(0xffffffffu, max(chunk_max(u[k]), rope == k ? m_rope : 0u));
        // max |q| = f 2^E, f in [1/2, 1), of a bf16's bits
        const int E = bits >= 0x80u ? (int)(bits >> 7) - 126 : 32 - __clz(bits) - 133;
        const int sh = bits != 0u && bits < 0x7F80u ? 8 - E : 0;  // max |q| 2^sh in [128, 256)
        const int half = min(sh, 127);                            // (sh from -120 to 140)
        const float sign = a.sm_scale_log2 < 0.f ? -1.f : 1.f;    // the column's factor is not negative
        // a query with a NaN or an infinity: every piece is NaN
        f0[k] = bits < 0x7F80u ? sign * __int_as_float((127 + half) << 23) : NAN;
        f1[k] = __int_as_float((127 + sh - half) << 23);
        const int n = quarter * kPrepCols + 2 * warp + k;
        if (lane == 0) c_head[slot * kCols + n] = mine[k] ? ldexpf(fabsf(a.sm_scale_log2), -sh) : 0.f;
    }
    const int l0 = 2 * warp;  // the columns' hi lanes are l0 and l0 + 1, their lo lanes 16 on
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint4 hi, lo;
        const bool second = k == 1 || (k == 2 && rope == 1);
        split_chunk(u[k], second ? f0[1] : f0[0], second ? f1[1] : f1[0], hi, lo);
        const int l = l0 + (second ? 1 : 0), ch = k < 2 ? lane : 32 + (lane & 3);
        if (ch < 28) {
            sm.piece[ch * kPieceStride + l] = hi;
            sm.piece[ch * kPieceStride + l + 16] = lo;
        } else if (k < 2 || rope < 2) {
            sm.tail[sw128_offset(l, (ch - 28) * 16) / 16] = hi;
            sm.tail[sw128_offset(l + 16, (ch - 28) * 16) / 16] = lo;
        }
    }
    __syncthreads();
    uint8_t *dst = img + slot * kImg;
    for (int i = tid; i < 28 * 32; i += kPrepThreads)
        *reinterpret_cast<uint4 *>(dst + ((i >> 5) * 128 + quarter * 32 + (i & 31)) * 16) = sm.piece[(i >> 5) * kPieceStride + (i & 31)];
    *reinterpret_cast<uint4 *>(dst + kQLat + quarter * 32 * 128 + tid * 16) = sm.tail[tid];
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
        mbar_init(&ms.s_free[0], kTeam / 32);  // one arrival for each warp
        mbar_init(&ms.s_free[1], kTeam / 32);
        for (int k = 0; k < kTeams; ++k) {
            mbar_init(&ms.s_full[k], 1);  // (a team's own: a waiter that skipped phases could take one for another)
            mbar_init(&ms.w_full[k], kTeam / 32);
            mbar_init(&ms.pv_done[k], 1);
        }
        mbar_init(&ms.q_ready, kTeam / 32);
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
                bar_wait(&ms.kv_full[i % kStages], (i / kStages) & 1, nullptr, a.err_word, kWaitCycles / 8);
        __syncwarp();
    } else if (warp == 1) {
        // ================================ scores ================================
        // The whole warp runs the loop and one elected lane issues: operands stay in uniform registers.  (Issued from
        // `if (lane == 0)` the same MMAs took 46 cycles each instead of 32 alone, and 85 beside the softmax warps.)
        // Scores and context products have a warp each: the tensor core's queue takes a few MMAs only, so the hundreds
        // of cycles that an issuer spends on its waits are the core's idle time unless another one issues meanwhile.
        const uint32_t id_s = idesc_e4m3_f32(128, kRows, false, false);
        // descriptors of stage 0 and of the query's part in shared memory: an offset adds to the address field
        const uint64_t k_desc = smem_desc(sbase + OFF_ST, 0, 1024, kSw128);
        const uint64_t kr_desc = smem_desc(sbase + OFF_ST + 4 * kBlk, 0, 512, kSw64);
        const uint64_t q_desc = smem_desc(sbase + OFF_Q, 0, 1024, kSw128);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = bar_wait(bar, parity, &ms.abort_flag, a.err_word);
            ok = __all_sync(0xffffffffu, ok);
        };
        int j = 0, sg = 0, s = 0, w3 = 0;  // tiles, segments, the stage, the team
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
                    for (int kk = 0; kk < 14; ++kk)
                        mma_f8f6f4_ts(d, tmem + TM_Q + kk * 8, k + (uint64_t)(((kk >> 2) * kBlk + (kk & 3) * 32) >> 4), id_s, kk != 0);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_f8f6f4(d, q_desc + (uint64_t)(kk * 2), kk < 2 ? k + (uint64_t)((3 * kBlk + 64 + kk * 32) >> 4) : kr + (uint64_t)((kk - 2) * 2),
                                   id_s, 1u);
                    mma_commit(&ms.s_full[w3]);
                }
                __syncwarp();
                w3 = w3 + 1 == kTeams ? 0 : w3 + 1;
                if (++s == kStages) {
                    s = 0;
                    s_ph ^= 1;
                }
            }
        }
        if (elect_one()) mma_commit(&ms.final_bar[0]);  // all issued MMAs complete before the CTA tears down
        __syncwarp();
        bar_wait(&ms.final_bar[0], 0, nullptr, a.err_word, kWaitCycles / 8);
        __syncwarp();
    } else if (warp == 3) {
        // ================================ context products ================================
        const uint64_t v_desc = smem_desc(sbase + OFF_ST, 0, 1024, kSw128);  // (the score's bytes, MN-major)
        const uint64_t w_desc = smem_desc(sbase + OFF_W, 0, 512, kSw64);
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok) ok = bar_wait(bar, parity, &ms.abort_flag, a.err_word);
            ok = __all_sync(0xffffffffu, ok);
        };
        int i = 0, s = 0, w3 = 0;  // tiles, the stage, the team
        uint32_t s_ph = 0, w_ph = 0;
        while (ok && walk.next<kCols, kRows>(a, seg)) {
            for (int t = seg.t0; ok && t < seg.t1; ++t, ++i) {
                wait(&ms.kv_full[s], s_ph);  // (complete since before the score)
                wait(&ms.w_full[w3], w_ph);
                tc_fence_after_sync();
                if (ok && elect_one()) {
                    const uint64_t v = v_desc + (uint64_t)(s * (kStage >> 4));
                    const uint64_t w = w_desc + (uint64_t)(w3 * (kW >> 4));
                    const uint32_t keep = t > seg.t0;
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            const uint64_t av = v + (uint64_t)((ch * kBlk + kk * 4096) >> 4);
                            const uint32_t sfb = tmem + TM_SFB + 4u * w3;
                            mma_mxf8(tmem + TM_O + 64u * ch, av, w + (uint64_t)((kk * 32) >> 4), idesc_mxf8(128, kCols, kk), tmem + TM_SFA,
                                     sfb, kk ? 1u : keep);
                            mma_mxf8(tmem + TM_O + 64u * ch, av, w + (uint64_t)((kW / 2 + kk * 32) >> 4), idesc_mxf8(128, kCols, kk),
                                     tmem + TM_SFA, sfb, 1u);
                        }
                    mma_commit(&ms.kv_free[s]);
                    mma_commit(&ms.pv_done[w3]);
                }
                __syncwarp();
                if (++w3 == kTeams) {
                    w3 = 0;
                    w_ph ^= 1;
                }
                if (++s == kStages) {
                    s = 0;
                    s_ph ^= 1;
                }
            }
        }
        if (elect_one()) mma_commit(&ms.final_bar[1]);
        __syncwarp();
        bar_wait(&ms.final_bar[1], 0, nullptr, a.err_word, kWaitCycles / 8);
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
                    float norm[2];
                    bool even = true;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float c = sc[2 * v + k];
                        const bool there = row[2 * v + k] >= 0;
                        in[k] = __ballot_sync(0xffffffffu, there);
                        zero[k] = __ballot_sync(0xffffffffu, there && c < kTiny);
                        ri.scale[32 * k + lane] = c;
                        const float lo = -warp_redux_max(-c), hi = warp_redux_max(c);
                        even = even && lo >= kTiny && hi <= 1.f / kTiny && hi <= 256.f * lo && in[k] == 0xffffffffu;
                        // (scales are compared, so a NaN is not even)
                        if (!__all_sync(0xffffffffu, c == c)) even = false;
                        int K;
                        frexpf(hi, &K);  // hi <= 2^K
                        norm[k] = even ? ldexpf(1.f, -K) : 0.f;
                    }
                    if (lane == 0) {
                        ri.in = in[0] | (uint64_t)in[1] << 32;
                        ri.zero = zero[0] | (uint64_t)zero[1] << 32;
                        ri.norm[0] = norm[0];
                        ri.norm[1] = norm[1];
                        ri.even = even;
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
        // After a wait that gave up (`ok` false) a thread skips its remaining waits but still reaches every named
        // barrier, so that no other warp waits for it.
        const int st = tid - 128;                     // 0..511
        const int q = warp & 3, w16 = (warp - 4) >> 2;
        const int team = w16 >> 1, set = w16 & 1;     // alternate tiles; rows 32 set .. 32 set + 31 of them
        // A 16-lane TMEM load of 8 columns hands lane l rows 2 (l % 4) and 2 (l % 4) + 1 of columns l / 4 and l / 4 + 8: the
        // hi and lo pieces' loads match register by register.  So a thread holds, for two columns, rows 8 i + 2 (l % 4)
        // and the next, i < 4, of its set's 32.
        const int n_a = 16 * q + (lane >> 2), n_b = n_a + 8;
        const int r0 = 32 * set + 2 * (lane & 3);     // its first row
        const uint32_t lane_addr = (uint32_t)(q * 32) << 16;
        const uint32_t s_addr = tmem + lane_addr + TM_S + 32u * set;
        const uint32_t o_addr = tmem + lane_addr + TM_O;
        // named barriers: 1 = all teams, 2 + team its own, 5 + team: it has decided, the next team waits
        const int team_bar = 2 + team, before = team == 0 ? kTeams - 1 : team - 1;
        // where its weights go: lane pairs exchange, so that an even lane stores rows 8 i + 4 (l % 4 / 2) .. + 3 of its set's
        // even i, an odd lane of its odd i; column b's are 512 bytes on
        const uint32_t w_row = 32 * set + 8 * (lane & 1) + 4 * ((lane & 3) >> 1);
        const uint32_t w_base = sbase + OFF_W + team * kW;
        const uint32_t w_addr[2] = {w_base + sw64_offset(n_a, w_row), w_base + sw64_offset(n_a, w_row + 16)};
        const uint32_t lo_first = lane & 1 ? 0x1054u : 0x5410u, hi_first = lane & 1 ? 0x3276u : 0x7632u;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok &= bar_wait(bar, parity, &ms.abort_flag, a.err_word);
        };
        grid_launch_dependents();
        // a group's queries: a quarter of the lane's 448 latent bytes to TMEM (the last: 64 bytes)
        auto image = [&](const TreeSegment &g) { return x.img + (tree_slot(g.q.q0, a.H, g.b) + g.g) * kImg; };
        auto load_queries = [&](const TreeSegment &g, int quarter) {
            uint4 query[8];
            const uint4 *src = reinterpret_cast<const uint4 *>(image(g)) + quarter * 8 * 128 + 32 * q + lane;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < 4 || quarter < 3) query[k] = __ldg(src + k * 128);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 *v = query + 4 * k;
                const uint32_t w[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                                        v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
                if (k == 0 || quarter < 3) tmem_st_32x32b_x16(tmem + lane_addr + TM_Q + quarter * 32 + 16 * k, w);
            }
        };
        // and by each warp of one team, after the barriers that order the quarters: the part in shared memory, by a copy
        auto queries_ready = [&](const TreeSegment &g) {
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if ((st & (kTeam - 1)) == 0) {
                mbar_arrive_expect_tx(&ms.q_ready, kQTail);
                bulk_load(smem + OFF_Q, image(g) + kQLat, kQTail, &ms.q_ready);
            } else if (lane == 0) {
                mbar_arrive(&ms.q_ready);
            }
        };
        // the value rows' factors are all 1
        if (w16 == 0) {
            tmem_st_32x32b_x2(tmem + lane_addr + TM_SFA, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            tmem_st_32x32b_x2(tmem + lane_addr + TM_SFA + 2, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            tmem_wait_st();
        }
        // One thread walks the share, two segments ahead of the others.
        if (st == 0) {
            ms.walk = walk;
            ms.more[0] = ms.walk.next<kCols, kRows>(a, ms.seg[0]);
            ms.more[1] = ms.walk.next<kCols, kRows>(a, ms.seg[1]);
        }
        if (st < kCols) ms.ref[st] = -INFINITY;
        named_sync(1, kSoftmax);
        if (ms.more[0]) {
            load_queries(ms.seg[0], w16);
            tmem_wait_st();
            tc_fence_before_sync();
            named_sync(1, kSoftmax);
            if (team == 0) queries_ready(ms.seg[0]);
        }
        int first_tile = 0;                    // tiles before the segment, modulo kTeams
        uint32_t own = 0;                      // the team's tiles so far
        int it = team, s_now = team;           // the team's next tile, and its stage
        uint32_t s_ph = 0;
        int end_tile = 0;                      // tiles up to the segment's end
        int segments = 0;
        for (int now = 0; ms.more[now]; ++segments) {
            const TreeSegment &sg = ms.seg[now];
            const int next = now == 2 ? 0 : now + 1, third = 3 - now - next;
            if (st == 0) ms.more[third] = ms.walk.next<kCols, kRows>(a, ms.seg[third]);
            first_tile = end_tile;
            end_tile += sg.t1 - sg.t0;
            const int plain_end = first_tile + (int)min(sg.q.len / kRows - sg.t0, (int64_t)(end_tile - first_tile));  // tiles of context only
            float c_a, c_b;
            {
                const float *c = x.c_head + (tree_slot(sg.q.q0, a.H, sg.b) + sg.g) * kCols;
                c_a = __ldg(c + n_a);
                c_b = __ldg(c + n_b);
            }
            float ref_a = -INFINITY, ref_b = -INFINITY;         // the references that z is relative to: the team's last
            uint64_t z_a = f2_pack(0.f, 0.f), z_b = f2_pack(0.f, 0.f);
            int zero_a = 0, zero_b = 0;                         // zero rows that the columns attend among this thread's
            for (; it < end_tile; it += kTeams, ++own) {
                const uint32_t own_ph = own & 1u;
                // ---- scores
                wait(&ms.s_full[team], own_ph);
                tc_fence_after_sync();
                uint32_t hi[16], lo[16];
                tmem_ld_16x256b_x4(s_addr + 64u * (it & 1), hi);
                tmem_ld_16x256b_x4(s_addr + 64u * (it & 1) + (16u << 16), lo);
                wait(&ms.row_full[s_now], s_ph);
                const RowInfo &ri = ms.rows[s_now];
                // every column attends every row, and the rows' scales are near one another
                const bool plain = it < plain_end && ri.even;
                tmem_wait_ld();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.s_free[it & 1]);
                // ---- dot products, row pairs packed: 0..3 of column a, 4..7 of column b
                uint64_t d2[8], sc2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 sc = *reinterpret_cast<const float2 *>(&ri.scale[r0 + 8 * i]);
                    sc2[i] = f2_pack(sc.x, sc.y);
                    d2[i] = f2_add(f2_pack(__uint_as_float(hi[4 * i]), __uint_as_float(hi[4 * i + 1])),
                                   f2_pack(__uint_as_float(lo[4 * i]), __uint_as_float(lo[4 * i + 1])));
                    d2[4 + i] = f2_add(f2_pack(__uint_as_float(hi[4 * i + 2]), __uint_as_float(hi[4 * i + 3])),
                                       f2_pack(__uint_as_float(lo[4 * i + 2]), __uint_as_float(lo[4 * i + 3])));
                }
                // ---- X of the block, over the column's four lanes: in a plain tile floor(max score) + K, else floor(max e)
                // (c is not negative, so that the largest d2 makes the largest score)
                float max_a = -INFINITY, max_b = -INFINITY, K, nm, ca = 1.f, cb = 1.f;  // scores: ca d2, cb d2 (log2 units)
                if (plain) {
                    nm = ri.norm[set];
                    K = -log2_whole(nm);
                    ca = c_a;
                    cb = c_b;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float e0, e1;
                        d2[i] = f2_mul(d2[i], sc2[i]);
                        d2[4 + i] = f2_mul(d2[4 + i], sc2[i]);
                        f2_unpack(d2[i], e0, e1);
                        max_a = fmaxf(max_a, fmaxf(e0, e1));
                        f2_unpack(d2[4 + i], e0, e1);
                        max_b = fmaxf(max_b, fmaxf(e0, e1));
                    }
                } else {
                    // the rows that the columns attend: those that are there, of the draft those of their masks
                    nm = 1.f;
                    K = 0.f;
                    const uint32_t in = (uint32_t)(ri.in >> r0), zr = (uint32_t)(ri.zero >> r0);
                    const int64_t j0 = (int64_t)(sg.t0 + it - first_tile) * kRows - sg.q.len;  // the tile's first row's index in the draft
                    const int c0 = sg.g * kCols, top = sg.q.n * a.H;
                    uint32_t on[2];  // bits 8 i and 8 i + 1 of each column
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        on[h] = in & (uint32_t)(tree_attended(a, sg.q.q0, min(c0 + (h ? n_b : n_a), top - 1) / a.H, j0) >> r0);
                        (h ? zero_b : zero_a) += __popc(on[h] & zr & 0x03030303u);
                        on[h] &= ~zr;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float s[2], e[2][2];
                        f2_unpack(sc2[i], s[0], s[1]);
                        f2_unpack(f2_mul(d2[i], f2_mul(sc2[i], f2_pack(c_a, c_a))), e[0][0], e[0][1]);
                        f2_unpack(f2_mul(d2[4 + i], f2_mul(sc2[i], f2_pack(c_b, c_b))), e[1][0], e[1][1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // a scale that is not a number, or so large that its term would be lost from z, must not meet the
                            // weight 0 of a column that leaves the row out, and makes that of a column that does not NaN
                            const bool fine = s[k] <= 1.f / kTiny;
                            const float lg = lg2_approx(s[k]);
                            s[k] = fine ? s[k] : 1.f;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const bool sees = on[h] >> (8 * i + k) & 1;
                                e[h][k] = !sees ? -INFINITY : fine ? e[h][k] : NAN;
                                (h ? max_b : max_a) = fmaxf(h ? max_b : max_a, sees ? e[h][k] + lg : -INFINITY);
                            }
                        }
                        sc2[i] = f2_pack(s[0], s[1]);
                        d2[i] = f2_pack(e[0][0], e[0][1]);
                        d2[4 + i] = f2_pack(e[1][0], e[1][1]);
                    }
                }
                max_a = fmaxf(max_a, __shfl_xor_sync(0xffffffffu, max_a, 1));
                max_b = fmaxf(max_b, __shfl_xor_sync(0xffffffffu, max_b, 1));
                max_a = floorf(ca * fmaxf(max_a, __shfl_xor_sync(0xffffffffu, max_a, 2))) + K;
                max_b = floorf(cb * fmaxf(max_b, __shfl_xor_sync(0xffffffffu, max_b, 2))) + K;
                // the context product of the team's tile before has read its weight buffer and factors (and the exponents
                // that they were made from)
                wait(&ms.pv_done[team], own_ph ^ 1u);  // (passes at once before the first)
                float(*const tops)[kCols] = ms.top[team];
                if ((lane & 3) == 0) {
                    tops[set][n_a] = max_a;
                    tops[set][n_b] = max_b;
                }
                // ---- the references, tile after tile: the other team has decided on the tile before.  (The barrier also
                // hands the blocks' exponents to the warps that write the scale factors.)
                if (it > first_tile) named_sync(5 + before, 2 * kTeam);
                float na = ms.ref[n_a], nb = ms.ref[n_b];
                const bool slow = bar_red_or(team_bar, kTeam, max_a > na + kRoom || max_b > nb + kRoom);
                auto moved = [&](int n, float r) -> float {  // a column's reference r from this tile on
                    const float x = fmaxf(tops[0][n], tops[1][n]);
                    return slow && x > r + kRoom ? (fabsf(x) <= kFar ? x : NAN) : r;
                };
                float move = 1.f;          // the factor of the accumulator column 32 set + lane
                float rl = ms.ref[lane], rh = ms.ref[32 + lane];  // of the columns whose factors this lane may write
                if (slow) {
                    rl = moved(lane, rl);
                    rh = moved(32 + lane, rh);
                    na = moved(n_a, na);
                    nb = moved(n_b, nb);
                    const float r = ms.ref[32 * set + lane], rn = moved(32 * set + lane, r);
                    move = r == -INFINITY || rn == r ? 1.f : ex2_approx(r - rn);
                    named_sync(team_bar, kTeam);
                    if (q == 0) ms.ref[32 * set + lane] = rn;  // (all have read the old ones)
                    __threadfence_block();                     // before the other team, which arrives below, reads them
                }
                if (it + 1 < end_tile) named_arrive(5 + team, 2 * kTeam);
                if (ref_a != na || ref_b != nb) {  // z, relative to the team's last references, to these
                    const float fa = ref_a == -INFINITY || ref_a == na ? 1.f : ex2_approx(ref_a - na);
                    const float fb = ref_b == -INFINITY || ref_b == nb ? 1.f : ex2_approx(ref_b - nb);
                    z_a = f2_mul(z_a, f2_pack(fa, fa));
                    z_b = f2_mul(z_b, f2_pack(fb, fb));
                    ref_a = na;
                    ref_b = nb;
                }
                // a block's factor 2^(byte - 127), byte = X - R + 60, at least 1: weights of a block that lies 2^59 below
                // the reference are that much smaller instead.  (As a float, whole: adding 2^23 leaves it in the low bits.)
                auto factor = [](float t, float r) -> float { return fminf(fmaxf(t - r + (float)kBase, 1.f), 254.f); };
                auto whole_bits = [](float f) -> uint32_t { return __float_as_uint(f + 8388608.f); };
                if (set == 0) {
                    tc_fence_after_sync();
                    tmem_st_32x32b_x2(tmem + lane_addr + TM_SFB + 4u * team,
                                      __byte_perm(whole_bits(factor(tops[0][lane], rl)), whole_bits(factor(tops[1][lane], rl)), 0x4040),
                                      __byte_perm(whole_bits(factor(tops[0][32 + lane], rh)), whole_bits(factor(tops[1][32 + lane], rh)), 0x4040));
                }
                // ---- weights: p = 2^(score - X + K + 7) times scale 2^-K, at most 2^8; z is the sum of p 2^-K
                {
                    const float f_a = factor(max_a, na), f_b = factor(max_b, nb);
                    // (nothing attended so far: the scores are -inf throughout, whatever is subtracted)
                    const float xa = na == -INFINITY ? 7.f : (float)(kBase + 7) - na - f_a + K;
                    const float xb = nb == -INFINITY ? 7.f : (float)(kBase + 7) - nb - f_b + K;
                    const uint64_t ra = f2_pack(xa, xa), rb = f2_pack(xb, xb), ca2 = f2_pack(ca, ca), cb2 = f2_pack(cb, cb), nm2 = f2_pack(nm, nm);
                    uint64_t za = f2_pack(0.f, 0.f), zb = za;
                    uint32_t pa[4], pb[4];  // pieces: hi in the low half, lo in the high half
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float e0, e1;
                        f2_unpack(f2_fma(d2[i], ca2, ra), e0, e1);
                        const uint64_t wa = f2_pack(ex2_approx(e0), ex2_approx(e1));
                        f2_unpack(f2_fma(d2[4 + i], cb2, rb), e0, e1);
                        const uint64_t wb = f2_pack(ex2_approx(e0), ex2_approx(e1));
                        const uint64_t f = f2_mul(sc2[i], nm2);
                        za = i == 0 ? wa : f2_add(za, wa);
                        zb = i == 0 ? wb : f2_add(zb, wb);
                        pa[i] = split_weights(f2_mul(wa, f));
                        pb[i] = split_weights(f2_mul(wb, f));
                    }
                    // neighbouring lanes hold neighbouring pairs of rows: each stores four rows of every other i
                    const bool odd = lane & 1;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t oa = odd ? pa[2 * k + 1] : pa[2 * k], ob = odd ? pb[2 * k + 1] : pb[2 * k];
                        const uint32_t ga = __shfl_xor_sync(0xffffffffu, odd ? pa[2 * k] : pa[2 * k + 1], 1);
                        const uint32_t gb = __shfl_xor_sync(0xffffffffu, odd ? pb[2 * k] : pb[2 * k + 1], 1);
                        // even lanes: rows of i = 2 k, own pair first; odd lanes: of i = 2 k + 1, the neighbour's first
                        st_shared_u32(w_addr[k], __byte_perm(oa, ga, lo_first));
                        st_shared_u32(w_addr[k] + kW / 2, __byte_perm(oa, ga, hi_first));
                        st_shared_u32(w_addr[k] + 512, __byte_perm(ob, gb, lo_first));
                        st_shared_u32(w_addr[k] + 512 + kW / 2, __byte_perm(ob, gb, hi_first));
                    }
                    const float fa = __uint_as_float(whole_bits(f_a) << 23) * nm, fb = __uint_as_float(whole_bits(f_b) << 23) * nm;
                    z_a = f2_fma(za, f2_pack(fa, fa), z_a);
                    z_b = f2_fma(zb, f2_pack(fb, fb), z_b);
                }
                // ---- rows that were not loaded, and NaN codes of drafted rows (attended columns have NaN weights
                // already): a weight of 0 must not meet them.  (A swizzle keeps a row's 128 bytes together.)
                if (!plain) {
                    // (complete since before the score: this makes the copy's bytes visible here too)
                    (void)bar_wait(&ms.kv_full[s_now], s_ph, &ms.abort_flag, a.err_word);
                    uint4 *p = reinterpret_cast<uint4 *>(smem + OFF_ST + s_now * kStage) + (st & (kTeam - 1));
                    const int64_t left = sg.q.len - (int64_t)(sg.t0 + it - first_tile) * kRows;  // the tile's rows of context
#pragma unroll
                    for (int k = 0; k < (int)(4 * kBlk / 16 / kTeam); ++k) {
                        const int r = ((st & (kTeam - 1)) + k * kTeam) >> 3 & (kRows - 1);
                        const bool there = ri.in >> r & 1;
                        if (there && r < left) continue;
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (there) v = p[k * kTeam];
                        p[k * kTeam] = make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
                    }
                }
                if (slow && it > first_tile && __any_sync(0xffffffffu, move != 1.f)) {
                    // this warp's part of the accumulators, 32 columns by 32 dims of each block, where a column moved,
                    // once the context product before is complete.  (The one before that is: the wait above.)
                    wait(&ms.pv_done[before], ((uint32_t)(it - 1) / kTeams) & 1u);
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        if (!__any_sync(0xffffffffu, (lane >> 4) == h && move != 1.f)) continue;
                        const uint32_t at = o_addr + 32u * set + 16u * h;
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
                if (set == 0) tmem_wait_st();
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.w_full[team]);
                s_now += kTeams;
                if (s_now >= kStages) {
                    s_now -= kStages;
                    s_ph ^= 1u;
                }
            }

            // ---- the next segment's queries, by the team that the last tile is not: the last score has read this one's
            if (ms.more[next] && ((uint32_t)(end_tile - 1) % kTeams) != (uint32_t)team) {
                wait(&ms.s_full[team ^ 1], ((uint32_t)(end_tile - 1) / kTeams) & 1u);
                tc_fence_after_sync();
                load_queries(ms.seg[next], 2 * set);
                load_queries(ms.seg[next], 2 * set + 1);
                queries_ready(ms.seg[next]);
            }
            // ---- output
            const int c0 = sg.g * kCols, nc = min(kCols, sg.q.n * a.H - c0);
            const bool whole = sg.first && sg.last;
            float *part = a.part + ((int64_t)blockIdx.x * 2 + (sg.first ? 1 : 0)) * tree_part_floats(kCols);
            // sums over a column's threads, four lanes of each set
            auto to_sets = [&](float u, float v) {
                u += __shfl_xor_sync(0xffffffffu, u, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                u += __shfl_xor_sync(0xffffffffu, u, 2);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if ((lane & 3) == 0) {
                    ms.red[w16][n_a] = u;
                    ms.red[w16][n_b] = v;
                }
            };
            auto over_sets = [&](int n) -> float {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < 2 * kTeams; ++w) v += ms.red[w][n];
                return v;
            };
            float nn = 0.f;
            if (bar_red_or(1, kSoftmax, (zero_a | zero_b) != 0)) {
                to_sets((float)zero_a, (float)zero_b);
                named_sync(1, kSoftmax);
                nn = over_sets(st & (kCols - 1)) * exp2f(-(float)kBase);
                named_sync(1, kSoftmax);
            }
            {
                const float ea = ms.ref[n_a], eb = ms.ref[n_b];  // both teams' last
                float u, v, fa = ref_a == -INFINITY ? 1.f : ex2_approx(ref_a - ea), fb = ref_b == -INFINITY ? 1.f : ex2_approx(ref_b - eb);
                f2_unpack(z_a, u, v);
                fa *= u + v;
                f2_unpack(z_b, u, v);
                fb *= u + v;
                to_sets(fa, fb);
            }
            named_sync(1, kSoftmax);
            if (st < kCols) {
                const float m_end = ms.ref[st], zz = over_sets(st);
                ms.ref[st] = -INFINITY;
                // nothing but zero rows: the accumulators are 0 and stay so
                const float all = nn == 0.f ? zz : zz + nn * exp2f(m_end == -INFINITY ? 0.f : -m_end);
                ms.zinv[st] = !whole ? 1.f : all == 0.f ? 0.f : 1.f / all;
                if (!whole) {
                    part[kCols * kKL + st] = tree_part_exponent(m_end, zz);
                    part[kCols * (kKL + 1) + st] = zz;
                    part[kCols * (kKL + 2) + st] = nn;
                }
            }
            wait(&ms.pv_done[(uint32_t)(end_tile - 1) % kTeams], ((uint32_t)(end_tile - 1) / kTeams) & 1u);
            tc_fence_after_sync();
            named_sync(1, kSoftmax);
            const bool odd = lane & 1;
            if (__all_sync(0xffffffffu, ok)) {
#pragma unroll 1
                for (int u = w16; u < 16; u += 2 * kTeams) {
                    // thread: dim 32 (u & 12) + 32 q + lane of columns h0 .. h0 + 15
                    const int h0 = 16 * (u & 3);
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(o_addr + 64u * (u >> 2) + (uint32_t)h0, o);
                    tmem_wait_ld();
                    const int d = 128 * (u >> 2) + 32 * q + lane;
#pragma unroll
                    for (int k4 = 0; k4 < 4; ++k4) {
                        const float4 a4 = *reinterpret_cast<const float4 *>(&ms.zinv[h0 + 4 * k4]);
                        o[4 * k4] = __float_as_uint(__uint_as_float(o[4 * k4]) * a4.x);
                        o[4 * k4 + 1] = __float_as_uint(__uint_as_float(o[4 * k4 + 1]) * a4.y);
                        o[4 * k4 + 2] = __float_as_uint(__uint_as_float(o[4 * k4 + 2]) * a4.z);
                        o[4 * k4 + 3] = __float_as_uint(__uint_as_float(o[4 * k4 + 3]) * a4.w);
                    }
                    if (!whole || !a.out_bf16) {
                        float *dst = (whole ? static_cast<float *>(a.out) + ((int64_t)sg.q.q0 * a.H + c0) * kKL : part) + h0 * kKL + d;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (h0 + j < nc) dst[j * kKL] = __uint_as_float(o[j]);
                    } else {
                        // even lanes store column j, odd lanes column j + 1: two dims each
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)sg.q.q0 * a.H + c0 + h0 + odd) * kKL + (d & ~1);
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float mine = __uint_as_float(odd ? o[j + 1] : o[j]);
                            const float other = __uint_as_float(__shfl_xor_sync(0xffffffffu, odd ? o[j] : o[j + 1], 1));
                            if (h0 + j + odd < nc)
                                *reinterpret_cast<__nv_bfloat162 *>(dst + j * kKL) =
                                    odd ? __floats2bfloat162_rn(other, mine) : __floats2bfloat162_rn(mine, other);
                        }
                    }
                }
            }
            tc_fence_before_sync();  // the accumulators are read before the next segment's first product
            named_sync(1, kSoftmax);
            now = next;
        }
        // the last copy of queries lands before the CTA ends
        if (st == 0 && segments) bar_wait(&ms.q_ready, (segments - 1) & 1, nullptr, a.err_word, kWaitCycles / 8);
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
    cfg.gridDim = dim3((unsigned)(1 + slots * (kCols / kPrepCols)));
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
