/*
 * kv8mla.h -- C ABI of the fp8 latent-KV absorbed MLA attention library (libkv8mla.so, sm_103a).
 *
 * The operations follow two web pages:
 *   [KV8]  "KV8 long-context CUDA: fp8 device shadow, split-T kernels, DSA-aware gather"
 *          (colibri pull request #300): first commit message (fp8 row format, c/kv_fp8.h codec,
 *          absorb attention, CUDA wrappers coli_cuda_attention_absorb8 / _absorb_batch8) and second
 *          commit message (device-resident shadow, split-T partial blocks + log-sum-exp merge,
 *          DSA gather attention_absorb_sel_kernel8 with NS <= 4096, batch cap lifted to 1M rows).
 *   [B1]   "B1 Mixed FP8/BF16 FMHA first pass", sections "New files" (C ABI launcher driven from
 *          Python through ctypes) and "Intentional first-pass limits" (an unsupported shape is an
 *          error code; there is no fallback path).
 *   [FMT8] "feat: fmt=8 (fp8-e4m3) decode on the kv_b absorb path, CPU and CUDA" (colibri pull
 *          request #1102): kv_b_proj as raw e4m3 bytes with one f32 scale per 128x128 block.
 *
 * Cache layout (one layer).  Row t of the latent cache is KV8_ROW_BYTES = 576 e4m3 bytes:
 * bytes 0..511 are Lc (kv_lora latent), bytes 512..575 are Rc (qk_rope key), followed in a separate
 * array by one f32 scale s_t = amax_t / 448 covering the whole row.  kv8 is [T][576] u8 row-major,
 * kv_scale is [T] f32.  The attended value of row t, head h:
 *     score[h,t] = sm_scale * s_t * ( q_lat[h].e4m3(Lc8_t) + q_rope[h].e4m3(Rc8_t) )
 *     cl[h]      = sum_t softmax_t(score[h,:]) * s_t * e4m3(Lc8_t)            (512 f32 per head)
 * (The latent row serves as key and as value, and the row scale is applied outside the dot product:
 * [KV8] first commit.)
 *
 * Conventions for every call:
 *   - Pointers are DEVICE pointers owned by the caller (unless stated).  The library allocates no
 *     memory, keeps no state between calls, never synchronises the device, and has no CPU
 *     fallback: an unsupported argument is an error code.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls are asynchronous:
 *     a return of KV8_OK means the kernels were enqueued; results are valid once the stream has
 *     reached that point.
 *   - Validation happens on the host before any launch: on any error nothing is enqueued.
 *   - Device buffers must be 16-byte aligned (TMA and vector loads).  Inputs and outputs must not
 *     overlap, except where stated.
 *   - Return values: KV8_OK (0) or a negative KV8_E* code.  kv8_strerror() names it.
 *   - Device-side conditions (a selected index out of range, a wait that timed out) are OR-ed
 *     into *err_word (a device int, optional: may be NULL) as KV8_ERR_* bits; the caller clears it
 *     beforehand and reads it after synchronising.
 */
#ifndef KV8MLA_H
#define KV8MLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KV8_API __attribute__((visibility("default")))
#else
#define KV8_API
#endif

#define KV8_ROW_BYTES 576      /* e4m3 bytes per cache row: Lc then Rc */
#define KV8_KL 512             /* kv_lora rank: latent width, also the context width */
#define KV8_KR 64              /* qk_rope width */
#define KV8_MAX_HEADS 128      /* query heads per call */
#define KV8_MAX_ROWS (1 << 20) /* rows per cache: the 1M cap of [KV8] second commit */
#define KV8_MAX_SELECT 4096    /* selected rows per sequence: NS <= 4096 ([KV8] second commit) */
#define KV8_NOPE 128           /* per-head no-position query / key width (kv_b_proj key rows per head) */
#define KV8_VHEAD 128          /* per-head value width (kv_b_proj value rows per head) */
#define KV8_KVB_BLOCK 128      /* fmt=8 scale block edge: one f32 scale per 128x128 weight block */
#define KV8_IDX_D 128          /* DSA indexer: index key / index query head width */
#define KV8_MAX_IDX_HEADS 128  /* DSA indexer: index heads per query (a multiple of 16) */
#define KV8_MX_NOPE 448        /* mixed cache: no-position values per row (e4m3 + row scale) */
#define KV8_MX_ROPE 64         /* mixed cache: RoPE values per row (bf16) */
#define KV8_MAX_WIDTH 65536    /* kv8_quant_blocks, kv8_matmul8: columns (K); kv8_rope: elements of a head */
#define KV8_MAX_NORM_WIDTH 16384 /* kv8_quant_blocks with a norm: columns */
#define KV8_MAX_ROPE 256       /* kv8_rope: rotated elements of a head */
#define KV8_MAX_SEQS 4096      /* paged calls: sequences per call */
#define KV8_MAX_TREE 256       /* paged calls: drafted tokens per sequence */
#define KV8_MIN_PAGE 16        /* paged calls: rows per page, a power of two from here ... */
#define KV8_MAX_PAGE 65536     /* ... to here */

/* return codes */
#define KV8_OK 0
#define KV8_EINVAL (-1)       /* null pointer, bad size, misalignment, or value outside the limits */
#define KV8_EWORKSPACE (-2)   /* workspace smaller than the matching *_workspace_bytes() */
#define KV8_ECUDA (-3)        /* a CUDA launch or attribute call failed */
#define KV8_EUNSUPPORTED (-4) /* the device is not sm_103 (or the shape has no kernel) */

/* bits OR-ed into *err_word by the device */
#define KV8_ERR_INDEX 1u    /* a selected row index was outside [0, T): that entry was skipped */
#define KV8_ERR_TIMEOUT 2u  /* a bounded wait in a kernel gave up: that output is not valid */
#define KV8_ERR_PAGES 4u    /* kv8_page_plan: the free pages, or the table, did not suffice for a sequence */

/* query element types */
#define KV8_F32 0
#define KV8_BF16 1

/* rotary layouts: which elements of the rotated part form pair i */
#define KV8_ROPE_INTERLEAVED 0 /* 2i and 2i + 1 */
#define KV8_ROPE_HALF 1        /* i and i + rope_dim / 2 */

/* -----------------------------------------------------------------------------------------------
 * kv8_encode_e4m3 -- the element encoder of the row quantizer, without scaling.
 * [KV8] first commit, c/kv_fp8.h item: round to nearest, ties to even; saturate at +-448 (inf
 * included); keep the sign of zero (so -0.0 and negative values that round to zero give 0x80);
 * store NaN as 0x00.
 *   y   [n] f32 in, out [n] u8 out (byte i encodes y[i]).  n >= 0 (n == 0 enqueues nothing).
 *   Alignment: y 16-byte aligned, out 4-byte aligned.
 * --------------------------------------------------------------------------------------------- */
KV8_API int kv8_encode_e4m3(const float *y, int64_t n, uint8_t *out, void *stream);

/* -----------------------------------------------------------------------------------------------
 * kv8_quant_rows -- quantize n f32 rows into cache rows ([KV8] first commit: the producer
 * quantizes the fresh normed/roped row; per-row quantizer with a subnormal-amax guard).
 *   x        [n][576] f32 in (Lc then Rc for each row)
 *   kv8      [n][576] u8 out: pass the cache base + 576*t to write rows t..t+n-1
 *   kv_scale [n] f32 out:     pass the scale base + t
 * Per row, in f32 with IEEE round-to-nearest: amax = max |x_i| over finite x_i; scale = amax/448;
 * y_i = x_i * (448/amax), or, when 448/amax overflows (subnormal amax), (x_i*2^64)*(448/(amax*2^64));
 * when amax == 0, y_i = x_i.  byte_i = kv8_encode_e4m3(y_i).  Bit-exact with the oracle.
 *   n >= 0.  x and kv8 16-byte aligned, kv_scale 4-byte aligned.
 * --------------------------------------------------------------------------------------------- */
KV8_API int kv8_quant_rows(const float *x, int64_t n, uint8_t *kv8, float *kv_scale, void *stream);

/* kv8_quant_rows_w -- the same row quantizer for rows of `width` elements: width = KV8_ROW_BYTES (cache
 * rows, as kv8_quant_rows), KV8_IDX_D (DSA index keys) or KV8_MX_NOPE (mixed-cache no-position parts).  x [n][width] f32 -> q [n][width] e4m3,
 * scale [n] f32.  Any other width is KV8_EINVAL. */
KV8_API int kv8_quant_rows_w(const float *x, int64_t n, int width, uint8_t *q, float *scale, void *stream);

/* -----------------------------------------------------------------------------------------------
 * Split-T decode ([KV8] second commit: flash-decoding style partial online-softmax blocks
 * (cl[K], m, z) plus a log-sum-exp merge kernel; the cache is device-resident, only new rows are
 * uploaded).  One query of H heads over rows 0..T-1.
 *
 * Partition p of P covers rows [floor(T*p/P), floor(T*(p+1)/P)).  The workspace begins with the
 * partial sets (f32), for B batch items (B = 1 for decode):
 *     cl [B][P][H][512]   unnormalised context of each partition, relative to its m
 *     m  [B][P][H]        the partition's reference: the max of score * log2(e) over its rows, or a
 *                         value at most 2 below it (the online softmax rescales lazily); -inf for a
 *                         partition without rows
 *     z  [B][P][H]        sum over the partition of 2^(score*log2(e) - m)
 * The decode workspace continues with the library's own staging (the prepared queries); its size
 * is included in mla_decode8_workspace_bytes.
 * mla_decode8_partitions:      the partition count P the library uses for (H, T, P_req):
 *                              P_req = 0 picks automatically (one CTA per SM of the current device,
 *                              N SMs (152 on GB300; 152 when no device is visible): min(ceil(T/128),
 *                              N/2 for H > 64, else N)), P_req > 0 is clamped to [1, T].  The count
 *                              depends on the device current at the call: size and launch on one device.
 * mla_decode8_workspace_bytes: workspace bytes for (H, T, P_req).
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_decode8_partitions(int H, int64_t T, int P_req, int *P_out);
KV8_API int mla_decode8_workspace_bytes(int H, int64_t T, int P_req, size_t *bytes);

/* mla_decode8_partial -- the partial kernel alone (fills the workspace for P partitions).
 *   q_lat [H][512], q_rope [H][64] of type q_dtype (KV8_F32 or KV8_BF16), 16-byte aligned.
 *   H in [1, 128]; T in [1, KV8_MAX_ROWS]; kv8 [T][576], kv_scale [T].
 *   sm_scale: finite.  err_word: optional (KV8_ERR_TIMEOUT).
 *   workspace: >= mla_decode8_workspace_bytes(H, T, P_req) bytes. */
KV8_API int mla_decode8_partial(const void *q_lat, const void *q_rope, int q_dtype, int H, const uint8_t *kv8,
                        const float *kv_scale, int64_t T, float sm_scale, int P_req, void *workspace,
                        size_t ws_bytes, int *err_word, void *stream);

/* mla_lse_merge8 -- the log-sum-exp merge of B*H partial sets into out [B][H][512] f32:
 *   M = max_p m_p;  w_p = 2^(m_p - M) (0 when m_p = -inf);  Z = sum_p w_p z_p;
 *   out = sum_p w_p cl_p / Z   (0 when Z == 0, i.e. no row was attended).
 * workspace as written by the partial kernels; P in [1, 65535]. */
KV8_API int mla_lse_merge8(const void *workspace, int B, int P, int H, float *out, void *stream);

/* mla_absorb_decode8 -- partial + merge on one stream: out [H][512] f32 = cl for each head. */
KV8_API int mla_absorb_decode8(const void *q_lat, const void *q_rope, int q_dtype, int H, const uint8_t *kv8,
                       const float *kv_scale, int64_t T, float sm_scale, int P_req, void *workspace,
                       size_t ws_bytes, int *err_word, float *out, void *stream);

/* -----------------------------------------------------------------------------------------------
 * mla_absorb_sel8 -- DSA gather decode ([KV8] second commit: attention_absorb_sel_kernel8 attends
 * the selected rows straight from the device cache by absolute index, NS <= 4096; when a
 * selection is active decode attends exactly the selection).
 *   B sequences; sequence b's cache is rows [b*seq_stride_rows, b*seq_stride_rows + T) of
 *   kv8 / kv_scale (seq_stride_rows >= T, or 0 when B == 1).
 *   q_lat [B][H][512], q_rope [B][H][64] (q_dtype); idx [B][NS] int32 absolute row indices into
 *   the sequence's own cache (any order; duplicates attend twice).  An index outside [0, T) is
 *   skipped and sets KV8_ERR_INDEX in *err_word.  out [B][H][512] f32.
 *   NS in [1, KV8_MAX_SELECT]; T in [1, KV8_MAX_ROWS]; H in [1, 128]; B >= 1.
 *   workspace >= mla_sel8_workspace_bytes(B, H, NS): the B x P partial sets, then staging for the
 *   prepared bf16 queries.  P spreads the list's 128-row tiles over one wave of CTAs, one per SM (B items x
 *   P x ceil(H/64)).  bf16 queries run on the tensor cores, which gather the selected rows from all
 *   items' caches with 32-bit row coordinates; f32 queries, and caches with
 *   (B-1)*seq_stride_rows + T >= 2^31 rows, run on the CUDA cores.
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_sel8_workspace_bytes(int B, int H, int NS, size_t *bytes);
KV8_API int mla_absorb_sel8(const void *q_lat, const void *q_rope, int q_dtype, int B, int H, const uint8_t *kv8,
                    const float *kv_scale, int64_t T, int64_t seq_stride_rows, const int32_t *idx, int NS,
                    float sm_scale, void *workspace, size_t ws_bytes, int *err_word, float *out, void *stream);

/* -----------------------------------------------------------------------------------------------
 * mla_absorb_prefill8 -- causal prefill of S new queries ([KV8] first and second commits: the
 * batch/prefill absorb path, coli_cuda_attention_absorb_batch8, tiled streaming, cap 1M rows).
 * Query i sits at position pos0 + i and attends rows 0..pos0+i (row index = position); its own
 * fresh row must already be quantized into the cache (kv8_quant_rows).
 *   q_lat [S][H][512], q_rope [S][H][64] (q_dtype); out [S][H][512] f32.
 *   S >= 1; pos0 >= 0; pos0 + S <= T <= KV8_MAX_ROWS; H in [1, 128].
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_absorb_prefill8(const void *q_lat, const void *q_rope, int q_dtype, int S, int H, int64_t pos0,
                        const uint8_t *kv8, const float *kv_scale, int64_t T, float sm_scale, int *err_word,
                        float *out, void *stream);

/* -----------------------------------------------------------------------------------------------
 * mla_absorb_decode8_noalloc -- mla_absorb_decode8 for callers that cannot allocate device memory.
 * The pages have no counterpart to this call; it exists for users of this library.
 *
 * Some callers cannot call cudaMalloc or reach an allocator for the workspace that the split-T
 * partials need: a plugin loaded into a host program whose memory pool already owns the GPU's
 * memory, a caller from another language runtime with no handle on the host's caching allocator,
 * or a latency-critical loop that must not take cudaMalloc's implicit device synchronisation.
 * This entry point keeps the partials in a fixed array of KV8_NOALLOC_SCRATCH_BYTES that is part of
 * the library's device image: every GPU that loads the library holds it until the process exits.
 * Apart from that module load (below), neither this call nor anything it calls allocates memory.
 *
 * Arguments as mla_absorb_decode8, without workspace / ws_bytes.  P_req == 0 picks the automatic
 * partition count, lowered if needed until the partials fit the array; an explicit P_req whose
 * partials do not fit returns KV8_EWORKSPACE (nothing is enqueued).
 * Every call looks up the array's address in the current device's context (a cheap host query; no
 * address is kept between calls, so a context that was reset and created again is handled).  The
 * first call in a context also loads the library's device module, which places the array: that step
 * can allocate device memory and synchronise, and it fails with KV8_ECUDA if the device has no room
 * left.  A caller whose memory pool takes the whole GPU should therefore make one warm-up call per
 * device at set-up time, before the pool grows and before any stream capture.
 * All calls share the one array and it keeps the last call's contents (each call writes every
 * partial it reads, so nothing needs clearing): calls whose kernels overlap on the GPU (two streams,
 * or two host threads) race on it and must be ordered by the caller.
 * --------------------------------------------------------------------------------------------- */
#define KV8_NOALLOC_SCRATCH_BYTES (16u << 20) /* 16 MiB per device */
KV8_API int mla_absorb_decode8_noalloc(const void *q_lat, const void *q_rope, int q_dtype, int H,
                                       const uint8_t *kv8, const float *kv_scale, int64_t T, float sm_scale,
                                       int P_req, int *err_word, float *out, void *stream);

/* -----------------------------------------------------------------------------------------------
 * mla_absorb_mixed_decode8 -- decode over the mixed-precision cache ([B1] "B1 Mixed FP8/BF16 FMHA first
 * pass": the no-position part of each KV row stored as e4m3 with a per-row f32 scale, the RoPE part as
 * bf16, the query's no-position part quantized from bf16 to e4m3 before the attention; head width
 * 512 = KV8_MX_NOPE + KV8_MX_ROPE; the row is both key and value).  For each head h:
 *     (q8[h], q_scale[h]) = the row quantizer (amax/448) applied to q_nope[h]
 *     score[h][t] = sm_scale * ( q_scale[h] * k_scale[t] * e4m3(q8[h]).e4m3(k8[t]) + q_rope[h].k_rope[t] )
 *     out[h] = sum_t softmax_t(score[h]) * [ k_scale[t] * e4m3(k8[t]) , k_rope[t] ]        (512 f32)
 *   q_nope [H][448], q_rope [H][64] of type q_dtype; k8 [T][448] e4m3 (kv8_quant_rows_w, width 448),
 *   k_scale [T] f32, k_rope [T][64] bf16; out [H][512] f32.  H in [1, 128]; T in [1, KV8_MAX_ROWS].
 *   workspace: >= mla_mixed_decode8_workspace_bytes(H, T) (split-T partial sets as for mla_decode8_partial,
 *   merged by mla_lse_merge8 inside the call; then staging for the query prep).  k8 and k_rope 16-byte aligned.  err_word: optional
 *   (KV8_ERR_TIMEOUT).  Runs on the tensor cores: the no-position product as e4m3 x e4m3 and the RoPE
 *   product as bf16 x bf16 (an f32 RoPE query as bf16 hi + lo), f32 accumulation; the softmax weights
 *   enter the value product as e4m3 hi + lo (no-position values) and bf16 (RoPE values).
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_mixed_decode8_workspace_bytes(int H, int64_t T, size_t *bytes);
KV8_API int mla_absorb_mixed_decode8(const void *q_nope, const void *q_rope, int q_dtype, int H, const uint8_t *k8,
                                     const float *k_scale, const void *k_rope, int64_t T, float sm_scale,
                                     void *workspace, size_t ws_bytes, int *err_word, float *out, void *stream);

/* -----------------------------------------------------------------------------------------------
 * mla_absorb_batch_decode8 -- one decode step for B sequences at once, each with its own cache and length
 * ([KV8] second commit: a device-resident cache per sequence to which each step appends the new rows;
 * the split-T partials and log-sum-exp merge as for one sequence).
 *   Sequence b's cache is rows b*seq_stride_rows .. b*seq_stride_rows + T_max - 1 of kv8 / kv_scale; it
 *   attends its first lens[b] rows (lens: device int32 [B], clamped to [0, T_max]; 0 rows give a zero
 *   output).  q_lat [B][H][512], q_rope [B][H][64] of type q_dtype; out [B][H][512] f32.
 *   B >= 1; H in [1, 128]; T_max in [1, KV8_MAX_ROWS]; seq_stride_rows >= T_max when B > 1.
 *   workspace: >= mla_batch_decode8_workspace_bytes(B, H, T_max) bytes (partial sets [B][P][H] first, as
 *   for one sequence, then the prepared queries).  err_word: optional (KV8_ERR_TIMEOUT).
 * kv8_quant_rows_scatter -- kv8_quant_rows writing input row r to cache row dst_rows[r] (device int64 [n]),
 *   e.g. one fresh row appended to each sequence; a destination outside [0, cache_rows) is skipped and sets
 *   KV8_ERR_INDEX in *err_word (optional).
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_batch_decode8_workspace_bytes(int B, int H, int64_t T_max, size_t *bytes);
KV8_API int mla_absorb_batch_decode8(const void *q_lat, const void *q_rope, int q_dtype, int B, int H,
                                     const uint8_t *kv8, const float *kv_scale, int64_t T_max, int64_t seq_stride_rows,
                                     const int32_t *lens, float sm_scale, void *workspace, size_t ws_bytes,
                                     int *err_word, float *out, void *stream);
KV8_API int kv8_quant_rows_scatter(const float *x, int64_t n, const int64_t *dst_rows, uint8_t *kv8,
                                   float *kv_scale, int64_t cache_rows, int *err_word, void *stream);

/* -----------------------------------------------------------------------------------------------
 * Absorb projections through kv_b_proj stored as fmt=8 ([FMT8] "feat: fmt=8 (fp8-e4m3) decode on
 * the kv_b absorb path, CPU and CUDA": raw e4m3 bytes plus one f32 scale per 128x128 block,
 * block-row-major; the absorbed attention of [KV8] first commit works in the 512-wide latent).
 *   w8 [H*256][512] e4m3 bytes: head h's rows 256h..256h+127 are W_UK (no-position key part,
 *      KV8_NOPE), rows 256h+128..256h+255 are W_UV (value part, KV8_VHEAD).
 *   w_scale [H*2][4] f32: block (r, c) covers rows 128r.., columns 128c..; the weight is
 *      W[o][i] = e4m3(w8[o][i]) * w_scale[(o/128)*4 + i/128].
 * mla_q_absorb8:    q_lat[s][h][c] = sum_{j<128} q_nope[s][h][j] * W[256h + j][c]      (c < 512)
 *   q_nope [S][H][128] of type q_dtype; q_lat [S][H][512] of type out_dtype (KV8_F32 / KV8_BF16;
 *   bf16 rounds the f32 sum to nearest even) -- the query the decode / selection / prefill calls take.
 * mla_out_project8: out[s][h][v] = sum_{c<512} W[256h + 128 + v][c] * ctx[s][h][c]     (v < 128)
 *   ctx [S][H][512] f32 (a normalised context, e.g. mla_lse_merge8's out); out [S][H][128] f32.
 * Sums in f32 over exactly decoded weights; the block scale is applied per 128-column block.  Up to 8
 * rows run on the CUDA cores (the weights read once); more on the tensor cores (kind::f16: every e4m3
 * weight is a bf16; f32 activations as bf16 hi + lo pieces).  err_word: optional (KV8_ERR_TIMEOUT).
 * S in [1, KV8_MAX_ROWS]; H in [1, 128]; all buffers 16-byte aligned; outputs must not overlap inputs.
 * The kernels are programmatic dependents of the kernel launched before them on the stream: they start
 * reading w8 and w_scale while that kernel finishes, and q_nope / ctx only after it has completed.  So
 * w8 and w_scale must not be written by the kernel launched just before this call on the same stream.
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_q_absorb8(const void *q_nope, int q_dtype, int S, int H, const uint8_t *w8, const float *w_scale,
                          void *q_lat, int out_dtype, int *err_word, void *stream);
KV8_API int mla_out_project8(const float *ctx, int S, int H, const uint8_t *w8, const float *w_scale, float *out,
                             int *err_word, void *stream);

/* -----------------------------------------------------------------------------------------------
 * dsa_index_topk8 -- the DSA lightning indexer and its top-k ([B1] page, the commit adding
 * indexer_fp8_score_topk: an e4m3 index query of 64 heads x 128 quantized from bf16, e4m3 index keys
 * read as they are, the score dequantized by q_scale * k_scale, ReLU, weighted sum over the heads,
 * top-k).  For each of B queries b and each position t < T of its key rows t' = b*seq_stride_rows + t:
 *     I[b][t] = sum_h w[b][h] * max(0, q_scale[b][h] * k_scale[t'] * sum_i e4m3(q8[b][h][i]) e4m3(k8[t'][i]))
 * where (q8[b][h], q_scale[b][h]) is the row quantizer applied to q_idx[b][h] (amax/448 per head row).
 *   q_idx [B][HI][128] of type q_dtype (KV8_F32 / KV8_BF16); w [B][HI] f32 (either sign);
 *   k8 [rows][128] e4m3 and k_scale [rows] f32 as written by kv8_quant_rows_w(width = KV8_IDX_D).
 *   scores [B][T] f32 (written: I); idx [B][NS] int32 (written): the min(NS, T) positions with the
 *   largest scores, the smaller position first among equal scores, in ascending position order -- the
 *   selection list mla_absorb_sel8 takes.  When NS > T, idx[b][T..NS-1] is left as it was.
 *   HI a multiple of 16 in [16, KV8_MAX_IDX_HEADS]; T in [1, KV8_MAX_ROWS]; NS in [1, KV8_MAX_SELECT];
 *   seq_stride_rows >= 0 and (B-1)*seq_stride_rows + T < 2^31 - 128; buffers 16-byte aligned.
 *   workspace: >= dsa_index_workspace_bytes(B) bytes (the top-k's histograms and the barrier counters of
 *   the CTAs that share a query; zeroed by the call itself).  err_word: optional (KV8_ERR_TIMEOUT).
 *   The scores run on the tensor cores (e4m3 x e4m3, f32 sums); the top-k is one cooperative launch
 *   whose CTAs meet at time-bounded barriers (a barrier that gives up sets KV8_ERR_TIMEOUT).
 * --------------------------------------------------------------------------------------------- */
KV8_API int dsa_index_workspace_bytes(int B, size_t *bytes);
KV8_API int dsa_index_topk8(const void *q_idx, int q_dtype, const float *w, int B, int HI, const uint8_t *k8,
                            const float *k_scale, int64_t T, int64_t seq_stride_rows, int NS, void *workspace,
                            size_t ws_bytes, float *scores, int32_t *idx, int *err_word, void *stream);

/* -----------------------------------------------------------------------------------------------
 * Paged caches and drafted tokens.  The pages have no counterpart to these calls; they exist for users
 * of this library who serve many sequences from one cache and verify several drafted tokens per step.
 *
 * A paged cache is one buffer of rows (kv8 [cache_rows][576], kv_scale [cache_rows], as everywhere) cut
 * into pages of page_size rows, page g being rows g*page_size .. (g+1)*page_size - 1.  Sequence b's
 * position t lives in cache row
 *     block_table[b][t / page_size] * page_size + t % page_size        (block_table: device int32 [B][max_pages])
 * page_size is a power of two in [KV8_MIN_PAGE, KV8_MAX_PAGE].  Table entries past a sequence's rows are
 * not read.
 *
 * A step adds n_b = q_start[b+1] - q_start[b] rows to sequence b, whose first lens[b] rows are already
 * there (device int32 lens [B], q_start [B+1], ascending from 0 to R): the step's row q_start[b] + i is
 * the sequence's drafted token i and lives at position lens[b] + i, whatever branch it stands on.  n_b may
 * differ between sequences and may be 0; n_b <= KV8_MAX_TREE; B in [1, KV8_MAX_SEQS].
 * A sequence whose numbers are not possible (lens[b] < 0, n_b < 0 or too large, rows outside [0, R), more
 * positions than its table holds) is skipped, what it would have written is left as it was, and
 * KV8_ERR_INDEX is set.  Where a possible sequence's rows begin before the end of an earlier possible one's
 * (which takes a q_start that falls between them), kv8_page_plan and mla_absorb_tree8 skip every sequence,
 * with KV8_ERR_INDEX; kv8_tree_mask leaves words of either in rows that two sequences claim.
 *
 * kv8_page_plan -- block tables and slot maps from the lengths.  Afterwards every sequence holds exactly
 * the pages of its lens[b] + n_b rows, and slots[q_start[b] + i] is the cache row of its position
 * lens[b] + i: the dst_rows that kv8_quant_rows_scatter takes.
 *   n_pages [B] int32 in/out: pages the sequence holds, block_table[b][0 .. n_pages[b]).
 *   block_table in/out: entries of new pages are written, all others left.
 *   free_list [free_cap] int32, n_free [1] int32 in/out: a stack of free pages, its top at n_free - 1.
 *   slots [R] int64 out.  free_cap >= 0, R >= 0 (free_list / slots may be NULL when 0).
 * First every sequence returns the pages it holds beyond its rows; then missing pages are taken from the
 * top, sequence by sequence in order.  Pages return in the order that makes the same growth take the same
 * pages again.  A sequence that wants more pages than are left after the ones before it (their wants
 * counted whether met or not), or more than max_pages (which counts as no want), keeps the pages it has,
 * gets -1 in its slots and sets KV8_ERR_PAGES.  The result depends on the arguments alone.  n_pages[b]
 * outside [0, max_pages], n_free outside [0, free_cap], or more returned pages than free_cap holds:
 * KV8_ERR_INDEX, as above (for n_free: every sequence).
 * Lengths of 0 return all of a sequence's pages.  A prompt of more than KV8_MAX_TREE rows is planned in
 * several calls of up to that many.
 * A page has one holder: it stands in one sequence's row of the table or on the free list.  Nothing here
 * counts the holders of a page that sequences share (a common prefix): each of them would return it, and
 * two would be given it.  Sequences may share pages as long as none shrinks below them.
 * --------------------------------------------------------------------------------------------- */
KV8_API int kv8_page_plan(int B, const int32_t *lens, const int32_t *q_start, int R, int page_size, int max_pages,
                          int32_t *n_pages, int32_t *block_table, int32_t *free_list, int free_cap, int32_t *n_free,
                          int64_t *slots, int *err_word, void *stream);

/* kv8_tree_mask -- from each drafted token's parent, the tokens it attends and its position.
 *   parent [R] int32: the index, within the sequence, of the token before it on its branch, smaller than
 *   its own; -1 for a token that follows the context directly (a sequence may have several).
 *   mask [R][mask_words] uint32 out: bit j of row q_start[b] + i (word j/32, bit j%32) is set when j is i
 *   or one of its ancestors.  mask_words in [1, KV8_MAX_TREE/32]; a sequence with more than 32*mask_words
 *   tokens is skipped (KV8_ERR_INDEX).
 *   position [R] int32 out (may be NULL): lens[b] + number of i's ancestors: the angle index of its RoPE.
 *   A parent outside [-1, i) counts as -1 and sets KV8_ERR_INDEX.  lens may be NULL (positions from 0). */
KV8_API int kv8_tree_mask(int B, const int32_t *q_start, const int32_t *lens, int R, const int32_t *parent,
                          uint32_t *mask, int mask_words, int32_t *position, int *err_word, void *stream);

/* -----------------------------------------------------------------------------------------------
 * mla_absorb_tree8 -- absorbed attention of every drafted token, over the paged cache.  For row
 * r = q_start[b] + i and head h, over the sequence's rows t with the cache row's bytes and scale s_t:
 *     score[t] = sm_scale * s_t * ( q_lat[r][h].e4m3(Lc8_t) + q_rope[r][h].e4m3(Rc8_t) )
 *     out[r][h] = sum_t softmax_t(score) * s_t * e4m3(Lc8_t)
 * where t runs over the context 0 .. lens[b]-1 and over lens[b] + j for every set bit j < n_b of r's mask
 * row.  Nothing to attend gives zeros.  mask NULL: token i attends drafted tokens 0 .. i (a chain; one
 * token per sequence is an ordinary decode step, several are a chunk of a causal prefill).
 * The drafted rows must be in the cache already (kv8_quant_rows_scatter).
 *   q_lat [R][H][512], q_rope [R][H][64] of type q_dtype; out [R][H][512] of type out_dtype (KV8_F32 /
 *   KV8_BF16; bf16 rounds to nearest even).  R in [1, KV8_MAX_ROWS]; H in [1, 128]; rows of out outside
 *   every sequence are left as they were.  cache_rows in [1, 2^31).
 *   mask [R][mask_words] uint32 as kv8_tree_mask writes it (any bits: it need not be a tree); bits past
 *   32*mask_words count as 0.
 *   A page outside the cache: its rows are left out and KV8_ERR_INDEX is set.  Rows that nobody attends
 *   may hold anything, NaN codes and scales included.  Scales are not negative.
 *   A NaN or an infinity in a query makes that (row, head)'s output NaN where it attends anything, and no
 *   other.
 *   bf16 queries: scales are 0 or from 2^-60 to 2^60.  An attended row with a larger one makes the output
 *   NaN; one with a smaller one (its values are below 3.9e-16) counts as a row of zeros: score 0, nothing
 *   added to the output, not even a query's NaN.
 *   Scores lie within 5.8e6 (2^23 log 2) of 0 for bf16 queries, 2.3e7 (2^25 log 2) for f32 queries: a
 *   (row, head) whose largest ones do not is NaN.
 *   workspace: >= mla_tree8_workspace_bytes(R, H, B, q_dtype) bytes; calls that may overlap on the GPU
 *   (graph replays included) need their own.  err_word: optional.
 * bf16 queries run on the tensor cores: a query element to 2^-17 of its head's largest, the weights
 * softmax_t s_t to 2^-8 of themselves, or of 2^-17 times the largest of their 32 rows (in 64 context rows
 * with scales within 2^8 of one another: times the largest softmax_t and scale).  f32 queries run there
 * too, a query element and a weight as two f16 values each (2^-22), with f32 sums.  The work is cut into equal shares of row tiles for the device's SMs, whatever the
 * lengths; what a share leaves unfinished is joined by log-sum-exp.
 * --------------------------------------------------------------------------------------------- */
KV8_API int mla_tree8_workspace_bytes(int R, int H, int B, int q_dtype, size_t *bytes);
KV8_API int mla_absorb_tree8(const void *q_lat, const void *q_rope, int q_dtype, int R, int H, int B,
                             const int32_t *q_start, const int32_t *lens, const uint32_t *mask, int mask_words,
                             const uint8_t *kv8, const float *kv_scale, int64_t cache_rows, const int32_t *block_table,
                             int max_pages, int page_size, float sm_scale, void *workspace, size_t ws_bytes,
                             int *err_word, void *out, int out_dtype, void *stream);

/* kv8_tree_commit -- after the target model has chosen a branch: moves the branch's rows next to the
 * context, in every layer's cache at once.  For k < n_accept[b], position lens[b] + accept[b][k] is
 * copied to position lens[b] + k (bytes and scale), and new_lens[b] = lens[b] + n_accept[b].
 *   accept [B][max_accept] int32, strictly ascending within the first n_accept[b], each in [0, n_b).
 *   kv8 [layers][cache_rows][576], kv_scale [layers][cache_rows], one block table for all layers.
 *   new_lens [B] int32 out, must not overlap lens.  max_accept in [1, KV8_MAX_TREE]; layers in [1, 65535].
 *   A branch that is not ascending or not in the draft, n_accept[b] outside [0, max_accept], a page
 *   outside the cache: nothing of the sequence moves, new_lens[b] = lens[b], KV8_ERR_INDEX.
 *   Sequences must not share the pages of the rows that move. */
KV8_API int kv8_tree_commit(int B, const int32_t *q_start, const int32_t *lens, const int32_t *accept,
                            const int32_t *n_accept, int max_accept, int layers, uint8_t *kv8, float *kv_scale,
                            int64_t cache_rows, const int32_t *block_table, int max_pages, int page_size,
                            int32_t *new_lens, int *err_word, void *stream);

/* -----------------------------------------------------------------------------------------------
 * What stands around the attention in a layer: the projections, the rotation of the query heads, and the
 * producer that [KV8]'s first commit speaks of, which quantizes the fresh normed / roped row.  In a layer's order:
 * kv8_quant_blocks (hidden states) -> kv8_matmul8 (query and latent projections) -> kv8_norm_rope_rows (rows into
 * the cache) and kv8_rope (query heads) -> mla_q_absorb8 -> an attention call -> mla_out_project8 ->
 * kv8_quant_blocks -> kv8_matmul8 (output projection).
 *
 * Rotary positions.  Pair i of a rotated part (u, v: KV8_ROPE_INTERLEAVED or KV8_ROPE_HALF) at position p becomes
 *     u' = rope_scale (u cos a - v sin a),   v' = rope_scale (u sin a + v cos a),   a = p inv_freq[i]
 * with inv_freq [rope_dim / 2] f32 (device; from -2^40 to 2^40), position [n] int32 (any value; a negative one turns back,
 * so -p undoes p where rope_scale is 1).  The frequency's part of a turn is held to 2^-65, the turn to |p| 2^-65, and its cosine
 * and sine to 6 roundings of f32 relative to themselves: neither positions of a million nor the smallest angles lose anything.
 * A scaling for long contexts is a choice of inv_freq, and of a factor on the scores.  rope_scale is a factor on the rotated
 * elements alone: on a head of which only a part is rotated (this library's: 64 elements of a key beside 512 or 128 others) it scales
 * that part's share of the scores and nothing else.  A factor on whole queries and keys belongs, squared, in sm_scale.
 *
 * kv8_rope_freqs -- such a choice, on the host: inv_freq [rope_dim / 2] and *rope_scale are HOST memory.
 *   f_i = theta^(-2i / rope_dim); with factor = 1 the table is f and the scale 1.  With factor > 1 the frequencies are
 *   interpolated by parts ("YaRN: Efficient Context Window Extension of Large Language Models", NTK-by-parts): a pair that
 *   makes more than beta_fast turns in `context` positions keeps f_i, one that makes fewer than beta_slow gets
 *   f_i / factor, and between the two pairs (their numbers rounded outward, limited to [0, rope_dim - 1]) the share of
 *   f_i / factor grows linearly with i; the scale is 0.1 ln(factor) + 1.  The method multiplies whole queries and whole keys with that
 *   scale.  Where a head is rotated as a whole, it is the rope_scale of both; for this library's heads rope_scale stays 1 and the
 *   attention call's sm_scale is multiplied by its square.
 *   rope_dim even in [2, KV8_MAX_ROPE]; theta > 1; factor >= 1; context >= 1; 0 < beta_slow <= beta_fast.
 * --------------------------------------------------------------------------------------------- */
KV8_API int kv8_rope_freqs(int rope_dim, double theta, double factor, double context, double beta_fast, double beta_slow,
                           float *inv_freq, float *rope_scale);

/* kv8_rope -- rotates elements [rope_at, rope_at + rope_dim) of each head and hands the two parts out apart, as
 * mla_q_absorb8 (the rest) and the attention calls (the rotated part) take them.
 *   x [n][heads][width] of type x_dtype, element (r, h, e) at x[r * x_row_stride + h * x_head_stride + e]; strides in
 *   elements, >= 0 (0 repeats).
 *   rot [n][heads][rope_dim], rest [n][heads][width - rope_dim] (the elements before the rotated part, then those after
 *   it) of type out_dtype, with strides of their own that keep them apart; rest may be NULL: it is not written.
 *   In place: rot = x + rope_at with x's strides and type, rest NULL.  No other overlap.
 *   n in [0, KV8_MAX_ROWS]; heads in [1, KV8_MAX_HEADS]; rope_dim even in [2, KV8_MAX_ROPE]; width up to KV8_MAX_WIDTH.
 *   Pointers are aligned to their elements; where pointers, strides, rope_at and both parts' widths are multiples of 8
 *   elements (and pointers of 16 bytes) the call is several times faster.
 *   f32 arithmetic, one rounding to out_dtype; the rest is copied.  NaN and infinities stay in their pair. */
KV8_API int kv8_rope(const void *x, int x_dtype, int64_t n, int heads, int width, int rope_at, int rope_dim,
                     int64_t x_row_stride, int64_t x_head_stride, const int32_t *position, const float *inv_freq,
                     float rope_scale, int layout, void *rot, int64_t rot_row_stride, int64_t rot_head_stride, void *rest,
                     int64_t rest_row_stride, int64_t rest_head_stride, int out_dtype, void *stream);

/* kv8_norm_rope_rows -- a projection's rows made into cache rows: of each row x [576], elements 0..511 are normed,
 *     y_i = x_i norm_w[i] / sqrt(mean over 512 of x^2 + eps),
 * elements 512..575 rotated, and the 576 results quantized as kv8_quant_rows does and written to cache row dst_rows[r].
 *   x [n][576] of type x_dtype, rows x_stride elements apart (>= 576; x and the rows 16-byte aligned): the rows may be
 *   part of a wider projection's output.  norm_w [512] f32; eps >= 0.
 *   dst_rows [n] int64, as kv8_page_plan's slots: rows that differ from one another; one outside [0, cache_rows) is
 *   skipped and sets KV8_ERR_INDEX (slots of -1 among them).
 *   Between x and the quantizer all arithmetic is f32 and nothing is rounded to fewer bits.  Rows of any finite magnitude
 *   are normed (squares that leave the f32 range are summed in f64).  A NaN or an infinity among the 512 makes their
 *   bytes 0, one among the 64 those of its pair (0, or the largest code), as kv8_quant_rows does with them. */
KV8_API int kv8_norm_rope_rows(const void *x, int x_dtype, int64_t n, int64_t x_stride, const float *norm_w, float eps,
                               const int32_t *position, const float *inv_freq, float rope_scale, int layout,
                               const int64_t *dst_rows, uint8_t *kv8, float *kv_scale, int64_t cache_rows, int *err_word,
                               void *stream);

/* kv8_quant_blocks -- rows to e4m3 with one f32 scale for each block of 128 columns: the left operand of kv8_matmul8.
 * Every block is quantized as kv8_quant_rows quantizes a row (amax / 448 over its finite values, the same bytes).
 *   x [n][width] of type x_dtype, rows x_stride elements apart (>= width; x and the rows 16-byte aligned).
 *   norm_w [width] f32 (16-byte aligned) or NULL: with it, x_i is first replaced by x_i norm_w[i] / sqrt(mean(x^2) + eps),
 *   in f32, not rounded in between; a row with a NaN or an infinity becomes bytes and scales of 0.
 *   q [n][width] u8; scale: block k of row r at scale[k * scale_stride + r] (f32, scale_stride >= n), so one block's
 *   scales of all rows lie together.  The last block is shorter where width is no multiple of 128.
 *   width a multiple of 16 in [16, KV8_MAX_WIDTH], with a norm up to KV8_MAX_NORM_WIDTH; n in [0, KV8_MAX_ROWS]. */
KV8_API int kv8_quant_blocks(const void *x, int x_dtype, int64_t n, int width, int64_t x_stride, const float *norm_w, float eps,
                             uint8_t *q, float *scale, int64_t scale_stride, void *stream);

/* kv8_matmul8 -- product of e4m3 rows with an fmt=8 weight ([FMT8]: one f32 scale per 128 x 128 block):
 *     out[m][n] = sum_kb sa[kb][m] w_scale[n / 128][kb] sum_{k in block kb} e4m3(a8[m][k]) e4m3(w8[n][k])
 *   a8 [M][K] u8, rows a_stride bytes apart (>= K, a multiple of 16); sa[kb][m] = a_scale[kb * a_scale_stride + m] as
 *   kv8_quant_blocks writes it, or a_scale_stride = 0: one scale a row.  The latter takes the rows of a latent cache as
 *   they lie (K = 512, a_stride = 576, a_scale = kv_scale): an expansion of cached rows through kv_b.
 *   w8 [N][K] u8, w_scale [ceil(N/128)][ceil(K/128)] f32.  out [M][N] of type out_dtype, rows out_stride elements apart.
 *   M in [0, KV8_MAX_ROWS]; N in [1, KV8_MAX_ROWS]; K a multiple of 16 in [16, KV8_MAX_WIDTH].  a8 and w8 16-byte
 *   aligned; out aligned to its elements, and faster where it and its rows lie on 16 bytes.
 *   err_word: optional (KV8_ERR_TIMEOUT).
 * The products are exact, a block's sum is taken by the tensor cores in f32, the scaled sums are added in f32; bf16 output
 * rounds once.  A NaN code makes the outputs of its row (of a8) or column (of w8) NaN.  A pair of scales whose product is
 * below 2^-126 or beyond f32 counts as that product is rounded in f32. */
KV8_API int kv8_matmul8(const uint8_t *a8, int64_t a_stride, const float *a_scale, int64_t a_scale_stride, int M, int N, int K,
                        const uint8_t *w8, const float *w_scale, void *out, int out_dtype, int64_t out_stride, int *err_word,
                        void *stream);

/* -----------------------------------------------------------------------------------------------
 * kv8_copy -- copy `bytes` bytes from src to dst with a kernel (the SMs' loads and stores, not a
 * copy engine).  The pages have no counterpart to this call; it exists for users of this library:
 * on a GPU whose host memory is coherently attached (NVLink-C2C), it moves a step's small inputs
 * and outputs between page-locked host memory and the device with less fixed cost per transfer
 * than a copy-engine memcpy.
 *   dst, src: device memory of the current device, managed memory, or page-locked host memory
 *   (cudaHostAlloc / cudaMallocHost / cudaHostRegister), in any combination and any alignment
 *   (16-byte aligned pointers take the vector path).  The ranges must not overlap.
 *   Pageable host memory, another device's memory or an unknown pointer is KV8_EINVAL (checked
 *   with cudaPointerGetAttributes on the host; nothing is enqueued).  bytes == 0 enqueues nothing.
 *   Stream-ordered and asynchronous like every call.
 * --------------------------------------------------------------------------------------------- */
KV8_API int kv8_copy(void *dst, const void *src, size_t bytes, void *stream);

/* -----------------------------------------------------------------------------------------------
 * kv8_wait_selftest -- diagnostic of the timeout path.  One CTA waits on an mbarrier that nothing
 * completes, through the bounded waits the library's tensor-core kernels use for their TMA, MMA,
 * softmax and cluster hand-offs, one after the other: one with its limit in nanoseconds, three in cycles of the SM's
 * clock (2 a nanosecond).  After limit_ns (in [1000, 1e9] ns; the last two, those of kv8_matmul8, after a quarter of it)
 * each gives up: KV8_ERR_TIMEOUT is OR-ed into *err_word, *wait_status is set to 2 (1 would mean that a wait completed,
 * or did not report) and the kernel returns normally, leaving the context usable.  err_word and wait_status: device ints (required).
 * --------------------------------------------------------------------------------------------- */
KV8_API int kv8_wait_selftest(uint64_t limit_ns, int *err_word, int *wait_status, void *stream);

/* Name of a return code (static string). */
KV8_API const char *kv8_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* KV8MLA_H */
