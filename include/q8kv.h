/*
 * q8kv.h -- C ABI of the q8-KV single-query decode-attention library for NVIDIA B200
 * (sm_100a). Shared library: decode_attention_int8_b200/libq8kv.so.
 *
 * The operation (Kestrel-LLM walk-through "flash_attn_single_q_q8_neon",
 * trdm.cn/news/511694, section 2 parts 1-3): for every batch entry b and query head h,
 *   1. quantise q[b][h] once to int8 in 32-element blocks: qm = max|q| (if qm < 1e-6 then
 *      qm = 1), qsc_j = qm * fl(1/127), code = clamp(round-half-to-even(q * fl(127/qm)),
 *      -127, 127), all in IEEE fp32;
 *   2. for every token t < seq_lens[b], with kv = h / (n_q_heads / n_kv_heads) (the GQA
 *      mapping of the llama2.c loop, aicoding.csdn.net, "attention core logic") and
 *      slot = block_table[b][t / kv_block_size] * kv_block_size + t % kv_block_size
 *      (beaiera.top "deepseek-attention-div64", "Top-K index global mapping"):
 *        dot_j = sum over the 32 channels of block j of code * K[slot][kv]   (int32, exact)
 *        s_t   = (sum_j dot_j * qsc_j) * kscale[slot][kv] * scale
 *   3. out[b][h] = sum_t exp(s_t - M) * vscale[slot][kv] * V[slot][kv] / sum_t exp(s_t - M),
 *      computed in one pass with a running max M and running sum S (online softmax) and
 *      one division at the end.
 * The scan is split over the sequence across thread blocks (flash-decoding) and the
 * pieces are merged by a log-sum-exp combine kernel launched right after the decode
 * kernel on the same stream; the result equals the single pass up to fp32 rounding order.
 * Both kernels use programmatic dependent launch: each may be scheduled while the kernel
 * before it on the stream drains, and waits for that kernel to complete before it reads
 * or writes global memory.
 *
 * Layouts (all row-major, C order):
 *   q            fp32  [B][n_q_heads][head_dim]
 *   out          fp32  [B][n_q_heads][head_dim]
 *   k_blocks     int8  [num_kv_blocks][kv_block_size][n_kv_heads][head_dim]
 *   v_blocks     int8  same shape as k_blocks
 *   kscale       fp32  [num_kv_blocks][kv_block_size][n_kv_heads]  (dequant multipliers:
 *   vscale       fp32  same shape                                   value = code * scale)
 *   block_table  int32 [B][max_blocks_per_seq]  physical block of each logical block;
 *                      entries past ceil(seq_lens[b] / kv_block_size) are never read
 *   seq_lens     int32 [B]
 * The same block table indexes both pools and both scale arrays; scales are indexed by
 * the physical slot.
 *
 * Pointers: device pointers owned by the caller; the library never frees or retains
 * them. q, out, k_blocks, v_blocks, kscale, vscale must be 16-byte aligned (any torch or
 * cudaMalloc allocation is).
 *
 * Asynchrony: every call enqueues work on `stream` (NULL = legacy default stream) and
 * returns without synchronising. Q8KV_OK means the work was enqueued; faults surface at
 * the caller's next synchronisation.
 *
 * Errors: argument checks run on the host before any launch and return
 * Q8KV_ERR_INVALID_ARG or Q8KV_ERR_UNSUPPORTED without touching the GPU. Data that only
 * the device can see is checked in the kernel without trapping: a seq_len below 0 is
 * treated as 0, one above max_blocks_per_seq * kv_block_size is clamped, a block-table
 * entry outside [0, num_kv_blocks) makes the kernel skip that block's tokens; each of
 * these sets a bit in a device-side error word that q8kv_device_errors() reads.
 *
 * Supported shapes of the decode kernel: head_dim 128; kv_block_size a power of two in
 * [16, 256]; n_q_heads a multiple of n_kv_heads; query rows per KV head R (the group
 * n_q_heads / n_kv_heads, times n_queries for q8kv_decode_attn_multi) at most 128; a tile
 * holds up to 8 / ceil_pow2(R / 16) KV heads, and when it holds fewer than n_kv_heads (its
 * scales then come through a 2-D copy whose rows must be 16-byte multiples) n_kv_heads
 * must be a multiple of 4; B <= 16384; num_kv_blocks * kv_block_size < 2^31. Other shapes
 * return Q8KV_ERR_UNSUPPORTED.
 */
#ifndef Q8KV_H
#define Q8KV_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    Q8KV_OK = 0,
    Q8KV_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, bad alignment, ... */
    Q8KV_ERR_UNSUPPORTED = 2, /* valid arguments outside the shapes the kernels handle */
    Q8KV_ERR_CUDA = 3,        /* a CUDA runtime call failed: see q8kv_last_cuda_error() */
    Q8KV_ERR_WORKSPACE = 4    /* workspace null or smaller than q8kv_workspace_bytes() */
} q8kv_status;

/* Device-side error bits reported by q8kv_device_errors(). */
#define Q8KV_DEVERR_SEQ_LEN 0x1u     /* a seq_len was negative or too long (clamped)     */
#define Q8KV_DEVERR_BLOCK_TABLE 0x2u /* a block-table entry was outside the pool (skipped) */
#define Q8KV_DEVERR_TIMEOUT 0x4u     /* a pipeline wait ran past its limit (kernel gave up) */
#define Q8KV_DEVERR_SLOT 0x8u        /* cache write: a slot past the pool (row skipped)     */
#define Q8KV_DEVERR_NONFINITE 0x10u  /* cache write: a row held inf or NaN (codes 0, NaN scale) */
#define Q8KV_DEVERR_META 0x20u       /* QUEST metadata: a metadata-table entry outside its pool
                                        (row skipped), or a table too short for a request */
#define Q8KV_DEVERR_POSITION 0x40u   /* rotary write: a position outside the table (clamped)  */
#define Q8KV_DEVERR_PROBS 0x80u      /* draft verification: a draft token or draft count out of
                                        range, or no probability to draw a token from         */

/* The first call of an entry point on a device sets up (the error word's address, the kernels'
 * attributes): make it before a stream capture begins. */

/* Element type of rows that may come in several (q8kv_rope_cache_write, q8kv_verify_draft). */
typedef enum { Q8KV_F32 = 0, Q8KV_F16 = 1, Q8KV_BF16 = 2 } q8kv_dtype;

/*
 * Decode attention with a library-managed workspace (one per device, grown on demand
 * under a lock, zero-initialised; the first call on a device, or a call that needs a
 * larger workspace, allocates and so must not happen during stream capture). Smaller ones are
 * kept, so a captured graph stays valid after such a call. Calls that
 * run concurrently on different streams of one device, replays of captured graphs among them,
 * must use q8kv_decode_attn_ws with separate workspaces.
 *
 *   out, q, k_blocks, v_blocks, kscale, vscale, block_table, seq_lens: see the layouts above
 *   B                  batch size (> 0)
 *   n_q_heads          query heads (> 0, a multiple of n_kv_heads)
 *   n_kv_heads         KV heads (> 0)
 *   head_dim           channels per head (128)
 *   kv_block_size      tokens per physical block
 *   max_blocks_per_seq row stride of block_table; seq_lens[b] <= max_blocks_per_seq *
 *                      kv_block_size
 *   num_kv_blocks      physical blocks in each pool (bounds every block-table entry)
 *   scale              softmax scale (finite; 1/sqrt(head_dim) in standard attention,
 *                      beaiera.top "deepseek-attention-div64", "derivation of the scale")
 */
q8kv_status q8kv_decode_attn(float *out, const float *q, const int8_t *k_blocks,
                             const int8_t *v_blocks, const float *kscale, const float *vscale,
                             const int32_t *block_table, const int32_t *seq_lens, int B,
                             int n_q_heads, int n_kv_heads, int head_dim, int kv_block_size,
                             int max_blocks_per_seq, int num_kv_blocks, float scale,
                             cudaStream_t stream);

/*
 * Decode attention with several new query tokens per sequence (speculative or multi-token
 * decode), library-managed workspace. The llama.cpp change on baguaai.com's FlashAttention
 * page moves quantised-KV decode from a per-query (VEC) kernel to a tiled (TILE) one; here
 * the n_queries tokens of a sequence share every K/V tile it streams, as extra rows of the
 * same tensor-core tiles, so the cache is read once for all of them.
 *
 *   q, out     fp32 [B][n_queries][n_q_heads][head_dim]
 *   seq_lens   tokens in the cache per sequence, the n_queries new ones included (they are
 *              its last n_queries tokens, written beforehand, e.g. by q8kv_cache_write)
 * Query i of sequence b attends causally to tokens t < seq_lens[b] - (n_queries - 1 - i),
 * with the single-query arithmetic of q8kv_decode_attn per (b, i, head); a query that sees
 * no token (seq_lens[b] < n_queries - i) gets a zero row. n_queries = 1 is
 * q8kv_decode_attn. Supported shapes: as above with R = n_queries * n_q_heads /
 * n_kv_heads rows per KV head. With n_queries > 1, 9 <= R <= 32 and n_kv_heads 1 or a
 * multiple of 4, the call runs on the fifth-generation tensor cores (tcgen05.mma with
 * int32 accumulators in tensor memory; rows padded to 16 or 32); other shapes on the warp
 * MMAs of q8kv_decode_attn. Both give the same results within the documented tolerance.
 * Other arguments, errors and asynchrony as q8kv_decode_attn.
 */
q8kv_status q8kv_decode_attn_multi(float *out, const float *q, const int8_t *k_blocks,
                                   const int8_t *v_blocks, const float *kscale,
                                   const float *vscale, const int32_t *block_table,
                                   const int32_t *seq_lens, int B, int n_queries, int n_q_heads,
                                   int n_kv_heads, int head_dim, int kv_block_size,
                                   int max_blocks_per_seq, int num_kv_blocks, float scale,
                                   cudaStream_t stream);

/*
 * Decode attention over a q4_0 KV cache (llama.cpp's q4_0 blocks, one of the quantised
 * KV-cache types of the llama.cpp change on baguaai.com's FlashAttention page),
 * library-managed workspace:
 *   k4_blocks, v4_blocks  uint8 [num_kv_blocks][kv_block_size][n_kv_heads][head_dim / 2]:
 *                         4-bit codes, channel 2i in the low nibble of byte i, 2i + 1 in
 *                         the high nibble
 *   kd, vd                binary16 bits [num_kv_blocks][kv_block_size][n_kv_heads]
 *                         [head_dim / 32]: the scale d of each 32-channel block
 * The value of channel c of a row is (code_c - 8) * d_(c / 32). With the query quantised
 * as in step 1 above, token t scores
 *   s_t = (sum_j dot_j * qsc_j * dk_tj) * scale,  dot_j = sum over block j of qi * (code - 8)
 * (exact int32), and out is the online-softmax average of the V values. Other arguments,
 * layouts and asynchrony as q8kv_decode_attn; kd and vd must be 8-byte aligned. Supported:
 * head_dim 128; group n_q_heads / n_kv_heads <= 16; B * n_kv_heads <= 65535. Two kernel
 * launches (per chunk of 256 tokens, then a merge of the chunks).
 * The workspace grows with B * max_blocks_per_seq, and a call that needs a larger one frees the
 * last: a graph captured before such a call must not be replayed after it (make the largest
 * call first).
 */
q8kv_status q8kv_decode_attn_q4(float *out, const float *q, const uint8_t *k4_blocks,
                                const uint8_t *v4_blocks, const uint16_t *kd,
                                const uint16_t *vd, const int32_t *block_table,
                                const int32_t *seq_lens, int B, int n_q_heads, int n_kv_heads,
                                int head_dim, int kv_block_size, int max_blocks_per_seq,
                                int num_kv_blocks, float scale, cudaStream_t stream);

/* Bytes of workspace q8kv_decode_attn_ws needs for these sizes on the current device
 * (0 if the sizes are invalid or unsupported). */
size_t q8kv_workspace_bytes(int B, int n_q_heads, int n_kv_heads, int head_dim);

/* Zero a caller-owned workspace. Optional and without effect on results: no part of the
 * workspace needs an initial value (every call writes the partial results its combine
 * step reads before that step reads them); it only gives a fresh workspace defined
 * contents. */
q8kv_status q8kv_workspace_init(void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Same as q8kv_decode_attn with a caller-owned workspace (device memory of at least
 * q8kv_workspace_bytes() bytes, 256-byte aligned, any contents). The call allocates
 * nothing. Calls that overlap on the GPU must not share a workspace. */
q8kv_status q8kv_decode_attn_ws(float *out, const float *q, const int8_t *k_blocks,
                                const int8_t *v_blocks, const float *kscale,
                                const float *vscale, const int32_t *block_table,
                                const int32_t *seq_lens, int B, int n_q_heads, int n_kv_heads,
                                int head_dim, int kv_block_size, int max_blocks_per_seq,
                                int num_kv_blocks, float scale, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/* Size of the scratch array that q8kv_decode_attn_static uses (12 MiB per device). */
#define Q8KV_STATIC_SCRATCH_BYTES (12u * 1024u * 1024u)

/*
 * Same as q8kv_decode_attn, but the call allocates no device memory at all: the partial
 * results of the split sequences live in a fixed device array inside the library,
 * Q8KV_STATIC_SCRATCH_BYTES bytes per device. None of the source pages has a counterpart
 * to this entry point; they describe the computation, not where its scratch lives.
 *
 * Who needs it: a caller that must not allocate while it serves requests. Examples are a
 * server whose pool allocator hands out all device memory at start-up (a cudaMalloc then
 * fails, or takes memory the pool had counted on), and a timed decode step that cannot
 * afford the device-wide synchronisation of cudaFree or the latency of a first cudaMalloc.
 * q8kv_decode_attn allocates on its first call per device and again when a shape needs a
 * larger workspace; q8kv_decode_attn_ws makes the caller allocate one.
 *
 * Set-up: the first call on each device (with that device current) looks up the array's
 * address (cudaGetSymbolAddress) and the kernels' attributes; later calls reuse them.
 * Make that first call before any stream capture begins.
 *
 * Initial state: nothing in the array needs to start at zero. Every call's decode kernel
 * writes the partial results (2 slots per CTA) that the same call's combine kernel reads,
 * and the combine reads no other slot.
 *
 * Races: every call on one device uses the same array. Two calls that may run at the
 * same time on the GPU (different streams with no ordering between them, or threads
 * issuing to different streams) corrupt each other's results. Order them on one stream,
 * or use q8kv_decode_attn_ws with one workspace per stream. Calls of the other entry
 * points never touch this array.
 *
 * Errors: as q8kv_decode_attn, plus Q8KV_ERR_WORKSPACE (and nothing enqueued) when the
 * shape needs more than Q8KV_STATIC_SCRATCH_BYTES, i.e. when q8kv_workspace_bytes() for
 * it is larger. On a 148-SM B200 that happens when one tile covers more than 80 query
 * heads (a tile holds up to 8 KV heads and all their query heads): n_q_heads 128 with
 * n_kv_heads 8 or 1 is rejected, 64 with 8 fits.
 */
q8kv_status q8kv_decode_attn_static(float *out, const float *q, const int8_t *k_blocks,
                                    const int8_t *v_blocks, const float *kscale,
                                    const float *vscale, const int32_t *block_table,
                                    const int32_t *seq_lens, int B, int n_q_heads,
                                    int n_kv_heads, int head_dim, int kv_block_size,
                                    int max_blocks_per_seq, int num_kv_blocks, float scale,
                                    cudaStream_t stream);

/*
 * KV-cache write: quantise n_tokens new K rows and V rows per KV head and store them, with
 * their scales, at the given physical slots of the pools the decode entry points read.
 *
 * Quantisation of each (token, KV head) row of head_dim values, for K and V alike (the
 * walk-through's cache keeps one scale per (token, KV head), kernel signature comment, and
 * forms the dequantisation multiplier as scale * 1/127, section 2 part 2; the quantiser is
 * step 1's, taken over the whole row), in IEEE fp32:
 *   amax = max|x| (1 when below 1e-6), scale = amax * fl(1/127),
 *   code = clamp(round-half-to-even(x * fl(127 / amax)), -127, 127)
 * kscale / vscale receive `scale` (the multiplier value = code * scale of the layouts
 * above). A row holding an infinity or a NaN is stored as codes 0 with a NaN scale and
 * sets Q8KV_DEVERR_NONFINITE.
 *
 * Placement (beaiera.top "deepseek-attention-div64", "Top-K index global mapping"):
 * token i goes to slot s = slot_mapping[i] = block * kv_block_size + offset; row h lands at
 * k_blocks[s][h][:] with its scale at kscale[s][h] (the same for V). A negative slot marks
 * padding: the token is skipped. A slot >= num_kv_blocks * kv_block_size is skipped and
 * sets Q8KV_DEVERR_SLOT. Slots must be distinct within one call (two tokens naming one
 * slot race; which one lands is unspecified).
 *
 *   k_blocks, v_blocks, kscale, vscale: the pools (layouts above), written in place
 *   k_new, v_new  fp32; row (i, h) starts at element i * token_stride + h * head_dim
 *                 (16-byte aligned)
 *   slot_mapping  int64 [n_tokens]
 *   n_tokens      >= 0 (0: nothing is enqueued, and k_new, v_new, slot_mapping may be null)
 *   head_dim      64, 128 or 256 (other multiples of 32: Q8KV_ERR_UNSUPPORTED)
 *   token_stride  floats between consecutive tokens' rows (0 = n_kv_heads * head_dim;
 *                 otherwise >= that and a multiple of 4, e.g. the row stride of a fused
 *                 QKV projection)
 * One kernel launch, asynchronous on `stream`; it may be scheduled while the previous
 * kernel on the stream drains and waits for it before reading anything (programmatic
 * dependent launch), and a decode call enqueued after it sees the written rows.
 */
q8kv_status q8kv_cache_write(int8_t *k_blocks, int8_t *v_blocks, float *kscale, float *vscale,
                             const float *k_new, const float *v_new,
                             const int64_t *slot_mapping, int n_tokens, int n_kv_heads,
                             int head_dim, int kv_block_size, int num_kv_blocks,
                             long long token_stride, cudaStream_t stream);

/*
 * KV-cache write in the q4_0 format (llama.cpp's q4_0 blocks, one of the quantised KV-cache
 * types of the llama.cpp change on baguaai.com's FlashAttention page), into the pools
 * q8kv_decode_attn_q4 reads: every (token, KV head) row of K and of V is quantised per
 * 32-channel block, in IEEE fp32 with every operation rounded on its own:
 *   m = the value of largest magnitude, sign kept (the first one on ties; +0 for an
 *       all-zero block), d = m / -8, id = d != 0 ? 1 / d : 0,
 *   code = min(15, trunc(x * id + 8.5))  (0..15; value = (code - 8) * d)
 * d is stored as binary16 (round to nearest even; beyond 65504 it becomes infinity, as in
 * the format). Codes are packed two per byte, channel 2i in the low nibble of byte i. A block
 * holding an infinity or a NaN is stored as codes 8 with a NaN scale (0x7e00) and sets
 * Q8KV_DEVERR_NONFINITE (a decode over it returns NaN); the row's other blocks are
 * quantised as usual.
 *
 *   k4_blocks, v4_blocks  uint8 [num_kv_blocks][kv_block_size][n_kv_heads][head_dim / 2],
 *                         16-byte aligned, written in place
 *   kd, vd                binary16 bits [num_kv_blocks][kv_block_size][n_kv_heads]
 *                         [head_dim / 32], 8-byte aligned, written in place
 *   k_new, v_new, slot_mapping, n_tokens, token_stride: as q8kv_cache_write (the same slot
 *                         rules: negative = padding, skipped; past the pool = skipped with
 *                         Q8KV_DEVERR_SLOT; distinct slots within one call)
 *   head_dim              64, 128 or 256 (the q4_0 decode reads head_dim 128)
 * One kernel launch, asynchronous on `stream`, programmatic dependent launch as
 * q8kv_cache_write.
 */
q8kv_status q8kv_cache_write_q4(uint8_t *k4_blocks, uint8_t *v4_blocks, uint16_t *kd,
                                uint16_t *vd, const float *k_new, const float *v_new,
                                const int64_t *slot_mapping, int n_tokens, int n_kv_heads,
                                int head_dim, int kv_block_size, int num_kv_blocks,
                                long long token_stride, cudaStream_t stream);

/*
 * QUEST-style per-block K metadata (CANN quest_prefill_metadata guide, xdnf.cn/news/235188):
 * for every request r, KV block j < ceil(seq_lens[r] / kv_block_size) and KV head h, the
 * per-channel maximum and minimum of the dequantised K (code * kscale, one fp32 product)
 * over the block's tokens (the last block: only its tokens < seq_lens[r]). A metadata block
 * holds kv_block_size rows, one per KV block: KV block j of request r is row
 * j % kv_block_size of physical metadata block meta_block_table[r][j / kv_block_size].
 * The rows of a request's last metadata block after its last KV block are set to zero in
 * both arrays; metadata blocks no request uses are not touched. QUEST bounds q . k over a
 * block from these two vectors to choose the blocks a decode step reads.
 *
 *   maxblocks, minblocks  fp32 [num_meta_blocks][kv_block_size][n_kv_heads][head_dim],
 *                         16-byte aligned, written
 *   k_blocks, kscale      the K pool and its scales (layouts above); v is not read
 *   block_table, seq_lens as for decode
 *   meta_block_table      int32 [B][max_meta_blocks_per_seq]
 *   head_dim              128
 * Device-side checks: a seq_len outside [0, max_blocks_per_seq * kv_block_size] is clamped
 * (Q8KV_DEVERR_SEQ_LEN); a block-table entry outside the pool skips its row
 * (Q8KV_DEVERR_BLOCK_TABLE); a metadata-table entry outside [0, num_meta_blocks), or a
 * request needing more than max_meta_blocks_per_seq metadata blocks, sets
 * Q8KV_DEVERR_META (the rows it cannot place are skipped). Host-side: Q8KV_ERR_UNSUPPORTED
 * for head_dim != 128, or when max_blocks_per_seq, num_kv_blocks, num_meta_blocks or
 * max_meta_blocks_per_seq times kv_block_size reaches 2^31. One kernel launch, asynchronous
 * on `stream`, programmatic dependent launch as the other kernels.
 */
q8kv_status q8kv_quest_metadata(float *maxblocks, float *minblocks, const int8_t *k_blocks,
                                const float *kscale, const int32_t *block_table,
                                const int32_t *seq_lens, const int32_t *meta_block_table, int B,
                                int n_kv_heads, int head_dim, int kv_block_size,
                                int max_blocks_per_seq, int max_meta_blocks_per_seq,
                                int num_kv_blocks, int num_meta_blocks, cudaStream_t stream);

/*
 * Decode attention that also gives the log-sum-exp of every row: lse[b][i][h] = ln sum_t
 * exp(s_t) over the tokens that query i of sequence b sees (-inf, with a zero output row, when
 * it sees none), fp32 [B][n_queries][n_q_heads]. `out` is what q8kv_decode_attn_multi gives
 * (n_queries = 1: q8kv_decode_attn), bit for bit except where that runs on tcgen05: there this
 * call's softmax weights carry three more bits. The statistics are what q8kv_attn_mass needs,
 * and what merges this output with attention over other tokens.
 *   workspace  NULL: the library-managed one (same rules as q8kv_decode_attn: one per device,
 *              not for calls that overlap). Otherwise caller-owned as in q8kv_decode_attn_ws,
 *              of at least q8kv_workspace_bytes(B, n_queries * n_q_heads, n_kv_heads,
 *              head_dim) bytes; calls that may overlap, two captured graphs among them, use
 *              one each.
 * A NaN in a query row counts as zero, as in the other decode calls (it has no part in its block's
 * maximum and its code is 0); an infinity gives lse NaN and an output without meaning.
 * q8kv_attn_mass answers NaN for both. Other arguments, shapes, errors and asynchrony as
 * q8kv_decode_attn_multi.
 */
q8kv_status q8kv_decode_attn_lse(float *out, float *lse, const float *q, const int8_t *k_blocks,
                                 const int8_t *v_blocks, const float *kscale,
                                 const float *vscale, const int32_t *block_table,
                                 const int32_t *seq_lens, int B, int n_queries, int n_q_heads,
                                 int n_kv_heads, int head_dim, int kv_block_size,
                                 int max_blocks_per_seq, int num_kv_blocks, float scale,
                                 void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Accumulated attention weights: for every sequence b, KV head kv and token t < seq_lens[b]
 *   mass[b][kv][t] = decay * mass[b][kv][t]
 *                    + sum over the head's query rows (i, h) of exp(s_t - lse[b][i][h]),
 * h over the group of kv, with the scores s_t of the decode (same int8 query, same block dots,
 * query i seeing tokens t < seq_lens[b] - (n_queries - 1 - i)) and the statistics that
 * q8kv_decode_attn_lse gave for the same q and cache. Summed over a sequence's tokens, one call
 * adds n_queries * n_q_heads / n_kv_heads per KV head (less the rows that see nothing).
 *
 *   mass   fp32 [B][n_kv_heads][max_blocks_per_seq * kv_block_size], updated in place; entries
 *          at or past seq_lens[b] are not written and have no effect (a new token's entry starts
 *          at whatever the caller left: zero it, or let q8kv_evict do so)
 *   decay  in [0, 1]: 1 adds up, less forgets, 0 writes the weights without reading mass
 *   lse    fp32 [B][n_queries][n_q_heads]
 * Tokens of a block whose table entry is outside the pool keep their mass
 * (Q8KV_DEVERR_BLOCK_TABLE); a seq_len out of range is clamped (Q8KV_DEVERR_SEQ_LEN). A query
 * row that holds an infinity or a NaN, or whose lse is NaN or +inf, gives NaN to every token that
 * it sees; a scale of NaN, which the cache writes give to such rows, gives NaN to its token.
 * Supported: head_dim 128; kv_block_size a power of two in [16, 256]; n_queries *
 * n_q_heads / n_kv_heads <= 128; n_kv_heads <= 4096; B <= 16384. One kernel launch, no
 * workspace, asynchronous on `stream`, programmatic dependent launch as the other kernels.
 */
q8kv_status q8kv_attn_mass(float *mass, const float *q, const float *lse, const int8_t *k_blocks,
                           const float *kscale, const int32_t *block_table,
                           const int32_t *seq_lens, int B, int n_queries, int n_q_heads,
                           int n_kv_heads, int head_dim, int kv_block_size,
                           int max_blocks_per_seq, int num_kv_blocks, float scale, float decay,
                           cudaStream_t stream);

/*
 * Eviction by accumulated attention weight: bound every sequence to `keep` tokens per KV head
 * and move the kept rows to new blocks. With L = seq_lens[b], and per KV head:
 *   L <= keep: every token is kept; otherwise the first `sink` tokens, the last `recent` ones,
 *   and the keep - sink - recent of largest mass among those between (NaN counts as the lowest
 *   value, equal masses go to the lowest position).
 * The kept tokens keep their order: the j-th becomes token j of the sequence under
 * new_block_table, with its K and V codes, scales and mass. Heads choose independently (a
 * decode sums over tokens, so token j of one head need not be token j of another). Afterwards
 * decode with new_block_table and new_lens, and append new tokens at position new_lens[b].
 *
 *   k_blocks, v_blocks, kscale, vscale  the pools; rows under new_block_table are written
 *   mass            fp32 [B][n_kv_heads][max_blocks_per_seq * kv_block_size], read
 *   new_mass        fp32 [B][n_kv_heads][new_max_blocks_per_seq * kv_block_size], another
 *                   buffer: the kept tokens' masses, then zeros
 *   kept            int32 [B][n_kv_heads][keep]: old position of each kept token, then -1
 *   new_lens        int32 [B], another buffer than seq_lens: min(seq_lens[b], keep)
 *   new_block_table int32 [B][new_max_blocks_per_seq]; ceil(min(L, keep) / kv_block_size)
 *                   entries are read. Its blocks must not be read by any sequence of the call
 *                   (fresh ones from the allocator; old blocks, which other sequences may
 *                   share, are left as they are), except that a sequence with L <= keep may
 *                   name its own old blocks in order and then moves nothing
 *   keep            >= 1, sink >= 0, recent >= 0, sink + recent <= keep <=
 *                   new_max_blocks_per_seq * kv_block_size
 * A table entry outside the pool skips the rows that need it (Q8KV_DEVERR_BLOCK_TABLE); a
 * seq_len out of range is clamped (Q8KV_DEVERR_SEQ_LEN). Supported: head_dim 64, 128 or 256;
 * B <= 16384; any kv_block_size; keep * n_kv_heads < 2^30. Two kernel launches, no workspace,
 * asynchronous on `stream`, programmatic dependent launch as the other kernels.
 */
q8kv_status q8kv_evict(int8_t *k_blocks, int8_t *v_blocks, float *kscale, float *vscale,
                       float *new_mass, int32_t *kept, int32_t *new_lens, const float *mass,
                       const int32_t *block_table, const int32_t *seq_lens,
                       const int32_t *new_block_table, int B, int n_kv_heads, int head_dim,
                       int kv_block_size, int max_blocks_per_seq, int new_max_blocks_per_seq,
                       int num_kv_blocks, int keep, int sink, int recent, cudaStream_t stream);

/*
 * Rotary positions with one to four axes, fused with the q8 cache write: rotate the new tokens'
 * query and key rows, write the queries as the fp32 rows the decode reads, and quantise and
 * store the rotated keys and the values as q8kv_cache_write does.
 *
 * Pair p of a rotated row (p < rotary_dim / 2) is channels (p, p + rotary_dim / 2), or (2p,
 * 2p + 1) with `adjacent`; channels past rotary_dim pass through. With (c, s) = cos_sin[pos][p],
 * cos_sin[pos][rotary_dim / 2 + p] at pos = positions[pair_axis[p]][i],
 *   x1' = x1 c - x2 s,  x2' = x2 c + x1 s,
 * products and sums rounded to fp32 one by one. Images and video give their tokens a time, a
 * height and a width position; text gives all axes the same.
 *
 *   q_out          fp32 [n_tokens][n_q_heads][head_dim]; may be q_new itself (fp32 rows without
 *                  gaps), otherwise must not overlap the inputs
 *   q_new, k_new, v_new  rows of type dtype (16-byte aligned): (i, h) starts at element
 *                  i * token_stride + h * head_dim
 *   slot_mapping   int64 [n_tokens], the slot rules of q8kv_cache_write (negative: K and V of
 *                  the token are skipped; its query is still rotated)
 *   positions      int32 [n_axes][n_tokens]; one outside [0, max_position) is clamped and sets
 *                  Q8KV_DEVERR_POSITION
 *   cos_sin        fp32 [max_position][rotary_dim], 16-byte aligned: the cosines of the pairs,
 *                  then their sines
 *   pair_axis      host array of rotary_dim / 2 bytes, each < n_axes, read before the call
 *                  returns; NULL: every pair on axis 0
 *   rotary_dim     a multiple of 8, at most head_dim
 *   q_token_stride, kv_token_stride  elements between tokens (0 = no gap; otherwise at least
 *                  the row and a multiple of 16 bytes)
 * n_tokens 0 enqueues nothing. Supported: head_dim 64, 128 or 256; 1 to 4 axes. One kernel
 * launch, asynchronous on `stream`, programmatic dependent launch as q8kv_cache_write.
 */
q8kv_status q8kv_rope_cache_write(float *q_out, int8_t *k_blocks, int8_t *v_blocks,
                                  float *kscale, float *vscale, const void *q_new,
                                  const void *k_new, const void *v_new,
                                  const int64_t *slot_mapping, const int32_t *positions,
                                  const float *cos_sin, const uint8_t *pair_axis, int n_tokens,
                                  int n_axes, int n_q_heads, int n_kv_heads, int head_dim,
                                  int rotary_dim, int adjacent, int max_position,
                                  q8kv_dtype dtype, int kv_block_size, int num_kv_blocks,
                                  long long q_token_stride, long long kv_token_stride,
                                  cudaStream_t stream);

/*
 * Verification of drafted tokens (speculative sampling) against the target's probabilities,
 * from given random numbers: the step after q8kv_decode_attn_multi scored the drafts. Sequence
 * b with n = n_drafts[b] drafts x_0 .. x_(n-1) accepts draft i while
 *   uniforms[b][i] * draft_probs[b][i][x_i] < target_probs[b][i][x_i].
 * At the first refusal i it draws from max(target_probs[b][i] - draft_probs[b][i], 0), or from
 * target_probs[b][i] when that is zero everywhere; with every draft accepted, from
 * target_probs[b][n]. The draw is the smallest token whose running sum of weights (lowest token
 * first) exceeds uniforms[b][max_drafts] times their total. Products and sums are fp64. Rows
 * need not sum to one; a weight that is not above zero (NaN too) counts as zero.
 *
 *   n_accepted    int32 [B]
 *   tokens        int32 [B][max_drafts + 1]: the accepted drafts, the drawn token, then -1
 *   target_probs  dtype [B][max_drafts + 1] rows of vocab, target_stride elements apart
 *   draft_probs   dtype [B][max_drafts] rows of weights >= 0, draft_stride elements apart; NULL
 *                 for drafts without probabilities (each is then certain: accepted while
 *                 uniform < target's, and a refusal draws from the target's row without it)
 *   draft_tokens  int32 [B][max_drafts] (may be NULL when max_drafts is 0)
 *   n_drafts      int32 [B], or NULL: max_drafts each
 *   uniforms      fp32 [B][max_drafts + 1], in [0, 1)
 *   strides       0 = vocab; otherwise at least vocab (rows that start on 16 bytes are read
 *                 with 16-byte loads)
 * A draft count out of range is clamped, a draft token outside the vocabulary is refused, and a
 * row without a positive finite total gives token -1; each sets Q8KV_DEVERR_PROBS. B = 0 enqueues
 * nothing. Supported: max_drafts <= 1024, vocab <= 2^30, B <= 2^24. One kernel launch (clusters of
 * up to 8 blocks), no workspace, asynchronous on `stream`, programmatic dependent launch.
 */
q8kv_status q8kv_verify_draft(int32_t *n_accepted, int32_t *tokens, const void *target_probs,
                              const void *draft_probs, const int32_t *draft_tokens,
                              const int32_t *n_drafts, const float *uniforms, int B,
                              int max_drafts, int vocab, long long target_stride,
                              long long draft_stride, q8kv_dtype dtype, cudaStream_t stream);

/* Debug: the Q quantisation alone (step 1) on n_rows rows of head_dim fp32 values
 * (head_dim a multiple of 32). qi int8 [n_rows][head_dim], qsc fp32
 * [n_rows][head_dim / 32]. Uses the device routine the decode kernel uses. */
q8kv_status q8kv_debug_quantize_q(int8_t *qi, float *qsc, const float *q, int n_rows,
                                  int head_dim, cudaStream_t stream);

/* Debug: the int32 block dot products of step 2, produced by the decode kernel itself
 * (same staging and tensor-core fragments) and written out as
 * dots int32 [B][n_q_heads][max_seq_len][head_dim / 32]; entries of tokens at or past
 * seq_lens[b] are left untouched. max_seq_len must be >= every seq_lens[b]. Also writes
 * `out` like q8kv_decode_attn. Uses the library-managed workspace. */
q8kv_status q8kv_debug_block_dots(int32_t *dots, int max_seq_len, float *out, const float *q,
                                  const int8_t *k_blocks, const int8_t *v_blocks,
                                  const float *kscale, const float *vscale,
                                  const int32_t *block_table, const int32_t *seq_lens, int B,
                                  int n_q_heads, int n_kv_heads, int head_dim,
                                  int kv_block_size, int max_blocks_per_seq, int num_kv_blocks,
                                  float scale, cudaStream_t stream);

/* Debug: q8kv_decode_attn with one pipeline fault injected, to exercise the bounded waits.
 * The producer warp of CTA stall_cta never arrives on, and never loads into, the stage of
 * that CTA's second tile (its first when it has only one), so nothing is in flight for that
 * stage and its phase never completes. That CTA's waits give up after limit_ns
 * (1e3 <= limit_ns <= 1e9; other CTAs keep the normal limit of one second): its consumer
 * warps stop computing and its producer stops issuing, Q8KV_DEVERR_TIMEOUT is set, and the
 * kernel returns normally, so the context stays usable. Rows whose split segments that CTA
 * contributes to are undefined; all other rows are what q8kv_decode_attn gives. A CTA
 * index past the grid injects nothing. Library-managed workspace, asynchronous. Returns
 * Q8KV_ERR_INVALID_ARG for stall_cta < 0 or limit_ns out of range. */
q8kv_status q8kv_debug_stall_pipeline(float *out, const float *q, const int8_t *k_blocks,
                                      const int8_t *v_blocks, const float *kscale,
                                      const float *vscale, const int32_t *block_table,
                                      const int32_t *seq_lens, int B, int n_q_heads,
                                      int n_kv_heads, int head_dim, int kv_block_size,
                                      int max_blocks_per_seq, int num_kv_blocks, float scale,
                                      int stall_cta, unsigned long long limit_ns,
                                      cudaStream_t stream);

/* Read (and, if clear != 0, reset) the device-side error word of the current device.
 * Synchronises the device. */
q8kv_status q8kv_device_errors(unsigned *flags, int clear);

/* Static description of a status code. */
const char *q8kv_status_string(q8kv_status status);

/* The cudaError_t of the last failing CUDA call made by this library on this thread
 * (0 if none). */
int q8kv_last_cuda_error(void);

/* Library ABI version (major * 100 + minor). */
int q8kv_version(void);

#ifdef __cplusplus
}
#endif
#endif
