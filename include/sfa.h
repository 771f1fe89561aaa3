/*
 * sfa.h -- C ABI of the GB300 (sm_103a) sparse MLA decode library (libsfa.so).
 *
 * One decode step of DeepSeek-style sparse attention (SFA) over a paged MLA
 * latent KV cache, plus the online-softmax merge of per-shard (out, lse)
 * partials used by decode context parallelism (DCP).
 *
 * Conventions for every call:
 *  - Pointers marked "device" must point to memory of the current CUDA device;
 *    pointers marked "host" to host memory (pinned memory gives asynchronous
 *    copies).  The caller allocates and owns every buffer; the library never
 *    allocates, frees or keeps a pointer after a call returns, with three stated
 *    exceptions: an sfa_host_plan keeps the pointers it was created with,
 *    sfa_decode_noalloc works in a fixed device array of the library's own, and
 *    sfa_decode_host creates its helper streams and events once per device.
 *  - `stream` is a cudaStream_t passed as an opaque pointer (NULL = the legacy
 *    default stream).  Calls only enqueue work on it and return without
 *    synchronising, except sfa_last_device_status() and the host-buffer entry
 *    point's error path, which say so.
 *  - Arguments are checked on the host before anything is launched; a bad
 *    argument returns an error code and launches nothing.  Problems only the
 *    device can see (a block-table entry outside [0, num_blocks) for a selected
 *    position, a bounded wait that ran out) are recorded in a per-device status
 *    word read by sfa_last_device_status().  The offending row is skipped,
 *    never dereferenced.
 *  - Layouts are dense, row-major, with no padding between rows.
 */
#ifndef SFA_H
#define SFA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SFA_OK = 0,
  SFA_ERR_INVALID_ARG = -1,    /* null pointer, negative size, misaligned buffer, bad value   */
  SFA_ERR_UNSUPPORTED = -2,    /* valid but outside what the kernels implement (e.g. h > 128)  */
  SFA_ERR_WORKSPACE = -3,      /* workspace / staging buffer missing or too small              */
  SFA_ERR_CUDA = -4,           /* a CUDA runtime call failed (launch error, copy error)        */
  SFA_ERR_DEVICE_TIMEOUT = -5, /* a bounded device-side wait gave up (device status only)      */
  SFA_ERR_DEVICE_BAD_BLOCK = -6, /* a selected position mapped to an invalid block (device)    */
  SFA_ERR_DEVICE_NO_BLOCKS = -7 /* a step plan ran out of blocks, table or token room (device) */
} sfa_status;

typedef void *sfa_stream; /* a cudaStream_t */

#define SFA_D_QK 576     /* kv_lora_rank (512) + qk_rope_head_dim (64) */
#define SFA_D_V 512      /* kv_lora_rank: V is the latent part of the row */
#define SFA_MAX_HEADS 128
#define SFA_MAX_SPLITS 64

/*
 * sfa_decode -- sparse attention of each query token over its selected latent
 * cache rows.
 *
 * Defined by: "RFC: MsModeling 支持 Decode Context Parallel 仿真" 2.1.4.1 (paged MLA
 * latent cache [N_blk, block_size, kv_lora_rank + qk_rope_head_dim] and block
 * table), 2.1.4.2 / 2.1.4.4 (attention output plus fp32 lse [B*Q, heads]), 1.1 and
 * 2.1.1 (KV sharded along the sequence, partial (out, lse) per shard);
 * "vllm-ascend PR #18870 解读" 4.3 / 4.5 (fused QK^T -> softmax -> .V over the
 * top-2048 selected entries, latent shared by all heads); "RFC: Context Parallel
 * Modeling for DeepSeek-Style Attention" 3.6 (bf16 SFA inputs).
 *
 * For query token t = b*Q + i (0 <= i < Q) and head hh:
 *   L_t   = seq_lens[b] - (Q - 1 - i)              (token i sees one more position than i-1)
 *   entry j is used iff 0 <= topk_idx[t, j] < L_t   (anything else, e.g. -1, is padding)
 *   row   = block_table[b, p / block_size] * block_size + p % block_size
 *   s_j   = scale * dot(q[t, hh, 0:576], kv[row, 0:576])
 *   out   = softmax(s) . kv[rows, 0:512],   lse = ln sum_j exp(s_j)   (natural log)
 *   no entry used -> out = 0, lse = -inf
 * Duplicate entries count once per list entry.
 *
 * Shards (n_splits > 1, decode context parallelism on one GPU): shard r covers
 * positions [r*c, (r+1)*c) of sequence b with c = ceil(seq_lens[b] / n_splits),
 * intersected with the token's causal range; each shard is attended on its own
 * into out_part[r], lse_part[r] (empty shard -> 0, -inf).
 *
 * Arguments:
 *   q           device, bf16 [B*Q, h, 576]
 *   kv          device, bf16 [num_blocks, block_size, 576]; V = columns 0..511
 *   block_table device, int32 [B, max_blocks_per_seq]; entries for blocks a sequence
 *               does not own are never read (any value)
 *   seq_lens    device, int32 [B]: cache length of each sequence (includes the Q new tokens)
 *   topk_idx    device, int32 [B*Q, top_k]: logical positions, -1 = padding
 *   B >= 0, Q >= 1, 1 <= h <= 128, top_k >= 0, num_blocks >= 1, block_size >= 1,
 *   max_blocks_per_seq >= 1, scale finite, 1 <= n_splits <= 64
 *   out, lse    device, fp32 [B*Q, h, 512] and [B*Q, h]: the final result.  Required
 *               when n_splits == 1.  When n_splits > 1 they may be NULL (only the
 *               partials are produced); if given, the partials are also merged
 *               into them on the same stream (as sfa_lse_merge does).
 *   out_part, lse_part  device, fp32 [n_splits, B*Q, h, 512] and [n_splits, B*Q, h];
 *               required when n_splits > 1, ignored otherwise.
 *   workspace   optional device scratch, 256-byte aligned.  With at least
 *               sfa_decode_workspace_bytes(...) bytes the kernel for 33-64 heads
 *               spreads the work of more (token, shard) units than SMs evenly over
 *               the SMs; with less (or NULL) the call runs all the same, one unit per
 *               SM at a time.  Contents need no initialisation and are undefined
 *               afterwards; calls that overlap on the GPU must not share it.
 *   All float/bf16 buffers must be 16-byte aligned.
 * Returns SFA_OK, or an error code with nothing launched.
 */
sfa_status sfa_decode(const void *q, const void *kv, const int32_t *block_table,
                      const int32_t *seq_lens, const int32_t *topk_idx, int B, int Q, int h,
                      int top_k, int num_blocks, int block_size, int max_blocks_per_seq,
                      float scale, int n_splits, float *out, float *lse, float *out_part,
                      float *lse_part, void *workspace, size_t workspace_bytes,
                      sfa_stream stream);

/*
 * sfa_decode_workspace_bytes -- device scratch that lets sfa_decode balance this
 * shape over the SMs of the current device (see `workspace` above).  Nonzero only
 * when 33 <= h <= 64 and B*Q*n_splits exceeds the SM count: then 2 partial
 * results (64 x 512 fp32 and 64 (max, sum) pairs) per SM, plus one counter per
 * (token, shard) unit, each part rounded up to 256 bytes.  0 otherwise, and 0
 * while sfa_set_kernel_path selects a fixed kernel.
 */
size_t sfa_decode_workspace_bytes(int B, int Q, int h, int top_k, int n_splits);

/*
 * sfa_lse_merge -- online-softmax merge of n_splits partial results.
 *
 * Defined by: "RFC: MsModeling 支持 Decode Context Parallel 仿真" 1.1 and 2.1.1 (the
 * local online-softmax merge after the all-to-all of output and lse) and 2.1.4.3
 * (both exchanged in fp32).  For each row x:
 *   M = max_r lse_part[r, x];  lse[x] = M + ln sum_r exp(lse_part[r, x] - M)
 *   out[x, :] = sum_r exp(lse_part[r, x] - lse[x]) * out_part[r, x, :]
 *   every lse_part[r, x] = -inf  ->  out[x, :] = 0, lse[x] = -inf
 *   an lse_part[r, x] that is NaN ->  out[x, :] and lse[x] are NaN
 *
 *   out_part device fp32 [n_splits, rows, dv], lse_part device fp32 [n_splits, rows]
 *   out      device fp32 [rows, dv],           lse      device fp32 [rows]
 *   (for decode partials rows = B*Q*h: the (token, head) pairs are merged alike, so
 *   they are passed flattened rather than as separate token and head counts)
 *   1 <= n_splits <= 64, rows >= 0, dv >= 1; float buffers 16-byte aligned.
 *   out/lse must not overlap out_part/lse_part.
 */
sfa_status sfa_lse_merge(const float *out_part, const float *lse_part, int n_splits, int rows,
                         int dv, float *out, float *lse, sfa_stream stream);

/*
 * sfa_decode_ex -- sfa_decode with the two layout options of decode context
 * parallelism ("RFC: MsModeling 支持 Decode Context Parallel 仿真", 2.1.4.1):
 *
 *   interleave_size  0: shard r of n_splits is the contiguous range [r*c, (r+1)*c) of
 *                    the sequence's cache, c = ceil(seq_lens[b] / n_splits) (as in
 *                    sfa_decode).  g > 0: the sequence's positions are dealt to the
 *                    shards g at a time, as cp_kv_cache_interleave_size deals them to
 *                    the DCP ranks: shard r holds the positions p with (p / g) % n_splits
 *                    == r.  Either way each shard is clipped to the token's causal range
 *                    and the merged result is the same (up to rounding).
 *   flags            SFA_BLOCK_TABLE_PER_TOKEN: block_table is [B*Q, max_blocks_per_seq],
 *                    one row per query token (the table flattened for speculative
 *                    decoding); otherwise [B, max_blocks_per_seq], one row per sequence.
 *
 * Every other argument, and the return codes, as in sfa_decode.  interleave_size < 0 or
 * an unknown flag bit returns SFA_ERR_INVALID_ARG.
 */
#define SFA_BLOCK_TABLE_PER_TOKEN 1
sfa_status sfa_decode_ex(const void *q, const void *kv, const int32_t *block_table, const int32_t *seq_lens,
                         const int32_t *topk_idx, int B, int Q, int h, int top_k, int num_blocks, int block_size,
                         int max_blocks_per_seq, float scale, int n_splits, int interleave_size, int flags,
                         float *out, float *lse, float *out_part, float *lse_part, void *workspace,
                         size_t workspace_bytes, sfa_stream stream);

/*
 * sfa_topk -- the indexer's top-k selection: for each query token, the positions of the
 * k largest indexer scores, the list sparse attention then visits ("vllm-ascend PR
 * #18870 解读", 4.5: only the top-2048 positions chosen by the indexer are attended).
 * The pages give no formula for the scores themselves; they are an input here.
 *
 *   scores      device fp32 [B*Q, row_stride]: row t holds the scores of positions 0..S-1
 *               of token t's sequence (columns S..row_stride-1 are never read);
 *               16-byte aligned, row_stride >= S and a multiple of 4
 *   seq_lens    device int32 [B] or NULL: token t = b*Q + i chooses among the positions
 *               [0, min(S, seq_lens[b] - (Q-1-i))) (the causal range sfa_decode uses);
 *               NULL: among [0, S)
 *   topk_idx    device int32 [B*Q, k], written: the chosen positions in ascending order,
 *               then -1 where fewer than k positions are candidates -- the layout
 *               sfa_decode reads
 *
 * The positions chosen are those of the k largest scores under IEEE 754 totalOrder
 * (-0 below +0; a NaN with the sign bit clear above +inf); among equal scores the lower
 * positions are chosen first.  1 <= k; 0 <= S <= SFA_TOPK_MAX_S.
 * Returns SFA_OK, SFA_ERR_INVALID_ARG (bad sizes, stride, alignment or NULL buffers) or
 * SFA_ERR_UNSUPPORTED (S above SFA_TOPK_MAX_S); nothing is launched on an error.
 */
#define SFA_TOPK_MAX_S 262144
sfa_status sfa_topk(const float *scores, long long row_stride, const int32_t *seq_lens, int B, int Q, int S, int k,
                    int32_t *topk_idx, sfa_stream stream);

/*
 * sfa_kv_write -- the latent-cache write that precedes attention: each new token's
 * latent row (kv_lora_rank + qk_rope_head_dim = 576 bf16) is stored at the cache slot
 * slot_mapping[t] ("RFC: MsModeling 支持 Decode Context Parallel 仿真", 2.1.4.1:
 * slot_mapping [total_num_tokens] int32; 1.3: the fused pre-attention op writes the
 * KV).  A slot is block * block_size + offset, i.e. a row of the cache seen as
 * [num_blocks * block_size, 576].
 *
 *   kv            device bf16 [num_blocks, block_size, 576] (num_slots rows), written in place
 *   slot_mapping  device int32 [T]: the slot of each new token; < 0 = padding (skipped)
 *   rows          device bf16 [T, 576]: the new latent rows
 *   T >= 0, num_slots >= 0; kv and rows 16-byte aligned.
 * Two tokens naming the same slot write it concurrently: the slot ends up holding parts
 * of their rows, which parts is not defined (a slot mapping names each slot once).  A
 * slot >= num_slots writes nothing and sets SFA_ERR_DEVICE_BAD_BLOCK in
 * the device status word.  Returns SFA_OK or a host-side argument error, nothing launched.
 */
sfa_status sfa_kv_write(void *kv, long long num_slots, const int32_t *slot_mapping, const void *rows, int T,
                        sfa_stream stream);

/*
 * sfa_uv_proj -- the W_UV up-projection that follows attention in the latent space:
 *   y[t, h, v] = sum_{c < 512} out[t, h, c] * w_uv[h, c, v],   v < 128
 * (MLA attends over the 512-wide latent; W_UV, derived from kv_b_proj, takes each head's
 * output to its 128-wide value space: "RFC: Context Parallel Modeling for
 * DeepSeek-Style Attention", 3.5).  A tcgen05 contraction per (head, 64 tokens).
 *
 *   out   device fp32 [T, h, 512] (sfa_decode's out); rounded to bf16 for the tensor cores
 *   w_uv  device bf16 [h, 512, 128]
 *   y     device bf16 [T, h, 128]
 *   T >= 0, 1 <= h <= 65535; out and w_uv 16-byte aligned, y 2-byte aligned.
 * Accuracy: |y - exact| <= 2^-8 * sum_c |out[c] * w[c, v]| + 2^-8 * |exact| (bf16 inputs,
 * fp32 accumulation, bf16 result).  A bounded wait that gives up sets
 * SFA_ERR_DEVICE_TIMEOUT in the device status word.  Returns SFA_OK or a host-side error.
 */
sfa_status sfa_uv_proj(const float *out, const void *w_uv, void *y, int T, int h, sfa_stream stream);

/*
 * sfa_decode_q8 -- sfa_decode over an 8-bit latent cache.  An MLA cache has one latent
 * "head", so a scale belongs to a group of consecutive slots: the value of column c of slot
 * s is e4m3(kv8[s, c]) * scales[s / group], and with it every formula is sfa_decode's.
 *
 *   kv8         device, e4m3 bytes [num_blocks, block_size, 576]; 16-byte aligned
 *   scales      device, fp32 [num_blocks, block_size / group], in [2^-100, 2^120]
 *               (sfa_kv_write_q8 writes powers of two; any others are taken as they are), or 0
 *               where nothing was written: such a group's rows are rows of zeros
 *   group       slots per scale: >= 1, divides block_size
 *   interleave_size, flags  as in sfa_decode_ex; SFA_OUT_BF16: `out` is bf16 [B*Q, h, 512]
 *               (16-byte aligned) instead of fp32.  lse and the shard partials are fp32.
 *   num_blocks * block_size <= INT_MAX (SFA_ERR_UNSUPPORTED above).
 * Everything else, and the return codes, as in sfa_decode_ex.
 *
 * Accuracy: lse carries fp32 rounding only (q is exact to 2^-22 of its head's largest value);
 * out, whatever its type, carries the rounding of the softmax weights, and then that of its own
 * type.  With w_j the weight of row j times its scale, w_j is off by at most 2^-8 w_j, or by 2^-21
 * of the largest w of the 32 used rows that it is taken with, where this is more; so out differs by
 * at most 2^-8 sum_j w_j |kv8_j|, and by about 2^-10 of its norm (as by sfa_decode's bf16 weights),
 * also where one row has most of the weight.  Rows whose w is below 2^-110 of the largest may count
 * as none, in lse too.  A NaN or infinity in a head of q makes that head's out and lse NaN, merged
 * or not; so does a score that is none.
 * sfa_set_kernel_path(1) selects a CUDA-core kernel here too, any other path the tensor cores'.
 */
#define SFA_OUT_BF16 2
sfa_status sfa_decode_q8(const void *q, const void *kv8, const float *scales, int group,
                         const int32_t *block_table, const int32_t *seq_lens, const int32_t *topk_idx, int B, int Q,
                         int h, int top_k, int num_blocks, int block_size, int max_blocks_per_seq, float scale,
                         int n_splits, int interleave_size, int flags, void *out, float *lse, float *out_part,
                         float *lse_part, sfa_stream stream);

/*
 * sfa_kv_write_q8 -- sfa_kv_write into the 8-bit latent cache sfa_decode_q8 reads.
 *
 * For each group G of `group` slots that slot_mapping names:
 *   before = 0 if the call writes G's first slot (the group starts anew), else scales[G]
 *            (taken as 0 unless positive and finite)
 *   after  = max(before, 2^k over the call's rows of G), 2^k the least power of two with
 *            amax / 2^k <= 448, -100 <= k <= 120, amax the row's largest finite magnitude
 *   the call's rows are stored as e4m3(x / after), rounded to nearest even; if 0 < before <
 *   after, G's other rows are stored again as e4m3(value * before / after); scales[G] = after
 * An infinity is stored as NaN (e4m3 has none); NaN stays NaN.
 *
 *   kv8           device, e4m3 bytes [num_slots, 576], in place; 16-byte aligned
 *   scales        device, fp32 [num_slots / group], in place
 *   num_slots     a multiple of group; 1 <= group <= SFA_Q8_MAX_WRITE_GROUP
 *   slot_mapping  device int32 [T]; < 0 = padding; a slot >= num_slots writes nothing and sets
 *                 SFA_ERR_DEVICE_BAD_BLOCK in the device status word
 *   rows          device bf16 [T, 576]; 16-byte aligned
 *   workspace     device, sfa_kv_write_q8_workspace_bytes(num_slots, group) bytes, 16-byte
 *                 aligned (none for group 1; SFA_ERR_WORKSPACE when missing or too small).  It
 *                 belongs to one cache, is zero before the first call and is left zero by every
 *                 call; calls on the same cache must not overlap.
 * A slot named twice ends up holding parts of its rows (as sfa_kv_write's); the rest of the
 * group is unaffected.
 */
#define SFA_Q8_MAX_WRITE_GROUP 64
size_t sfa_kv_write_q8_workspace_bytes(long long num_slots, int group);
sfa_status sfa_kv_write_q8(void *kv8, float *scales, long long num_slots, int group, const int32_t *slot_mapping,
                           const void *rows, int T, void *workspace, size_t workspace_bytes, sfa_stream stream);

/*
 * sfa_step_plan -- block tables and slot maps of one step from request lengths, on the GPU
 * ("RFC: MsModeling 支持 Decode Context Parallel 仿真", 2.1.4.1: block_table and slot_mapping).
 *
 * Request b has c = cached_lens[b] positions in the cache and gets n = new_lens[b] more
 * (negative lengths count as 0).  It holds ceil(c / block_size) blocks, its table's first
 * entries, and needs ceil((c + n) / block_size) of them; what it lacks is taken from
 * free_blocks, from entry *taken on, in request order.  With start_b the new tokens of the
 * requests before b, the step's token i = start_b + j is position c + j of request b.
 *
 *   cached_lens, new_lens  device int32 [B]; 0 <= B <= SFA_PLAN_MAX_REQUESTS
 *   block_table   device int32 [B, max_blocks_per_seq], in place: the entries of the blocks
 *                 taken are written, no others
 *   free_blocks   device int32 [num_free]: physical blocks no request holds
 *   taken         device int32 [1]: entries of free_blocks taken by earlier steps
 *   num_tokens    rows of positions and slot_mapping (the step's room for tokens)
 *   seq_lens      device int32 [B]: c + n                    (what sfa_decode and sfa_topk take)
 *   token_start   device int32 [B + 1]: start_b, and the number of new tokens last
 *   positions     device int32 [num_tokens]: a token's position; -1 behind the last one
 *   slot_mapping  device int32 [num_tokens]: its slot, block * block_size + position %
 *                 block_size; -1 (which the cache writes skip) behind the last one
 *   taken_out     device int32 [1]: *taken plus the blocks taken, at most num_free (or *taken)
 * The outputs must not overlap the inputs (block_table apart), so that taken and taken_out
 * change places from step to step.  A call repeated with the same inputs gives the same
 * outputs.  A table whose width, a free list whose length or a room whose size does not
 * suffice sets SFA_ERR_DEVICE_NO_BLOCKS in the device status word: table entries that find no
 * block are -1, so are the slots of the tokens in them, and tokens without room are left out.
 * A negative entry of a held or free block gives slot -1 and SFA_ERR_DEVICE_BAD_BLOCK.
 */
#define SFA_PLAN_MAX_REQUESTS 8192
sfa_status sfa_step_plan(const int32_t *cached_lens, const int32_t *new_lens, int B, int block_size,
                         int32_t *block_table, int max_blocks_per_seq, const int32_t *free_blocks, int num_free,
                         const int32_t *taken, int num_tokens, int32_t *seq_lens, int32_t *token_start,
                         int32_t *positions, int32_t *slot_mapping, int32_t *taken_out, sfa_stream stream);

/*
 * sfa_rope -- rotary positions of part of each head: the rope columns of queries (before
 * sfa_decode) and of new latent rows (before the cache write).
 *
 * For token t, head j and pair i < rot_dim / 2, with a = positions[t] * inv_freq[i]:
 *   (u, v) = mscale * (x cos a - y sin a, x sin a + y cos a)
 * where (x, y) and (u, v) are columns (2i, 2i + 1) with SFA_ROPE_INTERLEAVED, else
 * (i, i + rot_dim / 2).  SFA_ROPE_INVERSE turns by -a: the transpose, which takes the gradient
 * of (u, v) to that of (x, y).  Columns rot_dim .. width - 1 are copied.  The angle is reduced
 * to 2^-22 rad for every position and |inv_freq| < 1024; arithmetic is fp32, rounded once to the
 * type.  A frequency that is not finite gives NaN in its pair.
 *
 *   x, out      device, element (t, j, d) at t * token_stride + j * head_stride + d (strides in
 *               elements): bf16, fp16 or fp32 (dtype), T tokens of n heads.  out may be x
 *               itself (same strides); otherwise the two must not overlap.  A stride of x may be 0
 *               (a row shared by tokens or heads), of out only where it is not used.
 *   positions   device int32 [T]; < 0 = padding: that token's rows of out are left as they were,
 *               or with SFA_ROPE_COPY_PADDING are x's
 *   inv_freq    device double [rot_dim / 2]: radians a position
 *   2 <= rot_dim <= SFA_ROPE_MAX_DIM, even, <= width
 */
#define SFA_ROPE_INTERLEAVED 1
#define SFA_ROPE_INVERSE 2
#define SFA_ROPE_COPY_PADDING 8
#define SFA_ROPE_MAX_DIM 512
#define SFA_DTYPE_BF16 0
#define SFA_DTYPE_FP16 1
#define SFA_DTYPE_FP32 2
sfa_status sfa_rope(const void *x, long long x_token_stride, long long x_head_stride, void *out,
                    long long out_token_stride, long long out_head_stride, int dtype, int T, int n, int width,
                    int rot_dim, const int32_t *positions, const double *inv_freq, float mscale, int flags,
                    sfa_stream stream);

/*
 * sfa_decode_host -- one decode step whose per-step inputs and outputs live in
 * host memory, with the latent cache resident on the device (the form a serving
 * loop that keeps its cache in HBM uses).  Enqueues on `stream`: host->device
 * copies of q, block_table, seq_lens and topk_idx into `staging`, sfa_decode,
 * and device->host copies of out and lse.  The caller synchronises the stream
 * before reading out_host / lse_host.
 *
 *   q_host, block_table_host, seq_lens_host, topk_idx_host: host, layouts as in sfa_decode
 *   kv           device, as in sfa_decode
 *   out_host, lse_host: host fp32 [B*Q, h, 512] and [B*Q, h] (the merged result)
 *   staging      device scratch of at least sfa_decode_host_staging_bytes(...) bytes,
 *                256-byte aligned; holds the device copies, partials and workspace.
 * Host buffers must stay valid until the stream reaches the end of the copies.
 *
 * A batch whose out is at least 4 MiB is processed as up to 4 groups of whole
 * sequences.  Each group runs on a helper stream that the library creates once per
 * device, forked from `stream` by an event and joined back into it, so the call stays
 * ordered on `stream`.  A group's result copies overlap later groups' input copies
 * and kernels.  Calls from several host threads take turns at enqueueing (a mutex),
 * and their groups share the helper streams.  If an error is returned after some
 * groups were enqueued, that work may still run.
 */
size_t sfa_decode_host_staging_bytes(int B, int Q, int h, int top_k, int max_blocks_per_seq,
                                     int n_splits);
sfa_status sfa_decode_host(const void *q_host, const void *kv, const int32_t *block_table_host,
                           const int32_t *seq_lens_host, const int32_t *topk_idx_host, int B,
                           int Q, int h, int top_k, int num_blocks, int block_size,
                           int max_blocks_per_seq, float scale, int n_splits, float *out_host,
                           float *lse_host, void *staging, size_t staging_bytes,
                           sfa_stream stream);

/*
 * sfa_host_plan -- one sfa_decode_host step captured as a CUDA graph, for a serving loop
 * that calls it with the same buffers every step: the ~20 copies, launches and stream
 * joins of a step then cost one graph launch on the host instead of being enqueued one
 * by one (the host side of a step otherwise takes longer than the copy engines need).
 *
 *   sfa_host_plan_create  records the step exactly as sfa_decode_host with the same
 *                         arguments would enqueue it (same checks and return codes; nothing
 *                         runs).  The host buffers must be page-locked (pinned); a failed
 *                         capture returns SFA_ERR_CUDA and a NULL `plan` SFA_ERR_INVALID_ARG;
 *                         *plan is NULL unless SFA_OK.  The plan keeps the pointers: every launch copies q,
 *                         block_table, seq_lens and topk_idx in from those host buffers as
 *                         they are at that moment and writes out and lse back to theirs, so
 *                         the caller refills the inputs between launches.  The buffers must
 *                         outlive the plan; staging must not be used by anything else while
 *                         a launch may be in flight.
 *   sfa_host_plan_launch  enqueues one step on `stream` (asynchronous, like sfa_decode_host).
 *   sfa_host_plan_destroy releases the plan (NULL is ignored); no launch may be in flight.
 */
typedef struct sfa_host_plan_s *sfa_host_plan;
sfa_status sfa_host_plan_create(const void *q_host, const void *kv, const int32_t *block_table_host,
                                const int32_t *seq_lens_host, const int32_t *topk_idx_host, int B, int Q, int h,
                                int top_k, int num_blocks, int block_size, int max_blocks_per_seq, float scale,
                                int n_splits, float *out_host, float *lse_host, void *staging,
                                size_t staging_bytes, sfa_host_plan *plan);
sfa_status sfa_host_plan_launch(sfa_host_plan plan, sfa_stream stream);
void sfa_host_plan_destroy(sfa_host_plan plan);

/*
 * sfa_last_device_status -- synchronises `stream`, then returns and clears the
 * current device's status word: SFA_OK, SFA_ERR_DEVICE_TIMEOUT (a bounded wait
 * inside a kernel gave up; that kernel's outputs are undefined) or
 * SFA_ERR_DEVICE_BAD_BLOCK (a selected position's block-table entry was outside
 * [0, num_blocks); that row was skipped) or SFA_ERR_DEVICE_NO_BLOCKS (sfa_step_plan).
 * The first error since the last read is kept.  SFA_ERR_CUDA if the stream itself failed.
 */
sfa_status sfa_last_device_status(sfa_stream stream);

/*
 * sfa_decode_noalloc -- sfa_decode followed by the shard merge, for callers that
 * cannot allocate device memory.  No passage of the source pages corresponds to
 * it: it exists for deployments, not for the method.
 *
 * Some callers have no allocator: an engine that hands all free HBM to its cache
 * pool at start-up, a plugin host that passes a library only its inputs and
 * outputs, or a decode loop that cannot afford cudaMalloc's implicit device-wide
 * synchronisation.  This entry point takes only the inputs and the final out/lse
 * (layouts, alignment and argument rules as in sfa_decode; out and lse are
 * required for every n_splits) and keeps the shard partials and any workspace in
 * a fixed device array of SFA_NOALLOC_SCRATCH_BYTES that the library owns.  It
 * calls no cudaMalloc, cudaFree or other allocating routine.
 *  - Limit: a call whose partials (n_splits > 1: n_splits*B*Q*h*513 floats, each
 *    part rounded up to 256 bytes) plus workspace exceed SFA_NOALLOC_SCRATCH_BYTES
 *    returns SFA_ERR_WORKSPACE and launches nothing.
 *  - Every GPU that loads the library holds the array until the process exits.
 *  - The first call on each device looks the array's address up (with that
 *    device current); make that first call before any stream capture.
 *  - All calls share the one array: calls that overlap on the GPU (other streams,
 *    other threads) race.  Each call writes all the scratch it reads, so no
 *    clearing between calls is needed.
 *  - A call with n_splits == 1 uses no scratch and does not look the array up.
 *  - The looked-up address is cached per device for the life of the process; it is
 *    not valid after a device reset (cudaDeviceReset), so no call may follow one.
 *  - out or lse NULL returns SFA_ERR_INVALID_ARG before any other check.
 */
#define SFA_NOALLOC_SCRATCH_BYTES (72u << 20)
sfa_status sfa_decode_noalloc(const void *q, const void *kv, const int32_t *block_table,
                              const int32_t *seq_lens, const int32_t *topk_idx, int B, int Q, int h,
                              int top_k, int num_blocks, int block_size, int max_blocks_per_seq,
                              float scale, int n_splits, float *out, float *lse, sfa_stream stream);

/*
 * sfa_decode_launches -- how many kernels one sfa_decode call with these
 * arguments enqueues (merge != 0: out/lse given with n_splits > 1), and through
 * *tensor_core_path which kernel serves it: 2 = the small-head tcgen05 kernel
 * (h <= 32), 3 = the stacked-half tcgen05 kernel (33 <= h <= 64), 1 = the CTA-pair
 * tcgen05 kernel, 0 = the CUDA-core kernel.
 * tensor_core_path may be NULL.  Returns -1 for invalid arguments.
 */
int sfa_decode_launches(int B, int Q, int h, int top_k, int block_size, int n_splits, int merge,
                        int *tensor_core_path);

/*
 * sfa_set_kernel_path -- kernel family for sfa_decode calls made afterwards in
 * this process: 0 = automatic (the small-head tcgen05 kernel for h <= 32, the
 * stacked-half tcgen05 kernel for 33 <= h <= 64, the CTA-pair tcgen05 kernel
 * above), 1 = the CUDA-core kernel for every shape, 2 = the
 * CTA-pair tcgen05 kernel for every shape.  Paths 1 and 2 exist to cross-check the
 * kernels against each other.  Returns the previous setting, or -1 (and changes
 * nothing) for another value.
 */
int sfa_set_kernel_path(int path);

/* sfa_status_string -- static, human-readable name of a status code. */
const char *sfa_status_string(sfa_status s);

/*
 * sfa_set_wait_limit -- test hook for the failure path: sets the iteration cap
 * of every bounded device-side wait in kernels launched afterwards from this
 * process (0 restores the default).  With a tiny cap a wait gives up early and
 * the kernel reports SFA_ERR_DEVICE_TIMEOUT through sfa_last_device_status()
 * instead of hanging.  Returns the previous cap.
 */
long long sfa_set_wait_limit(long long iterations);

/*
 * sfa_set_stall_injection -- test hook for the failure path: with on != 0, the
 * kernels with bounded waits (the tcgen05 decode kernel and sfa_uv_proj) launched
 * afterwards from this process first wait on a barrier that nothing ever completes.
 * That wait runs out after the wait limit (sfa_set_wait_limit), the kernel records
 * SFA_ERR_DEVICE_TIMEOUT, drains its own copies and matrix operations and returns:
 * nothing faults, traps or hangs, and the context stays usable.  Returns the
 * previous setting.
 */
int sfa_set_stall_injection(int on);

#ifdef __cplusplus
}
#endif
#endif /* SFA_H */
