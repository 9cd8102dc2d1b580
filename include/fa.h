/*
 * fa.h -- C ABI of libfa.so: exact scaled-dot-product attention on GB300
 * (sm_103a), computed tile by tile with the online-softmax recurrence.
 *
 * What every call computes (the pages' definition; the kernels never write an
 * S x S matrix to device memory):
 *
 *   S = scale * Q K^T,  P = softmax(S) over the visible keys of each row,
 *   O = P V,  LSE_i = ln sum_j exp(S_ij)  (natural log, scale included)
 *
 *   -- "Flash Attention" history page, sections 1.1 (the attention formula),
 *      1.2 (running max m, denominator l, rescaled output), 1.3 (tiles live on
 *      chip and are discarded), 2.1 (parallelism over the query sequence,
 *      causal tiles skipped); FlashAttention_01 page, "online softmax
 *      derivation" (m, l, unnormalised u, divide once at the end; mask before
 *      the max; an explicit rule for rows with no visible key) and "backward
 *      recomputation" (save one logsumexp per row, rebuild P from it).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  * Tensors are bf16 (IEEE bfloat16 bit patterns), contiguous, layout
 *    [B, H, S, d] with d innermost.  Q, O, dO, dQ: [B, Hq, Sq, d].
 *    K, V, dK, dV: [B, Hkv, Sk, d].  LSE: fp32 [B, Hq, Sq].
 *  * Every pointer is a DEVICE pointer of the current CUDA device, 16-byte
 *    aligned.  The caller owns every buffer and the stream; the library never
 *    allocates, frees or retains device memory (scratch comes from the
 *    caller's workspace argument).
 *  * Grouped K/V heads (GQA/MQA, "Flash Attention" practitioner page 2.3):
 *    Hq % Hkv == 0 and query head h reads KV head h / (Hq / Hkv).
 *  * Visibility of key j to query row i of batch row b:
 *        k_start[b] <= j < k_end[b]   and   (causal == 0  or  j <= i + Sk - Sq)
 *    The causal rule is aligned to the bottom-right corner (for Sq == Sk it is
 *    the usual lower triangle).  k_start / k_end are optional device int32[B]
 *    arrays (NULL means 0 and Sk); values outside [0, Sk] are clamped.
 *  * A row with no visible key gets O = 0 and LSE = -inf, and contributes zero
 *    gradient; no -inf - (-inf) is ever evaluated.
 *  * d (head dimension) must be 64 or 128 (FA_ERR_UNSUPPORTED otherwise).
 *  * scale must be finite and >= 0 (FA_ERR_INVALID_ARG otherwise); scale 0
 *    gives uniform weights over the visible keys.
 *  * Calls are asynchronous: they validate, enqueue kernels on `stream` and
 *    return.  A validation failure returns before any launch and writes
 *    nothing.  Launch failures return FA_ERR_CUDA.  fa_last_error_detail()
 *    gives a one-line reason for the last non-OK status of the calling thread.
 *  * Device-side pipeline waits are bounded (1 s).  A wait that runs out
 *    records FA_ERR_TIMEOUT in a device status word and the kernel returns
 *    early; fa_device_status() reads (and optionally clears) that word.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* bad size, null or misaligned pointer, Hq % Hkv != 0 */
  FA_ERR_UNSUPPORTED = 2, /* head dimension other than 64 or 128, or no sm_103a device */
  FA_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than the *_workspace_size query */
  FA_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed */
  FA_ERR_TIMEOUT = 5      /* a device pipeline wait ran out (see fa_device_status) */
} fa_status;

/*
 * Forward pass.  O = softmax(scale * Q K^T) V over visible keys, and per-row
 * LSE (natural log, scale included).  lse may be NULL when the caller does
 * not need it; the backward needs it.
 *   q [B,Hq,Sq,d], k/v [B,Hkv,Sk,d], o [B,Hq,Sq,d] (written), lse [B,Hq,Sq]
 *   (written).  B, Hq, Hkv, Sq, Sk >= 1.
 * Follows: "Flash Attention" history page 1.2-1.3 and 2.1; FlashAttention_01
 * page, online-softmax derivation and the large-score worked example.
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                 int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                 const int32_t* k_start, const int32_t* k_end, cudaStream_t stream);

/* Bytes of device workspace fa_bwd needs: an fp32 dQ accumulator
   [B,Hq,Sq,d] and the fp32 row terms D_i = rowsum(dO * O) [B,Hq,Sq]. */
size_t fa_bwd_workspace_size(int B, int Hq, int Sq, int d);

/*
 * Backward pass by recomputation.  Given the forward's inputs, its bf16
 * output o and its lse, and the upstream gradient dout:
 *   D_i = rowsum(dO * O),  P = exp(scale * Q K^T - LSE) on visible entries,
 *   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - D),
 *   dQ = scale * dS K,  dK = scale * dS^T Q,
 * with dK/dV of a KV head summed over its query heads.  dq [B,Hq,Sq,d],
 * dk/dv [B,Hkv,Sk,d] are written (bf16).  The mask arguments, causal flag and
 * scale must be the ones the forward used.  workspace must hold at least
 * fa_bwd_workspace_size(B, Hq, Sq, d) bytes; its contents on entry are
 * ignored and on return are unspecified.
 * Follows: FlashAttention_01 page, "why the backward can recompute" and the
 * chain-rule section (dV, dP, dS, dQ = dS K / sqrt(d), dK = dS^T Q / sqrt(d)).
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Sq,
                 int Sk, int d, int causal, float scale, const int32_t* k_start,
                 const int32_t* k_end, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream);

/*
 * Per-key boolean masks and packed ragged ("varlen") sequences.
 * Follows: FlashAttention_01 page, "interface and implementation constraints"
 * (masks and ragged layouts are part of the kernel contract; statistics cover
 * only valid rows; a ragged layout tells logical row numbers from packed ones).
 *
 * Key mask bits: key j of mask row r is visible iff bit (j % 32) of word
 * bits[r * fa_key_mask_words(Sk) + j / 32] is set.  A hidden key is treated
 * like a key outside [k_start, k_end): it gets weight 0 in the softmax and
 * zero dK/dV.  A row that sees no key gives O = 0, LSE = -inf.  The bits
 * buffer is caller-owned device memory, 16-byte aligned; bits past Sk are
 * ignored.  fa_pack_key_mask builds it from one byte per key.
 */
size_t fa_key_mask_words(int Sk); /* uint32 words per mask row: 4 * ceil(Sk / 128) */

/* bits[rows][fa_key_mask_words(Sk)] = packed (mask[rows][Sk] != 0); device
   buffers, asynchronous on stream.  mask needs no alignment. */
fa_status fa_pack_key_mask(const uint8_t* mask, uint32_t* bits, int rows, int Sk,
                           cudaStream_t stream);

/* fa_fwd with a per-(batch row, key) mask: key_mask_bits has B mask rows
   (NULL = no mask, exactly fa_fwd). */
fa_status fa_fwd_masked(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                        const int32_t* k_start, const int32_t* k_end,
                        const uint32_t* key_mask_bits, cudaStream_t stream);

/* fa_bwd with the same key mask the forward used (NULL = exactly fa_bwd). */
fa_status fa_bwd_masked(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                        int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                        const int32_t* k_start, const int32_t* k_end,
                        const uint32_t* key_mask_bits, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/*
 * Packed ragged forward.  nseq sequences are concatenated along the row
 * axis: q/o [Hq, total_q, d], k/v [Hkv, total_k, d], lse [Hq, total_q].
 * Sequence s owns packed query rows [cu_seqlens_q[s], cu_seqlens_q[s+1]) and
 * packed keys [cu_seqlens_k[s], cu_seqlens_k[s+1]) and attends only within
 * itself; the causal rule is bottom-right within the sequence (logical key
 * j' <= logical row i' + Sk_s - Sq_s).  cu_seqlens_* are device int32[nseq+1],
 * non-decreasing, from 0 to total_q / total_k (values are clamped to
 * [0, total]).  max_seqlen_q/k are host upper bounds on the sequences'
 * query and key counts; they size the grid, and rows or keys of a sequence
 * past them are not processed (their outputs are left unwritten).  Packed
 * rows or keys that belong to no sequence are not written either.
 * Rows of a sequence without keys get O = 0 and LSE = -inf.  key_mask_bits
 * (nullable) is one mask row over the packed keys.
 */
fa_status fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                        const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int nseq,
                        int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int Hq,
                        int Hkv, int d, int causal, float scale, const uint32_t* key_mask_bits,
                        cudaStream_t stream);

/*
 * Packed ragged backward, the layout and arguments of fa_fwd_varlen: dq
 * [Hq, total_q, d] and dk/dv [Hkv, total_k, d] are written; workspace holds
 * fa_bwd_workspace_size(1, Hq, total_q, d) bytes.
 */
fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv,
                        const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int nseq,
                        int max_seqlen_q, int max_seqlen_k, int total_q, int total_k, int Hq,
                        int Hkv, int d, int causal, float scale, const uint32_t* key_mask_bits,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Dropout on the attention weights, with the random mapping fixed as part of
 * the forward/backward contract (FlashAttention_01 page, "why the backward
 * can recompute", "interface and implementation constraints" and "training
 * configuration and misuse boundaries": recomputation needs the same mask,
 * statistics, scale and dropout mapping).
 *   O_i = sum_j P_ij * keep_ij * r * v_j,  P the undropped softmax;
 *   LSE is the undropped one (what the backward needs to rebuild P).
 *   keep_ij <=> the 16-bit half (j mod 2) (0: low, 1: high) of word
 *   ((j mod 8) / 2) of Philox4x32-10 (Salmon et al., SC 2011) at counter
 *   (j / 8, i, b * Hq + h, offset) under key (seed & 0xffffffff, seed >> 32)
 *   is >= thr = floor(dropout_p * 2^16); i is the query row and j the key
 *   index within batch row b.  The keep probability is thus 1 - thr / 2^16,
 *   and kept weights are scaled by its reciprocal r = 2^16 / (2^16 - thr),
 *   so E[keep_ij * r] = 1 exactly (p below 2^-16: thr = 0, nothing is dropped
 *   and r = 1).
 * dropout_p must lie in [0, 1) (0 = no dropout); the backward must get the
 * forward's dropout_p, seed and offset.  Otherwise these are fa_fwd_masked /
 * fa_bwd_masked (key_mask_bits may be NULL).
 */
fa_status fa_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                         int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                         const int32_t* k_start, const int32_t* k_end,
                         const uint32_t* key_mask_bits, float dropout_p,
                         unsigned long long seed, unsigned int offset, cudaStream_t stream);

fa_status fa_bwd_dropout(const void* q, const void* k, const void* v, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                         int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                         const int32_t* k_start, const int32_t* k_end,
                         const uint32_t* key_mask_bits, float dropout_p,
                         unsigned long long seed, unsigned int offset, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/*
 * FP8 forward ("Flash Attention" history page 2.2: FA3 runs attention in
 * FP8).  q [B,Hq,Sq,128], k [B,Hkv,Sk,128] and vt [B,Hkv,128,Sk] (V
 * transposed: each head's value matrix stored head-dimension-major) hold
 * e4m3 (OCP FP8 E4M3, bias 7, max 448) bytes; the attention is computed for
 * Q = q_descale * q, K = k_descale * k, V = v_descale * v with the bf16
 * forward's visibility rules (key interval, causal, GQA).  o (bf16
 * [B,Hq,Sq,128]) and lse are written as by fa_fwd.  Both matrix products run
 * in FP8 with fp32 accumulation; the softmax weights are rounded to e4m3 for
 * the second product (O is normalised by the sum of the rounded weights, the
 * LSE uses the exact fp32 sum).  d must be 128 (FA_ERR_UNSUPPORTED
 * otherwise), Sk a multiple of 16, and the descale factors finite and > 0.
 */
fa_status fa_fwd_fp8(const void* q, const void* k, const void* vt, void* o, float* lse, int B,
                     int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                     float q_descale, float k_descale, float v_descale, const int32_t* k_start,
                     const int32_t* k_end, cudaStream_t stream);

/* Bytes of device workspace fa_decode needs for a cache of Sk_max positions:
   per (b, query head, split) partial outputs and logsumexps. */
size_t fa_decode_workspace_size(int B, int Hq, int Sk_max, int d);

/*
 * Single-query decode (Sq = 1) over a padded KV cache with split-KV and a
 * logsumexp merge.  q [B,Hq,1,d]; k_cache/v_cache [B,Hkv,Sk_max,d] of which
 * the first seqlens_k[b] positions of batch row b are valid; seqlens_k is a
 * device int32[B] (values clamped to [0, Sk_max]; 0 gives O = 0, LSE = -inf).
 * o [B,Hq,1,d] is written; lse [B,Hq] is written when not NULL.  The split
 * plan depends only on (B, Hq, Hkv, Sk_max, d), never on the values in
 * seqlens_k, so the call never reads device memory on the host.
 * workspace must hold fa_decode_workspace_size(B, Hq, Sk_max, d) bytes.
 * Follows: FlashAttention_01 page, "performance validation" (prefill with
 * Sq = Sk and decode with Sq = 1 are measured separately); the merge applies
 * the rescale rule of the "Flash Attention" history page 1.2 to whole
 * per-chunk states.
 */
fa_status fa_decode(const void* q, const void* k_cache, const void* v_cache, void* o,
                    float* lse, const int32_t* seqlens_k, int B, int Hq, int Hkv, int Sk_max,
                    int d, float scale, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream);

/* Size of the scratch array built into the library for fa_decode_noalloc. */
#define FA_DECODE_NOALLOC_MAX_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * fa_decode without a workspace argument, for callers that cannot allocate
 * device memory: callers whose interface only carries the input and output
 * buffers (a fixed operator or plugin signature with no workspace slot), and
 * callers that run where allocating is not possible or not wanted (a host
 * framework that owns all device memory through its own pool, or a
 * latency-critical loop that cannot pay for cudaMalloc and the device
 * synchronisation it implies).  The pages have no counterpart: it is an
 * interface variant of fa_decode, with the same arguments, results and errors
 * minus workspace/workspace_bytes.
 *
 * Scratch comes from one array of FA_DECODE_NOALLOC_MAX_SCRATCH_BYTES (64 MiB)
 * compiled into the library; each GPU on which it is used keeps that array
 * until the process exits.  No device memory is allocated by the call.
 *   - Problems whose fa_decode_workspace_size(B, Hq, Sk_max, d) exceeds the
 *     array are rejected with FA_ERR_WORKSPACE before any device work.
 *   - The first call on a device looks up the array's device address (with
 *     that device current); make that first call before any stream capture.
 *     The address is tied to the device's CUDA context: after cudaDeviceReset
 *     (or with another context current) the next call looks it up again, so
 *     that call, too, should come before any capture.
 *   - All calls on a device share the array: calls that can overlap on the GPU
 *     (different streams without ordering between them) race and corrupt each
 *     other's results.  Calls ordered on one stream are safe; nothing in the
 *     array needs to start at zero.
 */
fa_status fa_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, void* o,
                            float* lse, const int32_t* seqlens_k, int B, int Hq, int Hkv,
                            int Sk_max, int d, float scale, cudaStream_t stream);

/*
 * Paged 8-bit KV cache
 * ====================
 * Serving from a cache of pages: fa_kv_assign hands out pages and slots,
 * fa_kv_write_fp8 quantises new keys and values into them, fa_select_blocks
 * picks the blocks a query attends, fa_decode_paged_fp8 is the attention of
 * the last Sq tokens, and fa_kv_read_fp8 gives cached keys and values back as
 * packed bf16 for fa_fwd_varlen (a prompt chunk over a cached prefix).
 *
 *  * k_cache, v_cache: e4m3 bytes (OCP FP8 E4M3) [num_pages, Hkv, page_size, d],
 *    16-byte aligned; page_size is 16, 32, 64 or 128, d is 64 or 128.
 *  * k_scale, v_scale: fp32 [num_pages, Hkv], one per (page, KV head); a cached
 *    value is code * scale.  Scales lie in [2^-100, 2^119].
 *  * k_bounds: int8 [num_pages, Hkv, 2, d], 16-byte aligned: per channel the
 *    largest (row 0) and the smallest (row 1) key code of the page in units of 4
 *    codes, rounded outwards (up and down).  Only fa_select_blocks reads it.
 *  * block_table: int32 [B, max_blocks]; entry (b, i) is the page of positions
 *    [i * page_size, (i + 1) * page_size) of request b.  Entries outside
 *    [0, num_pages) mark absent pages: their keys are treated as hidden.
 *    Requests may share pages that nothing writes to.
 *  * Page and slot offsets are computed in 64 bits; a cache may be larger than
 *    2^32 bytes.  Packed tokens per call: at most 2^30.
 *  * A workspace belongs to one call at a time: calls that can overlap on the GPU
 *    (on streams without ordering between them, or in graphs that replay side by
 *    side) need workspaces of their own.  A call that writes pages must be
 *    ordered before the calls that read them, as any producer and consumer.
 */

/*
 * Block tables and slot maps from request lengths, in one launch.  Request b
 * holds seqlens[b] tokens and gets newlens[b] more (negative values count as 0).
 * With have = ceil(seqlens / page_size) and full = ceil((seqlens + newlens) /
 * page_size) it takes the next full - have pages of free_pages[0, n_free), in
 * request order, for its table entries [have, full).
 *   block_table [B,max_blocks]  entries [have, full) written, the rest kept
 *   slot_map int64 [total_new]  slot of every packed new token, page * page_size +
 *                               offset; -1 for a token without one and for the
 *                               packed rows behind the last request
 *   cu_new int32 [B+1]          offsets of the requests' packed new tokens
 *   seqlens_out int32 [B]       lengths after the call
 *   cu_seqlens_k int32 [B+1]    their prefix sums (fa_fwd_varlen's cu_seqlens_k)
 *   n_used int32 [1]            pages taken off the front of free_pages
 * A request is refused, whole, when it would need more than max_blocks blocks,
 * when its packed tokens end behind total_new, or when its pages end behind
 * n_free: it takes no page, its slots are -1 and its seqlens_out is seqlens.  The
 * pages a request without room in the free list asked for count as taken for
 * the requests after it.  Offsets saturate at 2^31 - 1.
 * Outputs must not overlap seqlens, newlens or free_pages.  slot_map needs
 * 8-byte alignment, the others 4-byte; free_pages may be NULL when n_free is 0
 * and slot_map when total_new is 0.
 */
fa_status fa_kv_assign(const int32_t* seqlens, const int32_t* newlens, int B, int page_size,
                       int32_t* block_table, int max_blocks, const int32_t* free_pages, int n_free,
                       int64_t* slot_map, int total_new, int32_t* cu_new, int32_t* seqlens_out,
                       int32_t* cu_seqlens_k, int32_t* n_used, cudaStream_t stream);

/*
 * Quantising write of n_tokens new keys and values.  k, v: bf16, element (head,
 * token, channel) at head * stride_h + token * stride_t + channel (strides in
 * elements, >= 0, multiples of 8; base pointers 16-byte aligned), so packed
 * [Hkv, n, d] and token-major [n, Hkv, d] inputs are both read in place.
 * slot_map int64 [n_tokens] as fa_kv_assign writes it; tokens with a slot
 * outside [0, num_pages * page_size) are skipped.
 * Consecutive tokens in consecutive slots of one page form a run; the run's
 * first offset n is the number of tokens the page holds before it.  Per head,
 * separately for K and V:
 *   s_tok = 2^e, e the smallest with amax <= 448 * 2^e over the run's finite
 *           values, e in [-100, 119]
 *   s     = max(s_old, s_tok) if n > 0 (s_old: the page's scale), else s_tok
 *   new codes  = x / s (in fp32) rounded to the nearest e4m3 value (ties to even),
 *                at most +-448; an infinity becomes +-448, a NaN the NaN code
 *   held codes [0, n) = code * s_old / s, rounded again, if s > s_old
 *   k_bounds (NULL: not kept) = the run's bounds, merged for n > 0 with the old
 *                ones times s_old / s, rounded outwards (for a ratio that is no power
 *                of two also rounded like the codes first: they enclose them either
 *                way); NaN codes count as 0
 * A scale only grows within a page until its offset 0 is written again.  With
 * power-of-two scales a held code changes only where it becomes subnormal.
 * Codes behind the run are left as they were.  A page must not appear in two
 * runs of one call (its content is unspecified then); fa_kv_assign never
 * makes such a slot map.
 */
fa_status fa_kv_write_fp8(const void* k, const void* v, long long k_stride_h, long long k_stride_t,
                          long long v_stride_h, long long v_stride_t, const int64_t* slot_map,
                          int n_tokens, void* k_cache, void* v_cache, float* k_scale,
                          float* v_scale, int8_t* k_bounds, int num_pages, int Hkv, int page_size,
                          int d, cudaStream_t stream);

/*
 * Dequantising read: packed bf16 k, v [Hkv, total_k, d], where sequence s owns rows
 * [cu_seqlens_k[s], cu_seqlens_k[s+1]) (device int32[nseq+1], non-decreasing) and
 * row cu_seqlens_k[s] + i is its position i: code * scale rounded to bf16 (exact
 * for power-of-two scales within bf16's range).  Positions without a page give
 * zeros; rows of no sequence are left as they were.
 */
fa_status fa_kv_read_fp8(const void* k_cache, const void* v_cache, const float* k_scale,
                         const float* v_scale, const int32_t* block_table,
                         const int32_t* cu_seqlens_k, void* k, void* v, int nseq, int max_blocks,
                         int num_pages, int total_k, int Hkv, int page_size, int d,
                         cudaStream_t stream);

/* Bytes of device workspace fa_select_blocks needs: a 32-bit key per block. */
size_t fa_select_blocks_workspace_size(int B, int Hkv, int max_blocks);

/*
 * Block selection: for each request and KV head the k_blocks blocks with the
 * largest score, an upper bound of the block's scores for 8-bit queries:
 *   q8_i = rint(q_i / 2^e), |q8_i| <= 127, e the smallest with amax |q| <= 127 * 2^e,
 *          e in [-100, 119], for each query row
 *   score = max over the Hq / Hkv * Sq query rows of the KV head of
 *           k_scale * 2^(e+2) * sum_i max(q8_i * bounds_i,0 , q8_i * bounds_i,1)
 * The sum is an exact integer and is multiplied by k_scale, then by 2^(e+2), in
 * fp32.  The first n_first and last n_last blocks of a request are always taken
 * (n_first + n_last <= k_blocks).  Equal scores: the lower block.  Blocks without
 * a page and NaN scores rank last.
 *   q bf16 [B,Hq,Sq,d]; seqlens_k int32 [B] (clamped to [0, max_blocks*page_size]);
 *   B * Hkv at most 65535
 *   sel int32 [B,Hkv,k_blocks]: block indices, ascending, then -1
 *   n_sel int32 [B,Hkv]: min(k_blocks, ceil(seqlens_k / page_size))
 */
fa_status fa_select_blocks(const void* q, const int8_t* k_bounds, const float* k_scale,
                           const int32_t* block_table, const int32_t* seqlens_k, int32_t* sel,
                           int32_t* n_sel, int B, int Hq, int Hkv, int Sq, int num_pages,
                           int max_blocks, int page_size, int d, int k_blocks, int n_first,
                           int n_last, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

/* Bytes of device workspace fa_decode_paged_fp8 needs (independent of the
   lengths and of the cache's size). */
size_t fa_decode_paged_fp8_workspace_size(int B, int Hq, int Hkv, int Sq, int d);

/*
 * Attention of the last Sq tokens of each request over the paged cache:
 * q, o bf16 [B,Hq,Sq,d], lse fp32 [B,Hq,Sq] (NULL when not needed).  Request b has
 * seqlens_k[b] keys (device int32[B], clamped to [0, max_blocks * page_size]; they
 * include the Sq tokens), and key j is visible to row i iff
 *   j <= i + seqlens_k[b] - Sq   (bottom-right causal; Sq = 1: every key)
 * and, when sel and n_sel are given (both or neither), j's block is one of
 * sel[b,hk,0 .. n_sel[b,hk]) of its KV head (int32 [B,Hkv,max_sel]; n_sel is
 * clamped to [0, max_sel]; entries outside the request's blocks are ignored, a
 * block listed twice counts twice).  Rows that see no key give O = 0, LSE = -inf.
 * What the pages hold behind a request's last key is never used.  A key that
 * holds NaN makes the rows that see it NaN, and no others.
 * V scales may lie as far apart as their range allows.  Weights are rounded to 11 bits
 * where they multiply the values; a weight * V scale below 2^-23 of the largest that its
 * row sees is off by at most 2^-34 of that largest.
 * Scores are formed in fp32: where k_scale * max|q| * scale * 448 * d passes 2^126, rows may
 * become NaN.  B * Hkv is at most 65535 (FA_ERR_INVALID_ARG; split larger batches).
 * Any Sq is accepted; for prompts, fa_kv_read_fp8 with fa_fwd_varlen is the
 * faster path (the rows of a KV head are served 32 at a time here).
 */
fa_status fa_decode_paged_fp8(const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale,
                              const int32_t* block_table, const int32_t* seqlens_k,
                              const int32_t* sel, const int32_t* n_sel, void* o, float* lse, int B,
                              int Hq, int Hkv, int Sq, int num_pages, int max_blocks, int max_sel,
                              int page_size, int d, float scale, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/*
 * Between a projection and the scores
 * ===================================
 * fa_qk_norm_rope takes a projection's rows [token][head][channel] and gives the head-major
 * tensors that the attention reads, in one pass: a norm of every query and key head vector, the
 * position rotation, and for serving the rows of a padded cache.
 *
 * A strided view [B, S, H, d] of bf16 with contiguous channels: element (b, s, h, c) at
 * ptr[b * stride_b + s * stride_t + h * stride_h + c].  ptr is 16-byte aligned; strides are in
 * elements, >= 0 and multiples of 8 (those of dimensions of one element do not matter).
 */
typedef struct {
  void* ptr;
  long long stride_b, stride_t, stride_h;
} fa_heads;

/*
 * For each token and head vector x of q and k (d is 64 or 128):
 *   u = x * r * (weight + weight_offset),  r = 1 / sqrt(mean(x^2) + eps);  u = x without a weight
 *   y = u with its first rot_dim channels turned: pair i, (a, b) -> (a c_i - b s_i, b c_i + a s_i),
 *       c_i, s_i = cos, sin of position[freq_axis[i]] * inv_freq[i] (radians); the pairs are channels
 *       (i, i + rot_dim / 2), or (2 i, 2 i + 1) when interleaved != 0
 * and v is copied.  Arithmetic is fp32, y is rounded to bf16 once; angles are reduced exactly, to 2^-31 turns
 * for every position and frequency, and c_i, s_i off by less than 2^-19.
 *   q view [B,S,Hq,d]; k, v views [B,S,Hkv,d]; v and v_out are NULL together
 *   q_weight, k_weight  bf16 [d], 16-byte aligned, or NULL: no norm
 *   positions  int32 [n_axes,B,S], any value; NULL: the token's row (below) on every axis
 *   inv_freq   fp32 [rot_dim / 2], finite, magnitudes below 2^24; rot_dim is 0 or a multiple of 16 up to d
 *   freq_axis  uint8 [rot_dim / 2] or NULL (axis 0); frequencies of axes >= n_axes do not turn
 *   q_out [B,Hq,S,d]; k_out, v_out [B,Hkv,S_out,d]: token s of batch row b is row
 *   row_start[b] + s (device int32[B]; NULL: 0).  Rows outside [0, S_out) are skipped, rows of no
 *   token are left as they were.
 * Outputs must not overlap inputs.
 */
fa_status fa_qk_norm_rope(const fa_heads* q, const fa_heads* k, const fa_heads* v, void* q_out,
                          void* k_out, void* v_out, const int32_t* row_start, int S_out,
                          const void* q_weight, const void* k_weight, float weight_offset,
                          float eps, const int32_t* positions, int n_axes, const float* inv_freq,
                          const uint8_t* freq_axis, int rot_dim, int interleaved, int B, int S,
                          int Hq, int Hkv, int d, cudaStream_t stream);

/* Bytes of device workspace fa_qk_norm_rope_bwd needs when a weight's gradient is asked for. */
size_t fa_qk_norm_rope_bwd_workspace_size(int d);

/*
 * Gradients of fa_qk_norm_rope without row_start.  q, k: the forward's inputs (only read, and only
 * needed, where there is a weight); dq_out [B,Hq,S,d], dk_out, dv_out [B,Hkv,S,d]: gradients of its
 * outputs (dv_out and dv NULL together).  Written: the views dq [B,S,Hq,d], dk, dv [B,S,Hkv,d],
 * none of which may overlap itself or another, and dq_weight, dk_weight fp32 [d] (NULL: not
 * wanted).  With g = dy turned back and a = g * (weight + weight_offset):
 *   dx = r * (a - x r mean(a x r)),   dweight = sum over tokens and heads of g x r
 * Sums are fp32 in a fixed order: the same call gives the same bits.
 */
fa_status fa_qk_norm_rope_bwd(const fa_heads* q, const fa_heads* k, const void* dq_out,
                              const void* dk_out, const void* dv_out, const fa_heads* dq,
                              const fa_heads* dk, const fa_heads* dv, float* dq_weight,
                              float* dk_weight, const void* q_weight, const void* k_weight,
                              float weight_offset, float eps, const int32_t* positions,
                              int n_axes, const float* inv_freq, const uint8_t* freq_axis,
                              int rot_dim, int interleaved, int B, int S, int Hq, int Hkv, int d,
                              void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Row intervals: documents, prefixes, windows
 * ===========================================
 * The visible keys of a row are an interval [lo, hi).  fa_row_bounds writes the intervals of the
 * usual masks (a caller may as well write its own), fa_mask_plan turns intervals into the tile
 * plan that fa_fwd_scored and fa_bwd_scored skip by.  Both are made once for all layers of a step.
 *
 * Row i of batch row b is position p = i + Sk - Sq of Sk.
 *   document [start, end): [0, Sk), or with cu_docs (device int32[n_docs + 1], non-decreasing offsets
 *            into the B * Sk flattened positions) the document that holds b * Sk + p, cut at the
 *            batch row's ends; positions of no document (and p < 0) see nothing
 *   causal:  hi = min(end, max(p + 1, start + prefix)), else hi = end
 *   window:  lo = max(start, p - window + 1) and, not causal, hi = min(hi, p + window); 0: none
 * prefix (device int32[n_docs], or int32[B] without cu_docs; NULL: 0) is the number of keys at a
 * document's start that all of its rows see (from its offset in cu_docs, or from the batch row's
 * start where that cuts it); negative: padding, whose rows see nothing.
 * row_lo, row_hi int32 [B,Sq] are written; rows without keys get 0, 0.
 * B * Sq and B * Sk must be below 2^31, B at most 65535.
 */
fa_status fa_row_bounds(const int32_t* cu_docs, const int32_t* prefix, int n_docs, int32_t* row_lo,
                        int32_t* row_hi, int B, int Sq, int Sk, int causal, int window,
                        cudaStream_t stream);

/* Bytes of a mask plan: 8 per row, some 45 per 128 rows and 60 per 128 keys. */
size_t fa_mask_plan_size(int B, int Sq, int Sk);

/* The tile plan of row_lo, row_hi int32 [B,Sq] (clamped to [0, Sk]; hi <= lo: no keys) into plan
   (16-byte aligned, fa_mask_plan_size bytes), which holds all that the attention needs of them.
   Sq and Sk are at most 2^31 - 257. */
fa_status fa_mask_plan(const int32_t* row_lo, const int32_t* row_hi, int B, int Sq, int Sk,
                       void* plan, size_t plan_bytes, cudaStream_t stream);

/*
 * Capped and biased scores
 * ========================
 * fa_fwd, fa_bwd and fa_decode on scores that are capped, biased by distance and masked by row
 * intervals.  For row i of query head h at position p = i + Sk - Sq:
 *   s_ij = scale * <q_i, k_j>
 *   t_ij = softcap * tanh(s_ij / softcap)      (softcap 0: t = s)
 *   z_ij = t_ij - slopes[h] * |p - j|          (slopes NULL: z = t)
 *   O = softmax(z) V, LSE_i = ln sum_j exp(z_ij), over the keys of the row's interval in the plan
 *   (plan NULL: all) and, when causal != 0, j <= p
 * softcap is 0 or in [2^-20, 2^20]; slopes device fp32[Hq], finite, any sign (constants: no gradient).
 * plan: fa_mask_plan of the same B, Sq, Sk; plan_bytes its size.  (A plan of others, with as many bytes, is
 * refused on the device: the outputs are not computed, and fa_device_status says so.)  Rows without keys give O = 0,
 * LSE = -inf and no gradient.  What q, dout and o hold in rows without keys, and k and v in keys that no row
 * of the batch row sees (causal counted in), is never used.  A NaN in a query, or in a key or value that some row
 * sees, reaches the rows that see it.  In a key or value, it and infinities may reach O of every row of a
 * 256-row block one of whose rows sees the key, and dq of every row between the first and the last 128-row block
 * that see a key of its 128-key tile; in a query or dout between those blocks, dk and dv of the tile.
 * t is off by at most 4e-7 of its value or 2^-22 * min(softcap, 256), whichever is larger.
 */
fa_status fa_fwd_scored(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                        float softcap, const float* slopes, const void* plan, size_t plan_bytes,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Bytes of device workspace (16-byte aligned) with which fa_fwd_scored splits the keys of few rows over
   the GPU; 0: such sizes are not split.  Without it (NULL) the call gives the same, later. */
size_t fa_fwd_scored_workspace_size(int B, int Hq, int Hkv, int Sq, int Sk, int d);

/* Its backward pass, by recomputation as fa_bwd: with P = exp(z - LSE) and dz = P * (dP - D),
   ds = dz * (1 - (t / softcap)^2), dQ = scale * ds K, dK = scale * ds^T Q, dV = P^T dO.  The scores'
   arguments are the forward's; workspace holds fa_bwd_workspace_size(B, Hq, Sq, d) bytes.  Where
   fa_bwd_scored_workspace_size is more and as much is there, the queries of few keys are split over
   the GPU: the same gradients, sooner.  In ds, weights below 2^-29 count in steps of 2^-39. */
fa_status fa_bwd_scored(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                        int Hq, int Hkv, int Sq, int Sk, int d, int causal, float scale,
                        float softcap, const float* slopes, const void* plan, size_t plan_bytes,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);

size_t fa_bwd_scored_workspace_size(int B, int Hq, int Hkv, int Sq, int Sk, int d);

/* Bytes of device workspace fa_decode_scored needs; 0: none, and its workspace may be NULL. */
size_t fa_decode_scored_workspace_size(int B, int Hq, int Hkv, int Sk_max, int d, int window);

/*
 * fa_decode on such scores.  The query of batch row b is position n - 1, n = seqlens_k[b] (clamped
 * to [0, Sk_max]); it sees the keys [max(0, k_start[b], n - window), n) (k_start device int32[B] or
 * NULL: 0; window 0: none).  No other key is used.  Grid and workspace depend on the arguments,
 * never on the values in seqlens_k and k_start.  A NaN reaches the batch rows that see it and no
 * others.  B * Hq must be below 2^31.
 */
fa_status fa_decode_scored(const void* q, const void* k_cache, const void* v_cache, void* o,
                           float* lse, const int32_t* seqlens_k, const int32_t* k_start, int B,
                           int Hq, int Hkv, int Sk_max, int d, float scale, float softcap,
                           const float* slopes, int window, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/* Reads the device status words of the current device (this synchronises the
   device).  Returns FA_OK, FA_ERR_TIMEOUT, or FA_ERR_INVALID_ARG where a kernel
   was given a mask plan of other sizes (code 4); *code_out (may be NULL) receives
   the raw word (low 16 bits: error code, high 16 bits: wait site).  When
   clear != 0 the words are reset to 0 afterwards. */
fa_status fa_device_status(unsigned int* code_out, int clear);

/* Self-test of the bounded device waits behind FA_ERR_TIMEOUT.  Enqueues on
   `stream` one small kernel whose two warps wait, with the helpers every
   attention kernel uses, on barriers that nothing arrives on: the first
   wait runs out after its 1 s limit, records the timeout at wait site 0x7e
   in the device status word and raises the kernel's abort flag; the second
   gives up on seeing the flag (no second record).  The kernel then returns
   normally and the context stays usable.  result is a device array of two
   unsigned ints (16-byte aligned), set to 1 for each wait that reported
   failure.  Afterwards fa_device_status() returns FA_ERR_TIMEOUT with the
   word 0x007e0001.  Takes about one second; for tests of the failure path
   only. */
fa_status fa_selftest_wait_timeout(unsigned int* result, cudaStream_t stream);

/* Profiling hook (the pages ask that a timing confirm which kernel actually
   ran).  start/stop are cudaEvent_t handles created by the caller.  The next
   fa_fwd, fa_bwd, fa_decode (their variants too) or fa_decode_paged_fp8 call made on this host thread records `start`
   on its stream right before its main kernel (fa_fwd: the attention kernel;
   fa_bwd: the key-tile kernel, not the preprocess or dQ-convert kernels;
   fa_decode and fa_decode_paged_fp8: the split partial kernel, not the merge)
   and `stop` right after it, then the hook disarms itself.  Passing NULL for both disarms it.  The
   events are not owned by the library. */
fa_status fa_profile_next_launch(cudaEvent_t start, cudaEvent_t stop);

/* Static text for a status code. */
const char* fa_status_string(fa_status s);

/* One-line detail of the last non-OK status returned on the calling thread
   ("" when none). */
const char* fa_last_error_detail(void);

/* Library version string. */
const char* fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
