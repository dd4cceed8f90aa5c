/*
 * exattn -- exact scaled-dot-product attention on one GB300 (sm_103a).
 *
 * C ABI. Every entry point takes plain pointers and sizes; no C++ or
 * framework types cross it and no exception leaves it.
 *
 * Common conventions
 *   Layout   q, o: [b, sq, h, d]; k, v: [b, sk, h, d]; contiguous, d
 *            innermost (the (b, s, h, d) layout "Why FlashAttention is
 *            fast" section 2 item 2 says flash_attn_func consumes directly,
 *            so no transposes are needed). lse: [b, h, sq], fp32.
 *   Memory   q, k, v, o, lse are DEVICE pointers on the current CUDA device
 *            (attn_fwd_host alone takes host pointers), owned by the caller;
 *            the library never frees or keeps them. q, k, v, o must be
 *            16-byte aligned, lse 4-byte aligned.
 *   Streams  every compute call is asynchronous on `stream` (0 = legacy
 *            default stream). Argument errors are returned before anything
 *            is enqueued. A wait inside a kernel that exceeds its bound
 *            (about two seconds) ends the kernel early and records a device
 *            status word; attn_get_device_status() reports it.
 *   Math     O = softmax(scale * Q K^T) V row by row, with fp32 accumulation
 *            and an online (running max / running sum) softmax, so the
 *            score matrix never reaches global memory ("Why FlashAttention
 *            is fast", sections 3.1-3.3). LSE[b, h, i] = ln sum_j
 *            exp(scale * q_i . k_j), natural log, of the scaled scores.
 *            O is rounded to nearest even into the input dtype.
 *   Sizes    b, sq, sk, h >= 1; d in {16, 32, 64, 128}; scale finite
 *            (0 and negative values are accepted). b and h at most 65535.
 */
#ifndef EXATTN_H
#define EXATTN_H

#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ATTN_FP16 = 0, ATTN_BF16 = 1 } attn_dtype_t;

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,    /* null/misaligned pointer, size < 1, non-finite scale, bad dtype */
    ATTN_ERR_UNSUPPORTED = 2,    /* d outside {16, 32, 64, 128}, or a size beyond the grid limits */
    ATTN_ERR_CUDA = 3,           /* a CUDA runtime/driver call failed (launch, tensor-map encode, ...) */
    ATTN_ERR_NO_MEMORY = 4,      /* a workspace (decode partials, backward, host forward) could not be allocated */
    ATTN_ERR_DEVICE_TIMEOUT = 5  /* a kernel gave up on a bounded wait (see attn_get_device_status) */
} attn_status_t;

/*
 * Forward attention: O and LSE for every query row.
 * Defined by "Why FlashAttention is fast" section 2 item 4 (S = Q K^T * scale,
 * softmax, times V; the call flash_attn_func(q, k, v) of item 5), computed
 * tile by tile with the online softmax of section 3.3. Non-causal, no
 * dropout. dtype selects fp16 or bf16 for q, k, v and o.
 * Inputs are taken to be finite: at d = 16 with h a multiple of 4, heads
 * are computed four at a time in one tile, and a key holding an infinity
 * or a NaN also turns the rows of the other three heads of its group to
 * NaN.
 * Returns ATTN_OK once the kernel is enqueued on `stream`.
 */
attn_status_t attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                       int b, int sq, int sk, int h, int d, float scale,
                       attn_dtype_t dtype, cudaStream_t stream);

/*
 * attn_fwd with a causal mask. Causal masking is not on the pages; the mask
 * is the bottom-right-aligned one: query row i (of sq) sees key j (of sk)
 * only if j <= i + sk - sq, so with sq == sk row i sees keys 0..i, and with
 * sq < sk the last query row sees every key (new tokens appended to a
 * cache). Rows that see no key (i < sq - sk) get O = 0 and LSE = -inf.
 * Key tiles wholly past a query tile's last visible key are skipped.
 * Arguments, layouts and errors are those of attn_fwd.
 */
attn_status_t attn_fwd_causal(const void *q, const void *k, const void *v, void *o, float *lse,
                              int b, int sq, int sk, int h, int d, float scale,
                              attn_dtype_t dtype, cudaStream_t stream);

/*
 * attn_fwd (causal != 0: attn_fwd_causal) on HOST buffers: q, k, v, o, lse
 * as in attn_fwd but in host memory, 16-byte aligned; pinned memory
 * (cudaHostAlloc, cudaHostRegister) lets the copies overlap, pageable
 * memory works but its copies serialise with the host. The call runs a
 * copy / compute / copy-back pipeline: the problem is cut into chunks of
 * whole batches (at most 8), or, for one non-causal batch of at least 512
 * query rows, into at most 4 ranges of query rows that are multiples of 256
 * (K and V go first); the chunk's inputs go up on a library copy stream,
 * its forward runs on `stream`, and its O and LSE come back on a second
 * copy stream while the next chunk goes up. Results are bit-identical to
 * attn_fwd on device copies of the same inputs. Device workspace for all
 * five tensors is taken stream-ordered from the device's default memory
 * pool on `stream` and returned. The call is stream-ordered on `stream`:
 * it starts after the work already queued there, and work queued there
 * afterwards starts once every copy-back is done, so o and lse may be read
 * after `stream` is synchronised (the host buffers must stay valid until
 * then). Errors as attn_fwd; ATTN_ERR_NO_MEMORY if the workspace cannot be
 * had; ATTN_ERR_UNSUPPORTED while `stream` is being captured into a graph
 * (the pipeline runs on the library's own copy streams).
 */
attn_status_t attn_fwd_host(const void *q, const void *k, const void *v, void *o, float *lse,
                            int b, int sq, int sk, int h, int d, float scale, attn_dtype_t dtype,
                            int causal, cudaStream_t stream);

/*
 * Backward pass of attn_fwd (non-causal): dq, dk, dv from q, k, v, the
 * forward's o and lse, and the upstream gradient dout. The flash-attn timing
 * issue times a backward pass; none of the pages writes one out, so it is
 * the chain rule of the forward's definition: with P = exp(scale Q K^T - LSE),
 *     dV = P^T dO,  dP = dO V^T,  D = rowsum(dO * O),  dS = P * (dP - D),
 *     dQ = scale dS K,  dK = scale dS^T Q.
 *   q, o, dout, dq   [b, sq, h, d]; k, v, dk, dv [b, sk, h, d]; lse fp32
 *                    [b, h, sq] as written by attn_fwd; all in `dtype`
 *                    except lse, device pointers, 16-byte aligned.
 * Every output element is written. A workspace of 4 * b * h * sq bytes is
 * taken stream-ordered from the device's default memory pool and returned.
 * The key-tile (dK, dV) and query-tile (dQ) kernels run at the same time,
 * the second on a library stream forked from and joined back to `stream` by
 * events (one after the other on `stream` while it is being captured into a
 * graph); the call stays stream-ordered on `stream`. Short problems (d 16
 * or 32, sq <= 256, sk <= 160, not causal, with b * h at least half the SM
 * count or sq, sk <= 128) run one kernel instead, which finishes each
 * (batch, head) in one CTA (all of its keys in one row of S).
 * Errors as attn_fwd; ATTN_ERR_NO_MEMORY if the workspace cannot be had.
 */
attn_status_t attn_bwd(const void *q, const void *k, const void *v, const void *o,
                       const float *lse, const void *dout, void *dq, void *dk, void *dv,
                       int b, int sq, int sk, int h, int d, float scale, attn_dtype_t dtype,
                       cudaStream_t stream);

/*
 * Backward pass of attn_fwd_causal: the same chain rule with P = 0 wherever
 * the forward's bottom-right-aligned mask hides a key (key j of row i is
 * hidden when j > i + sk - sq). lse must be the one attn_fwd_causal wrote
 * (-inf for rows that see no key; those rows get dq = 0, and keys that no
 * row sees get dk = dv = 0). Tiles that the mask hides wholly are skipped.
 * Arguments, layouts, workspace and errors are those of attn_bwd.
 */
attn_status_t attn_bwd_causal(const void *q, const void *k, const void *v, const void *o,
                              const float *lse, const void *dout, void *dq, void *dk, void *dv,
                              int b, int sq, int sk, int h, int d, float scale,
                              attn_dtype_t dtype, cudaStream_t stream);

/*
 * Split-KV decode, bf16 q/k/v/o ("where is flash decoding second stage
 * (reduce) code?" issue). seqlen_k is cut into num_splits ranges of whole
 * key blocks; split i writes its own O_i and LSE_i (fp32, library
 * workspace), and the reduce forms, with the max LSE taken out first,
 *     LSE = log(sum_i exp(LSE_i)),   O = sum_i exp(LSE_i - LSE) * O_i.
 * With sq == 1 the reduce runs inside the split kernel: the split of a
 * (batch, head) that finishes last reduces it, found through arrival
 * counters (zero between calls) that the library keeps per stream together
 * with the partials (calls on a stream are ordered, so each reuses them;
 * grown stream-ordered on demand, freed by attn_release_workspace). With
 * sq > 1 the partials come from the same per-stream workspace and a second
 * kernel reduces them. While the stream is being captured into a graph, on
 * cudaStreamPerThread, and on a stream whose handle was a destroyed stream's
 * before, the partials are taken per call as below and the second kernel
 * reduces.
 * num_splits = 0 lets attn_decode_num_splits() choose; a positive value is
 * clamped to the number of key blocks. With one split the first kernel
 * writes O and LSE directly and no workspace is used. Any sq >= 1 is
 * accepted (non-causal). With sq == 1 the splits run on a CUDA-core kernel
 * (key blocks of 16 KB per tensor). With sq > 1 they run on the tensor-core
 * forward kernel, so each K/V byte is read once for all query rows of a
 * head (the issue's case of 1 to 10 new tokens); its key blocks are tiles of
 * 128 keys and a requested count is lowered so that no split is empty.
 * The per-call workspace is taken stream-ordered from
 * the device's default memory pool and returned after the reduce; it is
 * kept cached in the pool until attn_release_workspace().
 */
attn_status_t attn_decode_splitkv(const void *q, const void *k, const void *v, void *o, float *lse,
                                  int b, int sq, int sk, int h, int d, float scale,
                                  int num_splits, cudaStream_t stream);

/* attn_decode_splitkv with an explicit dtype (fp16 or bf16). */
attn_status_t attn_decode_splitkv_ex(const void *q, const void *k, const void *v, void *o, float *lse,
                                     int b, int sq, int sk, int h, int d, float scale,
                                     int num_splits, attn_dtype_t dtype, cudaStream_t stream);

/*
 * attn_decode_splitkv_ex with the causal mask of attn_fwd_causal (bottom-right
 * aligned: the sq new query rows are the last sq positions of the sk keys).
 * With sq == 1 it is attn_decode_splitkv_ex. Splits wholly past a query
 * row's last visible key contribute nothing to it (LSE_i = -inf).
 */
attn_status_t attn_decode_splitkv_causal(const void *q, const void *k, const void *v, void *o,
                                         float *lse, int b, int sq, int sk, int h, int d,
                                         float scale, int num_splits, attn_dtype_t dtype,
                                         cudaStream_t stream);

/*
 * Split-KV decode of new query rows from a paged KV cache. Paged caches are
 * not on the pages beyond a mention ("Why FlashAttention is fast", section
 * 5, item 2: FlashAttention with a paged KV cache is the standard for long
 * contexts); the layout read here is the common one.
 *   q            [b, sq, h, d] (device, 16-byte aligned): the sq new rows of
 *                each sequence (the flash-decoding issue's 1 to 10 new tokens)
 *   k_pages,
 *   v_pages      page pools [num_pages, page_size, h, d] (device, 16-byte
 *                aligned); page_size must be a multiple of 16
 *                (ATTN_ERR_UNSUPPORTED otherwise)
 *   block_table  int32 [b, max_pages_per_seq] (device): logical page p of
 *                sequence i is pool page block_table[i * max_pages_per_seq + p]
 *   seqlens_k    int32 [b] (device): keys of sequence i, 0 <= seqlens_k[i]
 *                <= max_pages_per_seq * page_size (values outside are
 *                clamped; entries of the table past a sequence's last page
 *                are not used)
 *   o, lse       [b, sq, h, d] and fp32 [b, h, sq]
 *   causal       non-zero: the bottom-right-aligned mask of attn_fwd_causal,
 *                aligned to each sequence's own key count (row r of sequence
 *                i sees key j only if j <= r + seqlens_k[i] - sq); rows that
 *                see no key get O = 0 and LSE = -inf
 * With sq == 1 the splits run on the CUDA-core kernel (pages read in boxes of
 * at most a page); with sq > 1 on the tensor-core forward kernel, whose
 * 128-key tiles are gathered from the pages and whose rows past a
 * sequence's end are zero-filled or zeroed in shared memory, so stale page
 * data (even NaN) never reaches O. The split count (num_splits = 0: the
 * heuristic of attn_decode_num_splits) is chosen for the longest allowed
 * sequence, since the lengths are only known on the device; splits past a
 * sequence's end are empty. A sequence with no key gets O = 0 and
 * LSE = -inf. The reduce, the workspace and the errors are those of
 * attn_decode_splitkv_ex.
 */
attn_status_t attn_decode_paged_ex(const void *q, const void *k_pages, const void *v_pages,
                                   const int32_t *block_table, const int32_t *seqlens_k, void *o,
                                   float *lse, int b, int sq, int h, int d, int num_pages,
                                   int page_size, int max_pages_per_seq, float scale,
                                   int num_splits, int causal, attn_dtype_t dtype,
                                   cudaStream_t stream);

/* attn_decode_paged_ex with one new row per sequence (sq = 1, q [b, 1, h, d]). */
attn_status_t attn_decode_paged(const void *q, const void *k_pages, const void *v_pages,
                                const int32_t *block_table, const int32_t *seqlens_k, void *o,
                                float *lse, int b, int h, int d, int num_pages, int page_size,
                                int max_pages_per_seq, float scale, int num_splits,
                                attn_dtype_t dtype, cudaStream_t stream);

/*
 * ---------------------------------------------------------------------
 * Packed batches and grouped heads
 *
 * Sequences of different lengths lie one behind the other in one tensor of
 * rows: sequence i holds rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1 (int32
 * [b + 1], on the device, ascending; a sequence may be empty). Rows that
 * belong to no sequence are neither used nor written. Starts past the tensor
 * are clamped to its end, and a call whose starts are out of order may leave
 * its results unwritten: they then mean nothing, but no other memory is
 * touched.
 *
 * Grouped heads: h query heads share h_kv K/V heads, h a multiple of h_kv
 * and at most 128 h_kv (ATTN_ERR_UNSUPPORTED above); query head x uses K/V
 * head x / (h / h_kv). h_kv == h gives every head its own.
 *
 * q, k and v may be slices of wider rows: q_stride, k_stride and v_stride
 * are the distances in elements from one token's row to the next, at least
 * h * d (h_kv * d) and multiples of 8; within a row, heads are d apart. o,
 * dout and the page pools are contiguous. lse is fp32 [h, total_q].
 * Values of another sequence, of rows behind the last sequence, and stale
 * values in a page never reach a result, whatever they are; a row's own keys
 * are taken to be finite. Outputs may not overlap inputs or each other.
 */

/*
 * Forward over packed sequences: for each sequence, O and LSE of attn_fwd
 * (causal != 0: attn_fwd_causal, aligned to the sequence's own lengths) over
 * its own rows.
 *   q, o    [total_q, h, d]    k, v  [total_k, h_kv, d]
 *   max_seqlen_q  the most rows a sequence has, or 0 if not known (then
 *                 taken to be total_q). It only picks the kernel's form
 *                 (results are right whatever it is): units of one 128-row
 *                 tile where every sequence fits one (has at most floor(128
 *                 / (h / h_kv)) rows), else of two. Give it where it is
 *                 known: 64 requests with a token each over up to 8192 keys,
 *                 h32 on 8, take 150 us with it and 221 without.
 * A row that sees no key gets O = 0 and LSE = -inf. total_q, total_k >= 1. More
 * than 2^29 units (rows of a K/V head, floor(128 / (h / h_kv)) at a time in each
 * sequence) are ATTN_ERR_UNSUPPORTED.
 * How the work is dealt out is decided on the device from the lengths; ranges
 * of a row tile's keys that went to several SMs are joined in a fixed order,
 * so the same call gives the same bits. Workspace (fp32 partial results, at
 * most 80 MB) and arrival counters are kept per stream and freed by
 * attn_release_workspace(); while the stream is being captured into a graph,
 * on cudaStreamPerThread, and on a stream whose handle was a destroyed
 * stream's before, they are taken from the device's memory pool for the call
 * alone. Errors as attn_fwd.
 */
attn_status_t attn_fwd_packed(const void *q, const void *k, const void *v, const int32_t *cu_seqlens_q,
                              const int32_t *cu_seqlens_k, void *o, float *lse, int b, int total_q,
                              int total_k, int max_seqlen_q, int h, int h_kv, int d, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, float scale, int causal,
                              attn_dtype_t dtype, cudaStream_t stream);

/*
 * Backward pass of attn_fwd_packed with the same sequences, heads and mask:
 * attn_bwd's chain rule, where dk and dv of a K/V head are the sums over the
 * query heads that share it.
 *   o, dout  [total_q, h, d], lse [h, total_q] as attn_fwd_packed wrote them
 *   dq       [total_q, h, d], dk, dv [total_k, h_kv, d]; they too may be slices of
 *            wider rows (dq_stride, dk_stride, dv_stride)
 * Rows of sequences are written in full (a row without a key gets dq = 0, a
 * key that no row sees dk = dv = 0), rows of no sequence not at all. No
 * atomics add into the results: the same call gives the same bits.
 * Workspace (8 h total_q bytes, and fp32 partial sums of at most 60 MB) as
 * attn_fwd_packed's. Errors as attn_fwd.
 */
attn_status_t attn_bwd_packed(const void *q, const void *k, const void *v, const void *o,
                              const float *lse, const void *dout, const int32_t *cu_seqlens_q,
                              const int32_t *cu_seqlens_k, void *dq, void *dk, void *dv, int b,
                              int total_q, int total_k, int h, int h_kv, int d, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int64_t dq_stride, int64_t dk_stride,
                              int64_t dv_stride, float scale, int causal, attn_dtype_t dtype,
                              cudaStream_t stream);

/*
 * The new tokens of each request (one, a few, or a chunk of a prompt) over a
 * paged cache: attn_decode_paged_ex for grouped heads and requests with
 * different numbers of new tokens.
 *   q, o         [total_q, h, d]: request i's rows are cu_seqlens_q[i] ..
 *                cu_seqlens_q[i + 1] - 1
 *   k_pages, v_pages  [num_pages, page_size, h_kv, d], page_size a multiple of
 *                16 (ATTN_ERR_UNSUPPORTED otherwise)
 *   block_table  int32 [b, max_pages_per_seq]; seqlens_k int32 [b]: keys of
 *                request i, the new tokens' own included (they are in the
 *                cache already: attn_paged_write); clamped as in
 *                attn_decode_paged_ex
 *   causal       the bottom-right-aligned mask: row r of request i sees key j
 *                only if j <= r + seqlens_k[i] - (request i's rows)
 *   max_seqlen_q as in attn_fwd_packed
 * A long cache is spread over as many SMs as the batch leaves it. Rows
 * without a key, workspace and errors as attn_fwd_packed.
 */
attn_status_t attn_chunk_paged(const void *q, const void *k_pages, const void *v_pages,
                               const int32_t *block_table, const int32_t *cu_seqlens_q,
                               const int32_t *seqlens_k, void *o, float *lse, int b, int total_q,
                               int max_seqlen_q, int h, int h_kv, int d, int num_pages, int page_size,
                               int max_pages_per_seq, int64_t q_stride, float scale, int causal,
                               attn_dtype_t dtype, cudaStream_t stream);

/*
 * Block tables and slot maps of one step, built on the device from request
 * lengths (nothing is read back to the host).
 *   seqlens_k    int32 [b] keys each request has in the cache; new_lens int32
 *                [b] tokens it brings now (0 is fine; negative values count
 *                as 0)
 *   free_pages   int32 [num_free]: the free pages as a stack, of which the
 *                first free_count[0] (int32 [1], clamped to 0 .. num_free) are
 *                free; pages are taken from its top, in request order
 *   block_table  int32 [b, max_pages_per_seq], updated in place: the entries of the
 *                pages a request takes are written, the others left alone
 *   cu_seqlens_q int32 [b + 1] out: first of each request's new tokens
 *   seqlens_out  int32 [b] out: keys with the new tokens, at most
 *                max_pages_per_seq * page_size
 *   slot_map     int64 [max_tokens] out: new token t's row in the pools seen
 *                as [num_pages * page_size, h_kv, d]; -1 where it has none, and
 *                behind the last token
 *   free_left    int32 [1] out: free pages left. Negative: that many were
 *                lacking; the entries concerned are -1 in the table and in
 *                slot_map, and the step must not be run as it is
 * Outputs may not overlap inputs or each other (the inputs stay as they are,
 * so a call can be repeated). Errors as attn_fwd.
 * Two things only the caller can see, and such a step must not be run as it is
 * either: a request with more keys than its table row holds (seqlens_out below
 * seqlens_k + new_lens) has no slot for those past it, and tokens past
 * max_tokens are in cu_seqlens_q but not in slot_map. free_left counts neither.
 * Pages only leave the stack here. A finished request's go back by the caller,
 * on the device too: its table's entries behind the first free_count, and the
 * count raised by as many (free_pages needs room for every page of the pool).
 */
attn_status_t attn_paged_plan(const int32_t *seqlens_k, const int32_t *new_lens, int32_t *block_table,
                              const int32_t *free_pages, const int32_t *free_count, int32_t *cu_seqlens_q,
                              int32_t *seqlens_out, int64_t *slot_map, int32_t *free_left, int b,
                              int max_pages_per_seq, int page_size, int num_free, int64_t max_tokens,
                              cudaStream_t stream);

/*
 * New K and V rows into the pages: row t of k and v (token strides k_stride
 * and v_stride, as above) goes to row slot_map[t] of the pools seen as
 * [num_pages * page_size, h_kv, d]. Slots outside the pools (-1: a padding
 * token) are skipped. The same slot twice leaves each 16 bytes of it from one
 * of the two rows. k and v may lie in the pools (rows that move), but not in
 * slots that the call writes, and the two pools may not overlap. tokens >= 1;
 * errors as attn_fwd.
 */
attn_status_t attn_paged_write(const void *k, const void *v, const int64_t *slot_map, void *k_pages,
                               void *v_pages, int64_t tokens, int h_kv, int d, int num_pages,
                               int page_size, int64_t k_stride, int64_t v_stride, attn_dtype_t dtype,
                               cudaStream_t stream);

/*
 * ---------------------------------------------------------------------
 * Rotating appends and the 4-bit cache
 *
 * attn_paged_write with the position rotation on the way: a step's queries and
 * keys are rotated by their positions, the keys and values go into the pages,
 * the queries to q_out.
 *   q, q_out     [tokens, h, d]    k, v  [tokens, h_kv, d] (token strides as
 *                above; q_out may be q itself with q's stride)
 *   cos_sin      fp32 [max_positions, rot], 16-byte aligned: row p holds the
 *                cosines of the rot / 2 angles of position p, then their sines
 *   positions    int64 [tokens]; slot_map int64 [tokens] as in attn_paged_write
 *   rot          channels of a head that turn, from the first on: a multiple of
 *                16, at most d (ATTN_ERR_UNSUPPORTED otherwise); the others pass
 *   interleaved  0: channel i < rot / 2 is paired with i + rot / 2; otherwise
 *                channels 2 i and 2 i + 1 are a pair. Pair i, (x, y), becomes
 *                (x cos_i - y sin_i, y cos_i + x sin_i), in fp32, rounded once.
 * A slot outside the pools (-1: a padding token) gets no key and value, but the
 * token's queries are rotated. For a token whose position is outside 0 ..
 * max_positions - 1 nothing is written. Channels that do not turn, and v, are
 * copied bit by bit. Outputs may not overlap inputs (but for q_out) or each
 * other; the same slot twice leaves each 16 bytes of it from one of the two
 * rows. h need not be a multiple of h_kv. Errors as attn_fwd.
 */
attn_status_t attn_paged_append(const void *q, const void *k, const void *v, const float *cos_sin,
                                const int64_t *positions, const int64_t *slot_map, void *q_out,
                                void *k_pages, void *v_pages, int64_t tokens, int64_t max_positions,
                                int rot, int interleaved, int h, int h_kv, int d, int num_pages,
                                int page_size, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                int64_t q_out_stride, attn_dtype_t dtype, cudaStream_t stream);

/*
 * A cache held in 4 bits. A pool is uint8 [num_pages, h_kv, page_bytes],
 * 16-byte aligned, page_bytes = page_size * 9 d / 16 (attn_q4_page_bytes()): a
 * page of a head holds page_size rows of d / 2 bytes of codes (channel 2 i of
 * the row in the low half of byte i), then page_size rows of d / 16 scales.
 *   code   e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6, and 8 more with the sign
 *   scale  e4m3, not negative, one for 16 neighbouring channels of a row; NaN
 *          stands for a group that held no number
 *   value  code * scale * (the tensor's scale, k_scale or v_scale)
 * page_size is a multiple of 16 (ATTN_ERR_UNSUPPORTED otherwise), k_scale and
 * v_scale lie within 2^-64 .. 2^64 (ATTN_ERR_INVALID_ARG otherwise), and every
 * call on a pool gets the same ones. Choose them so that the largest value of
 * the tensor is at most 2688 times, and typical ones some 0.1 to 1000 times,
 * its scale: a group's scale is exact to 4 bits from 2^-6 on.
 */
/* Bytes of a page of one head; 0 for a page size or head dim that is not supported. */
int64_t attn_q4_page_bytes(int page_size, int d);

/*
 * attn_paged_append into 4-bit pages. Keys (rotated, not rounded before) and
 * values: a group of 16 channels with largest magnitude m gets the scale s =
 * e4m3(m / (6 k_scale)), a channel x the code e2m1(x / (s k_scale)), each
 * rounded to the nearest with ties to even and limited to the largest value; s =
 * 0 has codes of 0 with either sign. A group that holds an infinity or a NaN
 * gets the scale NaN, so that what reads it gets NaN. The same slot twice leaves
 * codes and scales of both rows side by side. Other arguments and errors as
 * attn_paged_append.
 */
attn_status_t attn_paged_append_q4(const void *q, const void *k, const void *v, const float *cos_sin,
                                   const int64_t *positions, const int64_t *slot_map, void *q_out,
                                   void *k_pages, void *v_pages, int64_t tokens, int64_t max_positions,
                                   int rot, int interleaved, int h, int h_kv, int d, int num_pages,
                                   int page_size, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                   int64_t q_out_stride, float k_scale, float v_scale,
                                   attn_dtype_t dtype, cudaStream_t stream);

/*
 * attn_chunk_paged over a 4-bit cache: the new tokens of each request (one, a
 * few, or a chunk of a prompt) over its pages. A cached value enters the
 * products as it stands (code * scale is exact in 16 bits, the tensor's scale
 * goes into the softmax's scale and into O), so results are those of exact
 * attention over the cache's values.
 *   k_pages, v_pages  4-bit pools [num_pages, h_kv, page_bytes]; k_scale, v_scale
 *                     as attn_paged_append_q4 got them; scale * k_scale finite
 *   max_seqlen_q      as in attn_fwd_packed. Requests with few rows to a K/V head
 *                     (tokens times h / h_kv) run on a kernel of their own, the
 *                     others on one for chunks. Where this says that no request
 *                     has more than 16 rows, all of them do; in other batches of
 *                     several requests those with at most floor(8 / (h / h_kv))
 *                     tokens, or with one token where h / h_kv is 9 to 16. So give
 *                     it: 64 requests with four tokens each over up to 8192 keys,
 *                     h32 on 8, take 95 us with it and 199 without.
 * Rows of a page past a request's end may hold anything. A key with a scale of
 * NaN in K or V makes the rows that see it NaN, O and LSE, and no others. Other
 * arguments, results, workspace (at most 120 MB) and errors as attn_chunk_paged.
 */
attn_status_t attn_chunk_paged_q4(const void *q, const void *k_pages, const void *v_pages,
                                  const int32_t *block_table, const int32_t *cu_seqlens_q,
                                  const int32_t *seqlens_k, void *o, float *lse, int b, int total_q,
                                  int max_seqlen_q, int h, int h_kv, int d, int num_pages, int page_size,
                                  int max_pages_per_seq, int64_t q_stride, float scale, float k_scale,
                                  float v_scale, int causal, attn_dtype_t dtype, cudaStream_t stream);

/*
 * Rows of a 4-bit cache back in 16 bits: row slot_map[t] of the pools to row t
 * of k and v [tokens, h_kv, d] (token strides as above); zeros where the slot is
 * outside the pools. A value is rounded once where the tensor's scale is a power of
 * two; with another one the product with it is rounded to fp32 before. A slot
 * may come up several times. Errors as attn_fwd.
 */
attn_status_t attn_paged_read_q4(const void *k_pages, const void *v_pages, const int64_t *slot_map,
                                 void *k, void *v, int64_t tokens, int h_kv, int d, int num_pages,
                                 int page_size, float k_scale, float v_scale, int64_t k_stride,
                                 int64_t v_stride, attn_dtype_t dtype, cudaStream_t stream);

/*
 * Split-KV decode that allocates no device memory. The pages have no
 * counterpart: this is a library convenience, not part of the method.
 *
 * For callers that cannot call cudaMalloc once they are running: an
 * application whose device memory is all owned by its own allocator or pool,
 * code under a fixed memory budget, or real-time code that forbids
 * allocation after start-up. attn_decode_splitkv_ex takes its per-split
 * partials from the device's memory pool; this entry point keeps them in
 * one fixed scratch array of ATTN_NOALLOC_SCRATCH_BYTES compiled into the
 * library instead, and calls no cudaMalloc, cudaFree or other allocating
 * routine. Every GPU that loads the library holds that array until the
 * process exits.
 *
 * Arguments, layouts and results are those of attn_decode_splitkv_ex; the
 * caller still passes all inputs and outputs. The kernels are the same:
 * with sq == 1 the CUDA-core split kernel, with sq > 1 the tensor-core
 * forward kernel split along the keys (tiles of 128 keys, a requested count
 * lowered so that no split is empty), each followed by the combine kernel;
 * num_splits = 0 picks the count attn_decode_num_splits() reports. With more
 * than one split the partials need 4 * splits * b * sq * h * (d + 1) bytes
 * (each part rounded up to 256); a request that needs more than the array
 * holds returns ATTN_ERR_UNSUPPORTED before anything is enqueued.
 *
 * The first call on a device does a one-time set-up (it looks up the
 * array's device address; nothing is written); make that first call before
 * any stream capture. All calls share the one array, which keeps the last
 * call's contents (every split rewrites all of its partials, so none is
 * read stale): calls that overlap on the GPU, from different streams or
 * host threads, race on it and must be serialised by the caller. A
 * bounded-wait timeout in this entry point's kernels is recorded in a
 * status word of its own, read by attn_get_noalloc_status(), not by
 * attn_get_device_status() (whose first use allocates its word).
 */
#define ATTN_NOALLOC_SCRATCH_BYTES (8u << 20)
attn_status_t attn_decode_splitkv_noalloc(const void *q, const void *k, const void *v, void *o,
                                          float *lse, int b, int sq, int sk, int h, int d,
                                          float scale, int num_splits, attn_dtype_t dtype,
                                          cudaStream_t stream);

/*
 * Status reader of attn_decode_splitkv_noalloc, allocating nothing either.
 * Synchronises `stream`, then reports and clears that entry point's status
 * word on the current device: ATTN_ERR_DEVICE_TIMEOUT if one of its kernels
 * abandoned a bounded wait since the last call (attn_last_timeout_site()
 * then names the kernel and wait), ATTN_ERR_CUDA if the stream reported an
 * error, ATTN_OK otherwise (also before the entry point's first call).
 */
attn_status_t attn_get_noalloc_status(cudaStream_t stream);

/*
 * The split heuristic for num_splits = 0 on the current device (same issue:
 * split only when the work units leave SMs idle; then one CTA per SM, at
 * most one split per key block and 128 splits). A work unit is one query
 * row of a (batch, head) when sq == 1, and 256 query rows of a (batch,
 * head) when sq > 1. Returns the split count (>= 1), or 0 on invalid sizes
 * or when no device can be queried.
 */
int attn_decode_num_splits(int b, int sq, int sk, int h, int d);

/* The same heuristic for an explicit SM count; pure host arithmetic. */
int attn_decode_num_splits_for_sms(int b, int sq, int sk, int h, int d, int num_sms);

/*
 * Synchronises `stream`, then reports and clears the current device's
 * status word: ATTN_ERR_DEVICE_TIMEOUT if a kernel abandoned a bounded wait
 * since the last call, ATTN_ERR_CUDA if the stream reported an error,
 * ATTN_OK otherwise.
 */
attn_status_t attn_get_device_status(cudaStream_t stream);

/* Where the last recorded timeout happened (kernel and wait site code), 0 if none. */
unsigned int attn_last_timeout_site(void);

/* Static, human-readable name of a status code. */
const char *attn_status_string(attn_status_t status);

/*
 * Waits for the current device to finish its work, frees the per-stream
 * workspaces of the split decode and of the packed and paged attention
 * (counters and partials; the next call on a stream makes them again; those
 * of destroyed streams go here too) and returns the memory the device's
 * default pool keeps cached to the system. No other call of this library
 * may run on the device meanwhile (from another host thread).
 */
void attn_release_workspace(void);

/*
 * Test hooks, host-side only and never needed in production; 0 restores
 * normal operation. ATTN_DEBUG_SKIP_LOADS makes the next launched kernels
 * issue no loads at all, so their first wait runs out and they return with
 * a timeout status instead of hanging. ATTN_DEBUG_GENERAL_FWD makes forward
 * calls with at most 256 keys and d <= 64, which normally run the short
 * forward kernel (all keys of a head in one tile), run the general
 * key-tile-loop kernel instead, so that both can be checked on one shape.
 * ATTN_DEBUG_GENERAL_BWD does the same for the short backward kernel: those
 * backward calls run the key-tile and query-tile kernels.
 */
#define ATTN_DEBUG_SKIP_LOADS 1u
#define ATTN_DEBUG_GENERAL_FWD 2u
#define ATTN_DEBUG_GENERAL_BWD 4u
void attn_debug_set_flags(unsigned int flags);

/*
 * Test hook, host-side only (launches nothing, needs no GPU): the plan the
 * short forward kernel (all keys of a head in one tile) would run a forward
 * of sq query rows, sk keys, h heads and head dim d with. grouped_ok != 0
 * allows heads in groups of four (attn_fwd allows it when the one-head tiles
 * outnumber the SMs). Returns 1 and writes 12 ints to out (caller-owned):
 *   out[0] key columns N of S (sk rounded up to 32)
 *   out[1] TMEM column of the O accumulator within a slot
 *   out[2] TMEM columns of one slot       out[3] slots (items in flight)
 *   out[4] bytes of one K or V tile       out[5] bytes of one stage
 *   out[6] stages                         out[7] 1 if heads are grouped
 *   out[8] 32-row query blocks per head (grouped; else 0)
 *   out[9] K/V stages (grouped; else 0)
 *   out[10] shared-memory bytes the tiles take
 *   out[11] shared-memory bytes available to them
 * Returns 0 and leaves out untouched when the short kernel does not take
 * the shape (sq, sk or h below 1, sk > 256, d not 16, 32 or 64) or out is
 * NULL.
 */
int attn_debug_short_plan(int sq, int sk, int h, int d, int grouped_ok, int *out);

/*
 * Test hook, host-side only: how a packed call of h query heads on h_kv K/V
 * heads would deal b sequences (host arrays of lengths) to ctas CTAs.
 * one_tile: units of one 128-row query tile instead of two; by_key != 0: the
 * key-tile units of the backward. Writes up to max_ranges rows of 9 ints:
 *   CTA, sequence, K/V head, unit, first step, steps, slot (-1: the unit is
 *   not cut; 0 / 1: a range that does not / does begin it), and of a cut unit
 *   the first CTA that shares it and how many do
 * and returns their number, or -1 on invalid arguments.
 */
int attn_debug_packed_plan(const int *seqlens_q, const int *seqlens_k, int b, int h, int h_kv,
                           int one_tile, int causal, int by_key, int ctas, int max_ranges, int *out);

/*
 * Test hook, host-side only: how attn_chunk_paged_q4 would deal requests with
 * few rows to warps: units of floor(rows / (h / h_kv)) tokens (rows 8 or 16),
 * steps of 32 keys. Otherwise as attn_debug_packed_plan, with warps for CTAs.
 */
int attn_debug_few_plan(const int *seqlens_q, const int *seqlens_k, int b, int h, int h_kv, int rows, int causal,
                        int warps, int max_ranges, int *out);

/*
 * Test hook, host-side only: attn_debug_packed_plan from starts as the kernels
 * read them (int32 [b + 1], whatever they hold) in tensors of total_q and
 * total_k rows: clamped, and nothing dealt out (0) where they are out of order.
 */
int attn_debug_packed_starts(const int *cu_seqlens_q, const int *cu_seqlens_k, int b, int total_q,
                             int total_k, int h, int h_kv, int one_tile, int causal, int by_key,
                             int ctas, int max_ranges, int *out);

/*
 * Test hook, host-side only: how many of ctas CTAs (at least 2) the packed
 * backward gives to its key tiles; out[0], out[1]: the logarithms of the units
 * in which the costs of its query-tile and key-tile work are counted (7: one
 * step). -1 on invalid arguments.
 */
int attn_debug_packed_shares(const int *seqlens_q, const int *seqlens_k, int b, int h, int h_kv,
                             int causal, int ctas, int *out);

/* Library ABI version (major * 100 + minor): 105. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EXATTN_H */
