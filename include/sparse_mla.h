/*
 * sparse_mla.h -- C ABI of the GB300 (sm_103a) sparse MLA attention forward (DSA top-k) and
 * its backward.
 *
 * The operation (FlashMLA PR #196, "Problem" and "Fix"; FlashMLA PR #216, "Summary";
 * FlashMLA PR #198, "Summary" item 2):
 *   For every query row t and head h, only the slots j of the row's index list that satisfy
 *       j < L_t   and   0 <= indices[t][j] < s_kv
 *   take part, where L_t = clamp(topk_length[t], 0, topk) when topk_length is given and
 *   L_t = topk otherwise.  With K = kv[:, :d_qk] and V = kv[:, :d_v] (the same latent row),
 *       logit_j   = sm_scale * <q[t,h,:], K[idx_j]>
 *       m         = max_j logit_j                         -> max_logits[t,h]
 *       lse[t,h]  = m + ln sum_j exp(logit_j - m)         (natural log, sink excluded)
 *       O[t,h,:]  = sum_j exp(logit_j - m) V[idx_j] / (sum_j exp(logit_j - m)
 *                                                      + [attn_sink] exp(attn_sink[h] - m))
 *   A row without any counted slot yields O = 0, lse = +inf, max_logits = -inf, with or
 *   without a sink.  Slots beyond L_t are never read, so their index values are unconstrained
 *   (e.g. INT_MAX padding is fine).  A duplicated index counts once per slot.
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers to contiguous row-major buffers.  The caller
 *     owns every buffer; the library allocates nothing and keeps no pointer after the call.
 *   - bf16 tensors are passed as `void*` holding IEEE bfloat16 values.
 *   - The work is enqueued on `stream` and is asynchronous: a return value of SMLA_OK only
 *     means the launch was accepted.  No launch happens when an error code is returned.
 *   - s_q == 0 is a no-op that returns SMLA_OK (pointers are then not inspected).
 *   - Supported shapes: h_q a positive multiple of 64 (<= 1024), d_qk in {512, 576},
 *     d_v == 512, topk >= 1, sm_scale finite and > 0, s_q * h_q <= INT32_MAX.
 *   - Alignment: q and kv (or kv_pool) 16-byte aligned; every other pointer 4-byte aligned.
 *   - Page planning, row append, dense chunk attention and the operators of a speculative step state their
 *     own shapes (any h_q up to 1024 among them), strides and alignment; those hold in place of the two rules above.
 *   - Requires an sm_103a device (GB300).
 */
#ifndef SPARSE_MLA_GB300_H_
#define SPARSE_MLA_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SMLA_ABI_VERSION 4

typedef struct CUstream_st* smla_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  SMLA_OK = 0,
  SMLA_ERR_NULL_PTR = 1,       /* a required pointer is NULL */
  SMLA_ERR_BAD_SHAPE = 2,      /* a size or scalar argument is outside the supported set */
  SMLA_ERR_MISALIGNED = 3,     /* a pointer violates the alignment rule above */
  SMLA_ERR_LAUNCH = 4,         /* the CUDA launch (or a CUDA query) failed */
  SMLA_ERR_DEVICE_TIMEOUT = 5, /* a device-side wait gave up (see sparse_mla_device_status) */
  SMLA_ERR_TENSOR_MAP = 6,     /* the TMA descriptor for an operand could not be encoded */
  SMLA_ERR_WORKSPACE = 7       /* split-KV workspace missing or smaller than required */
} smla_status;

/*
 * Sparse MLA forward over one shared latent KV (FlashMLA PR #196, "Problem": the sparse
 * prefill forward; one latent KV stream, h_kv = 1).
 *   q            [s_q, h_q, d_qk]  bf16
 *   kv           [s_kv, 1, d_qk]   bf16; V is kv[:, :, :d_v]
 *   indices      [s_q, 1, topk]    int32; any value, -1 / <0 / >= s_kv mean "no key"
 *   topk_length  [s_q]             int32 or NULL (FlashMLA PR #216, "Summary")
 *   attn_sink    [h_q]             fp32 or NULL (logit units of sm_scale * q.k)
 *   out          [s_q, h_q, d_v]   bf16   (written)
 *   lse          [s_q, h_q]        fp32   (written)
 *   max_logits   [s_q, h_q]        fp32   (written)
 * When topk_length is NULL, each row's work is bounded by its last valid slot, found by a
 * scan in the kernel prologue (FlashMLA PR #196, "Fix"); results are identical to passing
 * that length explicitly.  A row's counted slots are packed into dense 64-slot blocks, so
 * invalid entries anywhere in the row cost no compute; the result does not depend on where
 * they sit.
 */
smla_status sparse_mla_fwd(const void* q, const void* kv, const int32_t* indices,
                           const int32_t* topk_length, const float* attn_sink, float sm_scale,
                           int d_v, void* out, float* lse, float* max_logits, int64_t s_q,
                           int64_t s_kv, int h_q, int d_qk, int topk, smla_stream_t stream);

/*
 * Same forward over a paged KV cache (FlashMLA PR #216, "Dynamic top-k": decode with
 * per-request top-k token positions in a cache of 64-token pages).
 *   kv_pool      [pool_rows, 1, d_qk] bf16; pool_rows = number of pages * page_block
 *   block_table  [s_q / s_q_per_req, max_blocks] int32: page id of each page_block-token
 *                block of every request; a negative entry marks an unmapped page
 *   seqlens_k    [s_q / s_q_per_req] int32 KV length of each request, or NULL to use
 *                s_kv_per_req for all requests
 *   indices      [s_q, 1, topk] int32 token positions within the row's request
 * Query row t belongs to request t / s_q_per_req (s_q must be a multiple of s_q_per_req).
 * Position p of request b is read from pool row block_table[b][p / page_block] * page_block
 * + p % page_block, and counts iff 0 <= p < seqlens_k[b], p / page_block < max_blocks, the
 * table entry is >= 0 and the row is < pool_rows; any other position is an invalid slot and is
 * never used as an address (FlashMLA PR #216, "Summary").
 * All other arguments and outputs are as in sparse_mla_fwd.
 */
smla_status sparse_mla_fwd_paged(const void* q, const void* kv_pool, int64_t pool_rows,
                                 const int32_t* block_table, int max_blocks, int page_block,
                                 const int32_t* seqlens_k, int64_t s_kv_per_req, int s_q_per_req,
                                 const int32_t* indices, const int32_t* topk_length,
                                 const float* attn_sink, float sm_scale, int d_v, void* out,
                                 float* lse, float* max_logits, int64_t s_q, int h_q, int d_qk,
                                 int topk, smla_stream_t stream);

/*
 * Split-KV variants, for calls with fewer (row, 64-head group) items than SMs (small-batch
 * decode).  Each row's slot list [0, L_t) is cut into n_split contiguous ranges of
 * ceil(ceil(L_t / n_split) / 64) * 64 slots; every (row, head group, range) is one work unit
 * whose partial result (unnormalised O, exponent offset, sum, max) goes to `workspace`, and a
 * second kernel on the same stream merges a row's ranges with log-sum-exp weights (the sink
 * joins the denominator there) and writes out / lse / max_logits.  Same semantics and
 * outputs as sparse_mla_fwd / sparse_mla_fwd_paged up to summation order; with n_split == 1
 * they are the same call (no workspace needed).
 *   n_split          1 .. 64
 *   workspace        device buffer of at least sparse_mla_splitkv_workspace_size(s_q, h_q,
 *                    n_split) bytes, 256-byte aligned, owned by the caller; its contents
 *                    need no initialisation and are meaningless after the call.  Two calls
 *                    in flight at once must not share a workspace.
 * Errors as in the base calls, plus SMLA_ERR_BAD_SHAPE for n_split outside 1..64 and
 * SMLA_ERR_WORKSPACE when the workspace is NULL or too small (n_split > 1).
 */
size_t sparse_mla_splitkv_workspace_size(int64_t s_q, int h_q, int n_split);

smla_status sparse_mla_fwd_splitkv(const void* q, const void* kv, const int32_t* indices,
                                   const int32_t* topk_length, const float* attn_sink, float sm_scale,
                                   int d_v, void* out, float* lse, float* max_logits, int64_t s_q,
                                   int64_t s_kv, int h_q, int d_qk, int topk, int n_split,
                                   void* workspace, size_t workspace_bytes, smla_stream_t stream);

smla_status sparse_mla_fwd_paged_splitkv(const void* q, const void* kv_pool, int64_t pool_rows,
                                         const int32_t* block_table, int max_blocks, int page_block,
                                         const int32_t* seqlens_k, int64_t s_kv_per_req,
                                         int s_q_per_req, const int32_t* indices,
                                         const int32_t* topk_length, const float* attn_sink,
                                         float sm_scale, int d_v, void* out, float* lse,
                                         float* max_logits, int64_t s_q, int h_q, int d_qk, int topk,
                                         int n_split, void* workspace, size_t workspace_bytes,
                                         smla_stream_t stream);

/*
 * Allocation-free form of sparse_mla_fwd_paged_splitkv: the split-KV partial results go to a
 * scratch array that lives in the library itself (a 32 MiB __device__ array per device)
 * instead of a caller workspace, so the call needs no buffer besides its inputs and outputs.
 *   - Problems whose partial results do not fit, i.e. sparse_mla_splitkv_workspace_size(s_q,
 *     h_q, n_split) > 32 MiB (33554432 bytes), are rejected with SMLA_ERR_WORKSPACE before
 *     anything runs.
 *   - Nothing in the scratch has to start at zero (every work unit writes its whole partial
 *     result before the merge reads it), so the call clears nothing.
 *   - Races: all calls on one device share the one scratch array.  Two calls whose kernels
 *     may overlap (different streams, or different host threads without ordering) corrupt
 *     each other's partial results; callers must order them (same stream, or an event or
 *     synchronisation between them).  Calls on different devices are independent.
 * With n_split == 1 the scratch is not used.  Other arguments, outputs and errors are as in
 * sparse_mla_fwd_paged_splitkv.
 */
smla_status sparse_mla_fwd_paged_splitkv_static(
    const void* q, const void* kv_pool, int64_t pool_rows, const int32_t* block_table, int max_blocks,
    int page_block, const int32_t* seqlens_k, int64_t s_kv_per_req, int s_q_per_req,
    const int32_t* indices, const int32_t* topk_length, const float* attn_sink, float sm_scale, int d_v,
    void* out, float* lse, float* max_logits, int64_t s_q, int h_q, int d_qk, int topk, int n_split,
    smla_stream_t stream);

/*
 * End-to-end form of sparse_mla_fwd for inputs and outputs that live in HOST memory: the
 * host -> device copies of the inputs, the forward and the device -> host copies of the
 * outputs, pipelined over row chunks so that the copies of one chunk overlap the compute of
 * another.  Rows are independent, so the results are bit-identical to one sparse_mla_fwd call.
 *   *_host       host buffers with the layouts of sparse_mla_fwd (inputs read, outputs
 *                written); page-locked (pinned) memory is needed for the copies to overlap
 *   *_dev        caller-owned device buffers of the full sizes, with the alignment rules of
 *                sparse_mla_fwd; the inputs are copied into them and the outputs computed in
 *                them.  topk_length_dev / attn_sink_dev are NULL exactly when their host
 *                counterparts are (kv_host / kv_dev may be NULL only when s_kv == 0)
 *   n_chunks     1 .. 64: the rows are cut into n_chunks ranges of ceil(s_q / n_chunks) rows
 *   stream       the compute stream; when it has finished, every output copy has finished
 *   copy_in      stream of the host -> device copies (kv and attn_sink first, then each chunk)
 *   copy_out     stream of the device -> host copies
 * The copies start after the work already queued on `stream`, so the call is ordered on
 * `stream` as a whole.  The three streams are ordered with CUDA events from a pool that the
 * first call on a device creates and keeps until exit (no memory is allocated); calls from
 * several host threads take turns while they enqueue.  The call only enqueues work:
 * synchronise `stream` before reading the host outputs.  Every argument is checked before
 * anything is enqueued; SMLA_ERR_LAUNCH (a failed copy, event or launch) can come after
 * earlier chunks were enqueued.
 */
smla_status sparse_mla_fwd_host(const void* q_host, const void* kv_host, const int32_t* indices_host,
                                const int32_t* topk_length_host, const float* attn_sink_host, float sm_scale,
                                int d_v, void* out_host, float* lse_host, float* max_logits_host, int64_t s_q,
                                int64_t s_kv, int h_q, int d_qk, int topk, void* q_dev, void* kv_dev,
                                int32_t* indices_dev, int32_t* topk_length_dev, float* attn_sink_dev, void* out_dev,
                                float* lse_dev, float* max_logits_dev, int n_chunks, smla_stream_t stream,
                                smla_stream_t copy_in, smla_stream_t copy_out);

/*
 * Reads (and, when reset != 0, clears) the device-side status word that kernels set when one
 * of their bounded waits gave up: SMLA_OK or SMLA_ERR_DEVICE_TIMEOUT.  Synchronises with the
 * device (a blocking copy of one int); SMLA_ERR_LAUNCH if that copy fails.
 */
smla_status sparse_mla_device_status(int reset);

/*
 * Diagnostic of the failure-detection path: launches a one-thread kernel that runs the same
 * bounded mbarrier wait the forward kernels use, on a barrier nothing ever completes.  After
 * limit_ns (1 .. 2e9 ns) of device time the wait gives up, the kernel sets the status word to
 * SMLA_ERR_DEVICE_TIMEOUT and returns; the context stays usable.  Read the result with
 * sparse_mla_device_status after synchronising.  SMLA_ERR_BAD_SHAPE for a limit out of range.
 */
smla_status sparse_mla_selftest_wait_timeout(uint64_t limit_ns, smla_stream_t stream);

/*
 * Sparse MLA backward over one shared latent KV (FlashMLA PR #198, "Summary" item 1: the
 * sparse MLA backward, dK / dV scattered into the shared latent rows).  It returns the
 * gradients of  L = sum_{t,h,d} dout[t,h,d] * O[t,h,d]  for the forward above:
 *   p_j      = exp(sm_scale <q[t,h,:], K[idx_j]> - lse_full[t,h]),
 *              lse_full = ln(exp(lse[t,h]) + [attn_sink] exp(attn_sink[h]))
 *   D[t,h]   = <dout[t,h,:], out[t,h,:]>,   dS_j = p_j (<dout[t,h,:], V[idx_j]> - D[t,h])
 *   dq[t,h,:]            = sm_scale sum_j dS_j K[idx_j]
 *   dkv[idx_j, :d_qk]   += sm_scale dS_j q[t,h,:]     (summed over every row, head and slot)
 *   dkv[idx_j, :d_v]    += p_j dout[t,h,:]
 *   dsink[h]            += -exp(attn_sink[h] - lse_full[t,h]) D[t,h]
 * over the same counted slots as the forward (j < L_t and 0 <= idx < s_kv; duplicated indices
 * count once per slot).  A row without a counted slot contributes nothing (its dq is 0).
 *   q, kv, indices, topk_length, attn_sink, sm_scale, d_v: as for sparse_mla_fwd
 *   out          [s_q, h_q, d_v]   bf16   the forward's output (16-byte aligned)
 *   dout         [s_q, h_q, d_v]   bf16   gradient of the loss w.r.t. out (16-byte aligned)
 *   lse          [s_q, h_q]        fp32   the forward's lse (natural log, sink excluded)
 *   dq           [s_q, h_q, d_qk]  fp32   (written)
 *   dkv          [s_kv, d_qk]      fp32   (written: zeroed on the stream, then accumulated
 *                                          with fp32 atomics, so the summation order and the
 *                                          last bits vary from run to run); may be NULL only
 *                                          when s_kv == 0
 *   dsink        [h_q]             fp32 or NULL (written when attn_sink is given: zeroed,
 *                                          then accumulated; zeroed otherwise)
 * Every row's work is bounded by L_t (topk_length, or topk); slots in [0, L_t) that do not
 * count are masked.  Uses no workspace and allocates nothing.  With s_q == 0, dkv and dsink
 * are zeroed and nothing else happens.  Every error except SMLA_ERR_LAUNCH is returned before
 * anything is enqueued; SMLA_ERR_LAUNCH may come after the zeroing of dkv and dsink was
 * queued, which then leaves them zeroed.
 */
smla_status sparse_mla_bwd(const void* q, const void* kv, const void* out, const void* dout,
                           const int32_t* indices, const int32_t* topk_length, const float* attn_sink,
                           const float* lse, float sm_scale, int d_v, float* dq, float* dkv, float* dsink,
                           int64_t s_q, int64_t s_kv, int h_q, int d_qk, int topk, smla_stream_t stream);

/*
 * Page planning of one serving step, on the device: which cache pages and rows the step's new
 * tokens get, from the requests' lengths alone.  For request b, with o_b = max(seqlens[b], 0)
 * cached and m_b = max(new_lens[b], 0) new tokens:
 *   cu_seqlens_q  [n_req + 1]  running sums of m_b from 0, clamped to n_tokens; c_b is the
 *                              difference of entries b + 1 and b
 *   seqlens_k     [n_req]      o_b + c_b
 *   block_table   [n_req, max_blocks]  columns ceil(o_b / page_block) .. ceil(seqlens_k[b] /
 *                              page_block) - 1 (those below max_blocks) get the next pages of
 *                              the free list, request by request and column by column, -1 once
 *                              the list is used up; every other column is left as it is
 *   positions     [n_tokens]   o_b + t - cu_seqlens_q[b] for token t of request b, -1 behind
 *                              the last token
 *   slots         [n_tokens]   table entry of the position * page_block + position % page_block;
 *                              -1 behind the last token, past the table's last column, or where
 *                              the entry is negative
 *   counts        [3]          tokens placed, index of the first free page not handed out,
 *                              pages that were needed but not there
 *   free_pages    [n_free]     page ids; the pages are handed out from index free_start[0]
 *                              (device memory, NULL: 0; negative: 0).  The previous step's
 *                              counts + 1 is a valid free_start, in another buffer.
 * The block table, the lengths and the sums have the layouts that sparse_mla_fwd_paged,
 * sparse_mla_append_kv and sparse_mla_chunk_fwd_paged read.  With the same inputs a second call
 * writes the same values.  n_tokens may exceed the step's tokens (a padded batch).  Sizes are
 * at least 0; max_blocks and page_block at least 1, their product, n_tokens, n_free and every
 * o_b + c_b at most INT32_MAX.  Pointers are 4-byte aligned; those of empty arrays may be
 * NULL.  SMLA_ERR_BAD_SHAPE when an output overlaps an input or another output.
 */
smla_status sparse_mla_plan_pages(const int32_t* seqlens, const int32_t* new_lens, int32_t* block_table,
                                  const int32_t* free_pages, const int32_t* free_start, int32_t* seqlens_k,
                                  int32_t* cu_seqlens_q, int32_t* slots, int32_t* positions, int32_t* counts,
                                  int64_t n_req, int64_t n_free, int64_t n_tokens, int max_blocks, int page_block,
                                  smla_stream_t stream);

/*
 * Appends the latent rows of n new tokens to a paged cache, and turns the queries' rotary columns
 * in the same launch.  Row slots[t] of kv_pool becomes
 *   [0, 512)    c_kv[t, d] * norm_weight[d] / sqrt(mean(c_kv[t]^2) + eps), or c_kv[t] as it is
 *               when norm_weight is NULL
 *   [512, 576)  (d_qk 576 only) k_pe[t] with each pair (x, y) of columns 2i, 2i + 1 turned to
 *               (x cos - y sin, y cos + x sin); as it is when rope is NULL
 * and, when q_pe is given, q[t, h, 512:] becomes q_pe[t, h] turned by the same angles.
 *   c_kv         [n, 512] bf16, row stride c_stride elements (a multiple of 8), 16-byte aligned
 *   k_pe         [n, 64] bf16, row stride k_stride (even), 4-byte aligned; given exactly when
 *                d_qk is 576
 *   slots        [n] int32 pool rows; a negative one, or one >= pool_rows, is not written
 *   positions    [n] int32 rows of the rope table (with rope only)
 *   rope         [max_pos, 64] fp32, 16-byte aligned: 32 cosines, then 32 sines of a position; NULL
 *                for none.  A token whose position lies outside [0, max_pos) is not written, neither
 *                its cache row nor its q columns: negative positions are padding, those at or past
 *                max_pos an error of the caller's, which sparse_mla_append_kv_counted reports.  The
 *                planner gives a token a slot wherever the block table has a page for its position, and
 *                the attention reads that row; with max_pos >= max_blocks * page_block every such row is
 *                written.
 *   norm_weight  [512] bf16, 16-byte aligned, or NULL; eps finite and >= 0
 *   q_pe         [n, h_q, 64] bf16, strides q_stride_t and q_stride_h elements (multiples of 8),
 *                16-byte aligned, or NULL; needs rope.  It may be q[..., 512:] itself.
 *   q            [n, h_q, 576] bf16, 16-byte aligned; given exactly when q_pe is
 *   kv_pool      [pool_rows, d_qk] bf16, 16-byte aligned
 * A stride over a single token (n == 1) or head (h_q == 1) is not looked at.
 * Arithmetic is fp32, each value is rounded to bf16 once; without a norm weight (without rope) the
 * bits are copied.  Two tokens with one slot leave that row undefined.  SMLA_ERR_BAD_SHAPE when
 * kv_pool or q overlaps an input or the other; q_pe may lie in q in its own place alone.
 * n == 0 is a no-op.
 */
smla_status sparse_mla_append_kv(const void* c_kv, int64_t c_stride, const void* k_pe, int64_t k_stride,
                                 const int32_t* slots, const int32_t* positions, const float* rope, int64_t max_pos,
                                 const void* norm_weight, float eps, const void* q_pe, int64_t q_stride_t,
                                 int64_t q_stride_h, void* q, int h_q, void* kv_pool, int64_t pool_rows, int d_qk,
                                 int64_t n, smla_stream_t stream);

/*
 * The same, and adds the number of tokens whose position is at or past max_pos to past_rope[0] (device
 * memory, int32, 4-byte aligned, outside kv_pool, q, slots and positions; zeroed by the caller when the
 * count is to start).  After such a token its request's keys are incomplete, and its q columns were not turned.
 */
smla_status sparse_mla_append_kv_counted(const void* c_kv, int64_t c_stride, const void* k_pe, int64_t k_stride,
                                         const int32_t* slots, const int32_t* positions, const float* rope,
                                         int64_t max_pos, const void* norm_weight, float eps, const void* q_pe,
                                         int64_t q_stride_t, int64_t q_stride_h, void* q, int h_q, void* kv_pool,
                                         int64_t pool_rows, int d_qk, int64_t n, int32_t* past_rope,
                                         smla_stream_t stream);

/*
 * Dense attention of a chunk of new tokens over a paged latent cache: the operation of
 * sparse_mla_fwd_paged with every visible position counted instead of an index list, for ragged
 * requests of one token (decode) to whole prompts (chunked prefill).
 *   q             [n_tok, h_q, d_qk] bf16; rows cu_seqlens_q[b] .. cu_seqlens_q[b + 1] - 1 are
 *                 request b's q_b new tokens (values are clamped to [0, n_tok]; they must not
 *                 decrease).  Rows of no request are left unwritten in every output.
 *   kv_pool       [pool_rows, 1, d_qk] bf16
 *   page_block    any size; multiples of 32 are fastest, of 16 take up to 1.25 times as long, of 8 up
 *                 to 1.7 times, other sizes 3 to 4 times
 *   block_table   [n_req, max_blocks] int32, as in sparse_mla_fwd_paged
 *   seqlens_k     [n_req] int32: keys of request b, its new tokens' own rows among them
 *   causal        nonzero: token i of request b (at position seqlens_k[b] - q_b + i) sees the
 *                 positions up to its own; zero: it sees every position below seqlens_k[b].  A
 *                 token at a negative position sees none.
 *   out, lse, max_logits, attn_sink, sm_scale, d_v: as in sparse_mla_fwd, an empty row's values
 *                 included (O = 0, lse = +inf, max_logits = -inf)
 * A position counts only if its page lies in the table's max_blocks columns, the entry is >= 0
 * and the row is < pool_rows; any other is an invalid slot and never an address.  Rows of
 * positions at or past seqlens_k[b] are not read into any product: they may hold anything, NaN
 * among it.  Rows below it must be finite: NaN in one reaches every token that sees it, and may reach
 * the request's others.  A (token, head) row of q with NaN in it gives NaN in that row's out, lse and
 * max_logits and in no other's, and a score above fp32's range NaN in that row's out and lse.  One below
 * it (-inf) counts as a masked one.
 * Scores and softmax sums are fp32.  The softmax weights are rounded to bf16, the type of V, before their product
 * with V (2^-8 of a weight at most; lse and max_logits take the unrounded ones), and out once more.
 *   h_q           1 .. 1024 (any: all heads of a token share the one latent row)
 *   n_tok * h_q   at most INT32_MAX
 *   workspace     device buffer of at least sparse_mla_chunk_workspace_size(n_tok, h_q) bytes,
 *                 256-byte aligned, owned by the caller; needs no initialisation, its contents
 *                 are meaningless after the call.  Two calls in flight at once must not share it.
 * q, kv_pool and out are 16-byte aligned, the rest 4-byte.  SMLA_ERR_BAD_SHAPE when out, lse,
 * max_logits or the workspace overlaps an input or another of them.  The result does not depend on
 * anything but the arguments (no atomics): two calls give the same bits.
 * n_tok == 0 or n_req == 0 is a no-op.
 */
size_t sparse_mla_chunk_workspace_size(int64_t n_tok, int h_q);

smla_status sparse_mla_chunk_fwd_paged(const void* q, const void* kv_pool, int64_t pool_rows,
                                       const int32_t* block_table, int max_blocks, int page_block,
                                       const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int64_t n_req, int causal,
                                       const float* attn_sink, float sm_scale, int d_v, void* out, float* lse,
                                       float* max_logits, int64_t n_tok, int h_q, int d_qk, void* workspace,
                                       size_t workspace_bytes, smla_stream_t stream);

/* sparse_mla_device_status of sparse_mla_chunk_fwd_paged's kernel, which has its own word. */
smla_status sparse_mla_chunk_device_status(int reset);

/*
 * sparse_mla_selftest_wait_timeout of that kernel's waits: its two forms give up after limit_ns each, a third
 * wait at once on the flag that the first has set; the chunk kernel's status word says so.
 */
smla_status sparse_mla_chunk_selftest_wait_timeout(uint64_t limit_ns, smla_stream_t stream);

/*
 * A speculative step: a request's new tokens are the nodes of a tree, node 0 its last known token and the
 * others drafts, each behind its parent.  sparse_mla_plan_pages gives them rows, sparse_mla_plan_tree masks and
 * positions, sparse_mla_append_kv writes the rows, sparse_mla_tree_fwd_paged attends, sparse_mla_verify_tree finds the
 * path that is kept, and sparse_mla_commit_tree moves its rows together and gives back the pages behind them.  The
 * host reads nothing in between.
 *
 * Masks and positions of the trees.  With node i of request b in row t = cu_seqlens_q[b] + i, n_b nodes and
 * A_i = {i} and the nodes on its way up:
 *   parents      [n_tok] int32: index of the parent within the request, below the node's own; anything else (-1)
 *                means none: the node comes straight behind the cached tokens
 *   cu_seqlens_q [n_req + 1], seqlens_k [n_req]: as for sparse_mla_tree_fwd_paged
 *   tree_mask    [n_tok, mask_words] int32 (written): bit j of word w of row t is set when node 32 w + j is in A_i.
 *                Nodes from 32 mask_words on are in no mask.
 *   positions    [n_tok] int32 (written): seqlens_k[b] - n_b + |A_i| - 1, the position for the rotary columns
 * Rows of no request get an empty mask and position -1.  mask_words is 1 .. 1024, n_tok at most 2^30.  All pointers 4-byte
 * aligned.
 * SMLA_ERR_BAD_SHAPE when an output overlaps an input or the other output.  n_tok == 0 is a no-op.
 */
smla_status sparse_mla_plan_tree(const int32_t* parents, const int32_t* cu_seqlens_q, const int32_t* seqlens_k,
                                 int32_t* tree_mask, int32_t* positions, int64_t n_req, int64_t n_tok, int mask_words,
                                 smla_stream_t stream);

/*
 * Dense attention of the nodes of trees over a paged latent cache: sparse_mla_chunk_fwd_paged with another rule of
 * what a token sees.  Node i of request b (n_b nodes) sees every position below seqlens_k[b] - n_b, and position
 * seqlens_k[b] - n_b + j exactly when bit j % 32 of word j / 32 of its row of tree_mask is set (j may be above i).
 *   tree_mask     [n_tok, mask_words] int32, mask_words 1 .. 1024; nodes from 32 mask_words on are seen by none
 * Everything else is as there: ragged requests, page rules, workspace (sparse_mla_chunk_workspace_size), empty
 * rows (a node that sees nothing: O = 0, lse = +inf, max_logits = -inf), NaN, rows that are left unwritten, errors.
 * In particular every row below seqlens_k[b] must be finite, those of nodes that a token does not see among them: NaN
 * in one reaches lse and max_logits of the tokens that see it, and may reach out of all of the request's.
 * A causal mask (bits 0 .. i) gives the values of the causal form up to the order of its sums.
 */
smla_status sparse_mla_tree_fwd_paged(const void* q, const void* kv_pool, int64_t pool_rows,
                                      const int32_t* block_table, int max_blocks, int page_block,
                                      const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int64_t n_req,
                                      const int32_t* tree_mask, int mask_words, const float* attn_sink, float sm_scale,
                                      int d_v, void* out, float* lse, float* max_logits, int64_t n_tok, int h_q, int d_qk,
                                      void* workspace, size_t workspace_bytes, smla_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given random numbers.  A request's nodes
 * lie in rows cu_seqlens_q[b] .. (clamped to [0, n_tok], as in the attention).  The walk starts at node 0; a current
 * node's children are tried in index order, with p and q the current node's rows of target_probs and draft_probs, x a
 * child's token and u its accept_u:
 *   with draft_probs (children drawn independently from q):
 *     C = 0, Z = 1, r(v) = max(p(v) - C q(v), 0) rounded to fp32; the child is kept when u q(x) Z < r(x), else
 *     C becomes C + Z (fp32) and Z the sum of the new r
 *   without (children chosen outright, the likeliest tokens for example):
 *     r = p, Z = 1; the child is kept when u Z < r(x), else Z becomes Z - r(x) and r(x) 0
 *   A child that is kept becomes the current node.
 * When no child is left, or max_keep nodes are kept, the request's last token is drawn from the current r: the first v
 * with r(0) + .. + r(v) > sample_u[b] * sum r (the last v with r(v) > 0 where rounding leaves none; with r all zero,
 * p's; -1 when p has no positive value).  The tokens kept and drawn follow the target's distribution, whatever the
 * drafts.  Products (of 2^-100 and more), sums of r, Z and the comparisons hold 46 bits and more, in an order that depends on the
 * sizes alone.
 *   target_probs [n_tok, vocab] fp32, vocab 1 .. 2^30, row stride target_stride elements (>= vocab); rows sum to 1; NaN and negative
 *                values count as 0
 *   draft_probs  [n_tok, vocab] fp32, row stride draft_stride, or NULL; row t is what node t's children were drawn
 *                from (rows of nodes without children are not read); values >= 0
 *   tokens       [n_tok] int32; a child whose token lies outside [0, vocab) is passed over
 *   parents      [n_tok] int32 as for sparse_mla_plan_tree; a node without a parent is never tried (node 0 apart)
 *   accept_u     [n_tok] fp32, sample_u [n_req] fp32: numbers in [0, 1)
 *   keep         [n_req, max_keep] int32 (written): node 0 and the kept nodes, in order; -1 behind them
 *   out_tokens   [n_req, max_keep] int32 (written): the kept drafts' tokens and the drawn one; -1 behind them
 *   n_keep       [n_req] int32 (written): entries of both; 0 for a request without nodes
 * Nodes of a request from 1024 on are not tried.  max_keep >= 1, n_req * max_keep <= INT32_MAX.  All pointers
 * 4-byte aligned.  The stride of a single row is not looked at.  SMLA_ERR_BAD_SHAPE when an output overlaps an
 * input or another output.  The same inputs give the same result.  n_req == 0 is a no-op.
 */
smla_status sparse_mla_verify_tree(const float* target_probs, int64_t target_stride, const float* draft_probs,
                                   int64_t draft_stride, const int32_t* tokens, const int32_t* parents,
                                   const int32_t* cu_seqlens_q, const float* accept_u, const float* sample_u,
                                   int32_t* keep, int32_t* out_tokens, int32_t* n_keep, int64_t n_req, int64_t n_tok,
                                   int vocab, int max_keep, smla_stream_t stream);

/*
 * Commits what was kept of a step.  For request b with n_b = cu_seqlens_q[b + 1] - cu_seqlens_q[b] new tokens behind
 * before = seqlens_k[b] - n_b cached ones, and m = n_keep[b], at most n_b and max_keep:
 *   the row of position before + keep[b, i] goes to that of position before + i for i = 0 .. m - 1, in every layer;
 *   seqlens[b] = before + m; the pages of table columns ceil(seqlens[b] / page_block) .. ceil(seqlens_k[b] /
 *   page_block) - 1 go back to the free list.
 * n_keep[b] < 0 ends the request: no row moves, seqlens[b] = 0 and all of its pages go back.
 *   keep         [n_req, max_keep] int32, n_keep [n_req] int32: as sparse_mla_verify_tree writes them.  A request's
 *                entries ascend and are below n_b; where they do not, its rows from before on are undefined.
 *   seqlens_k    [n_req], cu_seqlens_q [n_req + 1], block_table [n_req, max_blocks]: those of the attention, but the sums are taken as
 *                they are, since no n_tok is known here: 0 <= cu_seqlens_q[b] <= cu_seqlens_q[b + 1] <= n_tok of the step's other
 *                calls, as sparse_mla_plan_pages writes them.  (Those clamp sums to n_tok; with sums past it they would take the
 *                first new position to be another than this call does, and other rows would be moved.)  The table
 *                is not changed: entries behind the new length are stale, and sparse_mla_plan_pages writes over them.
 *                A row without a page is neither moved nor written.
 *   kv_pool      [n_layers, pool_rows, d_qk] bf16, layers layer_stride elements apart (a multiple of 8, at least
 *                pool_rows * d_qk), 16-byte aligned; n_layers 0: no rows are moved.  Rows from before on lie in pages of
 *                the request's own.
 *   free_pages   [n_free] int32 (written below free_start); NULL or empty: no page goes back.  sparse_mla_plan_pages hands out
 *                from index free_start on; pages come back in front of it, request by request and column by
 *                column, each to the index below the last.
 *   free_start   [1] int32 or NULL for n_free (clamped to [0, n_free])
 *   seqlens      [n_req] int32 (written)
 *   counts       [3] int32 (written): tokens kept, the next free_start, pages for which there was no room in front of
 *                free_start (they stay in the table only); the latter two 0 without free_pages
 * counts + 1 is the next sparse_mla_plan_pages' free_start, seqlens its seqlens.  All other pointers 4-byte aligned; those
 * of empty arrays may be NULL.  The stride of a single layer is not looked at.  SMLA_ERR_BAD_SHAPE when an output
 * overlaps an input or another output.
 */
smla_status sparse_mla_commit_tree(const int32_t* keep, const int32_t* n_keep, int max_keep, const int32_t* cu_seqlens_q,
                                   const int32_t* seqlens_k, const int32_t* block_table, int max_blocks, int page_block,
                                   int64_t n_req, void* kv_pool, int n_layers, int64_t layer_stride, int64_t pool_rows,
                                   int d_qk, int32_t* free_pages, int64_t n_free, const int32_t* free_start,
                                   int32_t* seqlens, int32_t* counts, smla_stream_t stream);

/* Static, human-readable description of a status code.  Never NULL. */
const char* sparse_mla_status_string(smla_status status);

/* SMLA_ABI_VERSION of the loaded library. */
int sparse_mla_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_MLA_GB300_H_ */
