/*
 * fabwd.h -- C ABI of libfabwd.so, a single-pass flash-attention backward
 * for NVIDIA GB300 (sm_103a).
 *
 * The operation (cited by page title and section):
 *   "PyPTO-Gym SK-16: single-pass Attention backward (FA Grad)" article,
 *   section 3 (kernel skeleton with inputs q, k, v, o, do, l, m and outputs
 *   dq, dk, dv over packed variable-length batches with cumulative offsets
 *   actual_q / actual_kv), section 3.1 (the eight per-block steps) and
 *   section 4.2 (dtype table).  For each sequence b and head h, with
 *   X = scale * Q K^T (masked entries -inf):
 *       P  = exp(X - m) / l              (m, l given, never recomputed)
 *       dP = dO V^T,  D = rowsum(O * dO), dS = P * (dP - D)
 *       dV = P^T dO,  dK = scale * dS^T Q,  dQ = scale * dS K
 *   The causal mask is top-left aligned (key j visible to query i iff
 *   j <= i, local indices; the JAX cuDNN wrapper's MaskType.CAUSAL).
 *
 * Conventions shared by every entry point:
 *   - Tensors are packed and contiguous.  q, o, dout, dq: [total_q, H, d];
 *     k, v, dk, dv: [total_kv, H, d], or [total_kv, Hkv, d] in the entry
 *     points that take heads_kv (grouped-query attention, Hkv divides H);
 *     m, l, D: [total_q, H] (float32).
 *     Element type fa_bf16 is the raw 16-bit pattern of a bfloat16.
 *     The head h of row r sits at element offset (r * H + h) * d.
 *   - cu_q / cu_kv are int32 cumulative offsets with batch+1 entries,
 *     cu[0] = 0, non-decreasing, cu[batch] <= total.  Sequence b owns
 *     rows [cu[b], cu[b+1]).  Rows at or beyond cu[batch] are padding.
 *     Entry points that take both a device and a host copy need both to
 *     hold the same values: the host copy sizes the launch.
 *   - All device pointers are caller-owned device memory, 16-byte aligned.
 *     The library allocates no device memory on these paths.
 *   - head_dim must be 64, 128 or 256 (the JAX cuDNN wrapper's
 *     check_is_flash_attention admits head dims up to 256); heads >= 1.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; 0 = legacy
 *     default stream) and returns FA_OK or an error code.  Arguments are
 *     checked on the host before anything is launched; on an error nothing
 *     is launched and fa_last_error() describes the problem.
 *   - Device-side waits are bounded (20 s of wall time each).  A kernel
 *     whose internal wait runs out records FA_ERR_TIMEOUT in a device
 *     status word and returns early, leaving its outputs incomplete;
 *     fa_check_device_status() reads and clears the word.  A call's outputs
 *     are valid only once a later fa_check_device_status() has returned
 *     FA_OK (the Python binding's high-level functions do this by default).
 */
#ifndef FABWD_H
#define FABWD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t fa_bf16;               /* bfloat16 bit pattern */
typedef struct CUstream_st* fa_stream_t;  /* same type as cudaStream_t */

enum fa_status {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,   /* null pointer, bad offsets, bad sizes, misalignment */
    FA_ERR_UNSUPPORTED = 2,   /* head_dim not in {64, 128, 256}, no sm_103a device */
    FA_ERR_CUDA = 3,          /* a CUDA runtime or driver call failed */
    FA_ERR_TIMEOUT = 4        /* a device-side bounded wait ran out */
};

enum fa_dq_mode {
    FA_DQ_ATOMIC = 0,         /* dQ partials added with fp32 atomics, in any order */
    FA_DQ_DETERMINISTIC = 1   /* bitwise reproducible dQ.  head_dim 64 / 128: the key-block-outer
                                 kernel computes dK and dV only, and a query-block-outer kernel sums
                                 each row of dQ in one CTA in ascending key-block order (no atomics,
                                 no waits between CTAs, no workspace).  The two kernels are
                                 independent: the dQ kernel runs on a second stream that the library
                                 keeps per device and context, forked from `stream` and joined back
                                 into it with events (calls stay ordered on `stream`; while `stream`
                                 is being captured into a graph, both run in order on it).
                                 head_dim 256: dQ partials
                                 added in a fixed key-block order through counters in
                                 fa_bwd_workspace_size() bytes of workspace */
};

/* Masks of the _ex entry points (local indices i of the query, j of the key
 * within one sequence of s1 queries and s2 keys).  JAX
 * fused_attention_stablehlo.py, MaskType and the sliding_window_length
 * argument of dot_product_attention. */
enum fa_mask {
    FA_MASK_NONE = 0,                  /* every key visible */
    FA_MASK_CAUSAL = 1,                /* top-left: j <= i (MaskType.CAUSAL) */
    FA_MASK_CAUSAL_BOTTOM_RIGHT = 2    /* diagonal through the last key: j <= i + s2 - s1
                                          (the pages define no alignment for s1 != s2;
                                          this is the other usual one) */
};

/* Forward statistics used to build consistent backward inputs (support
 * step; the SK-16 article, section 5, says the forward skeleton supplies
 * l and m).  Writes O = softmax(scale*QK^T) V (bf16), m_i = max_j of the
 * scaled scores and l_i = sum_j exp(scaled score - m_i) (float32) for every
 * row of every sequence.  Rows of a sequence with no keys get O = 0,
 * m = -inf, l = 0.  Padding rows are not written.  Runs on the tensor cores
 * (a CTA owns one 128-row query block, or two of them at head_dim 128
 * sharing each key/value tile; O accumulates in tensor memory); q, k, v
 * and o must be 16-byte aligned. */
int fa_fwd_stats(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v,
                 fa_bf16* o, float* m, float* l,
                 const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
                 const int32_t* cu_q_host, const int32_t* cu_kv_host,
                 int batch, int total_q, int total_kv, int heads, int head_dim,
                 int causal, float scale, fa_stream_t stream);

/* fa_fwd_stats for grouped-query attention: k and v have heads_kv heads
 * ([total_kv, heads_kv, d]); query head h uses key/value head
 * h / (heads / heads_kv) (consecutive groups; the JAX cuDNN wrapper's
 * q_N != kv_N case of JAX fused_attention_stablehlo.py,
 * `_dot_product_attention_bwd_cuda_lowering`).
 * heads must be a positive multiple of heads_kv.  fa_fwd_stats is this
 * call with heads_kv = heads. */
int fa_fwd_stats_gqa(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v,
                     fa_bf16* o, float* m, float* l,
                     const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
                     const int32_t* cu_q_host, const int32_t* cu_kv_host,
                     int batch, int total_q, int total_kv, int heads, int heads_kv, int head_dim,
                     int causal, float scale, fa_stream_t stream);

/* fa_fwd_stats_gqa with a mask and a sliding window: mask is an fa_mask;
 * window = W > 0 restricts a causal mask to the left window (pos - W, pos]
 * with pos = i (top-left) or i + s2 - s1 (bottom-right), i.e. query i sees
 * keys j with pos - W < j <= pos (JAX dot_product_attention,
 * sliding_window_length); window = 0 means no window, and a window needs
 * a causal mask.  Rows that see no key get O = 0, m = -inf, l = 0. */
int fa_fwd_stats_ex(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v,
                    fa_bf16* o, float* m, float* l,
                    const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
                    const int32_t* cu_q_host, const int32_t* cu_kv_host,
                    int batch, int total_q, int total_kv, int heads, int heads_kv, int head_dim,
                    int mask, int window, float scale, fa_stream_t stream);

/* fa_fwd_stats_ex writing the single softmax statistic per row instead of
 * (m, l): lse[r, h] = m + ln(l) (natural log; -inf for rows that see no
 * key).  JAX fused_attention_stablehlo.py keeps one float32 softmax_stat of
 * shape (B, N, T) between its forward and backward calls; lse is the
 * reading of what it holds.  lse: [total_q, H] float32. */
int fa_fwd_lse(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v,
               fa_bf16* o, float* lse,
               const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
               const int32_t* cu_q_host, const int32_t* cu_kv_host,
               int batch, int total_q, int total_kv, int heads, int heads_kv, int head_dim,
               int mask, int window, float scale, fa_stream_t stream);

/* Backward preprocess (section 3.1 step 4; section 4.2 row "D"):
 * D[r, h] = sum_k float(O[r,h,k]) * float(dO[r,h,k]) for every row
 * r < total_q, and dq_acc[r, h, :] = 0 (float32 accumulator of
 * [total_q, H, d]; the SK-16 host pre-zeroes its atomic targets, section 4).
 */
int fa_bwd_preprocess(const fa_bf16* o, const fa_bf16* dout, float* D, float* dq_acc,
                      int total_q, int heads, int head_dim, fa_stream_t stream);

/* Bytes of device workspace fa_bwd needs for these shapes and dq_mode
 * (0 for FA_DQ_ATOMIC).  The JAX cuDNN wrapper
 * (fused_attention_stablehlo.py, _dot_product_attention_bwd_cuda_lowering)
 * likewise returns a workspace buffer sized for the backward call, and the
 * SK-16 article (section 6) sizes the kernel's scratch with its
 * max_workspace_kb option; here the caller allocates it.  Returns 0 and
 * sets fa_last_error() on bad arguments, so check fa_last_error() when a
 * mode needs workspace. */
size_t fa_bwd_workspace_size(const int32_t* cu_q_host, const int32_t* cu_kv_host,
                             int batch, int heads, int head_dim, int causal, int dq_mode);

/* The single-pass backward (section 3: C1 -> V1 -> C2 -> V2), key-block
 * outer.  Each CTA owns one (sequence, head, 128-row key block), keeps
 * its dK and dV accumulators in tensor memory for the whole query sweep and
 * writes them once; the unscaled dS K partial of every (query block, key
 * block) pair is added into dq_acc (float32, zeroed by fa_bwd_preprocess).
 * Inputs: q, k, v, dout (bf16), m, l (the forward statistics, consumed as
 * given: section 4.1) and D from fa_bwd_preprocess.  Outputs: dk = bf16(scale
 * * dS^T Q) and dv = bf16(P^T dO) for every key row of every sequence
 * (exact zeros for keys no query sees), zeros in padding rows
 * [cu_kv[batch], total_kv).  dq_acc must then go through
 * fa_bwd_dq_finalize.  workspace: at least fa_bwd_workspace_size() bytes
 * (may be NULL when that is 0); its contents need no initialisation. */
int fa_bwd(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, const fa_bf16* dout,
           const float* m, const float* l, const float* D,
           float* dq_acc, fa_bf16* dk, fa_bf16* dv,
           const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
           const int32_t* cu_q_host, const int32_t* cu_kv_host,
           int batch, int total_q, int total_kv, int heads, int head_dim,
           int causal, float scale, int dq_mode,
           void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* fa_bwd for grouped-query attention: q, dout, m, l, D, dq_acc have heads
 * query heads; k, v, dk, dv have heads_kv heads ([total_kv, heads_kv, d]);
 * query head h attends with key/value head h / (heads / heads_kv).  The
 * gradients of a shared key/value head are the sums over its query heads:
 * one CTA per (sequence, key/value head, key block) sweeps the query blocks
 * of every query head of the group, accumulating dK and dV on chip.
 * fa_bwd is this call with heads_kv = heads; the workspace size is that of
 * fa_bwd with `heads` query heads. */
int fa_bwd_gqa(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, const fa_bf16* dout,
               const float* m, const float* l, const float* D,
               float* dq_acc, fa_bf16* dk, fa_bf16* dv,
               const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
               const int32_t* cu_q_host, const int32_t* cu_kv_host,
               int batch, int total_q, int total_kv, int heads, int heads_kv, int head_dim,
               int causal, float scale, int dq_mode,
               void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* fa_bwd_gqa with a mask and a sliding window (as in fa_fwd_stats_ex).
 * A CTA visits only the query blocks whose tiles the band of visible
 * (query, key) pairs meets; gradients of keys no query sees are exact
 * zeros.  fa_bwd and fa_bwd_gqa are this call with mask = causal and
 * window = 0.  In FA_DQ_DETERMINISTIC mode the key-block order of the dQ
 * additions is fixed for a given mask, so runs are bitwise reproducible.
 *
 * head_dim 256 (all backward entry points): the dK and dV accumulators of a
 * 128-row key block would fill the whole tensor memory, so two CTAs share
 * each (sequence, key/value head, key block), one per half of the head
 * dimension; each computes the full scores and dP and its half of dK, dV
 * and dQ, over 64-row query blocks.  In FA_DQ_DETERMINISTIC mode the
 * workspace then holds one counter per (batch, head, 64-row query block,
 * head-dim half, 32-dim quarter) and one work-item counter from which the
 * CTAs take their order as they start; fa_bwd_workspace_size accounts for
 * both. */
int fa_bwd_ex(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, const fa_bf16* dout,
              const float* m, const float* l, const float* D,
              float* dq_acc, fa_bf16* dk, fa_bf16* dv,
              const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
              const int32_t* cu_q_host, const int32_t* cu_kv_host,
              int batch, int total_q, int total_kv, int heads, int heads_kv, int head_dim,
              int mask, int window, float scale, int dq_mode,
              void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* fa_bwd_ex consuming the single statistic lse = m + ln(l) (as written by
 * fa_fwd_lse) instead of (m, l): P = exp(scale * S - lse).  Everything else,
 * including the workspace, is as in fa_bwd_ex. */
int fa_bwd_lse(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, const fa_bf16* dout,
               const float* lse, const float* D,
               float* dq_acc, fa_bf16* dk, fa_bf16* dv,
               const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
               const int32_t* cu_q_host, const int32_t* cu_kv_host,
               int batch, int total_q, int total_kv, int heads, int heads_kv, int head_dim,
               int mask, int window, float scale, int dq_mode,
               void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* dQ write-back (section 3, V2 applies scale to dq; section 4.2 row dQ:
 * fp32 accumulate, then bf16): dq[e] = bf16_rne(scale * dq_acc[e]) for all
 * total_q * heads * head_dim elements. */
int fa_bwd_dq_finalize(const float* dq_acc, fa_bf16* dq, int total_q, int heads,
                       int head_dim, float scale, fa_stream_t stream);

/* Bytes of the library's fixed scratch array used by fa_bwd_noalloc. */
#define FA_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)

/* The full backward (fa_bwd_preprocess -> fa_bwd in FA_DQ_ATOMIC mode ->
 * fa_bwd_dq_finalize) without any caller-provided scratch and without any
 * device allocation.  The SK-16 article has no counterpart: this is an
 * interface for callers that cannot call cudaMalloc, such as runtimes that
 * own all device memory through their own planner and give a kernel
 * library nothing but its inputs and outputs, serving loops in which an
 * allocation would stall the device, and hosts with a fixed device-memory
 * budget.  The caller passes inputs (q, k, v, o, dout, m, l, offsets) and
 * outputs (dq, dk, dv) with the layouts above; head_dim 64, 128 or 256
 * (FA_ERR_UNSUPPORTED otherwise), causal 0 or 1.  D and the fp32 dQ
 * accumulator live in one static device array of FA_NOALLOC_SCRATCH_BYTES
 * that every GPU which loads the library keeps until process exit; a
 * problem needing more (total_q * heads * (head_dim + 1) * 4 bytes,
 * rounded up) is rejected with FA_ERR_INVALID_ARG.  Every argument is
 * checked before anything is launched.  Each call looks up the array's
 * device address in the current context (cudaGetSymbolAddress), so it
 * stays valid across context switches and device resets; the first call in
 * a context loads the library's device code, so make it before any stream
 * capture.  Every call shares the array: calls whose work overlaps on the
 * GPU race, so order them on one stream.  Each call re-zeroes what must
 * start at zero. */
int fa_bwd_noalloc(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, const fa_bf16* o,
                   const fa_bf16* dout, const float* m, const float* l,
                   fa_bf16* dq, fa_bf16* dk, fa_bf16* dv,
                   const int32_t* cu_q_dev, const int32_t* cu_kv_dev,
                   const int32_t* cu_q_host, const int32_t* cu_kv_host,
                   int batch, int total_q, int total_kv, int heads, int head_dim,
                   int causal, float scale, fa_stream_t stream);

/* ------------------------------------------------------------------------
 * Paged key/value cache: the serving side of the forward above.
 *
 * Keys and values of past tokens live in pages of page_size slots, k_cache
 * and v_cache apart but laid out alike: slot s of page p, key/value head h
 * starts at element p * page_stride + s * slot_stride + h * head_stride, d
 * elements long (strides in elements, multiples of 16 bytes).  The packed
 * layout of the other entry points, [num_pages, page_size, Hkv, d], has
 * strides (page_size * Hkv * d, Hkv * d, d); [num_pages, Hkv, page_size, d]
 * and a cache that interleaves K and V pages are other strides of the same.
 * A request's tokens 0, 1, ... occupy the slots of the pages its row of the
 * block table names, in order; an entry that is no page of the cache
 * (< 0 or >= num_pages) holds no keys.  A slot's number is
 * page * page_size + place in the page.
 *
 * Device contents are not read on the host: lengths below 0 count as 0,
 * and page and slot numbers are bounds-checked on the device.
 * ------------------------------------------------------------------------ */
enum fa_kv_type {
    FA_KV_BF16 = 0,
    FA_KV_E4M3 = 1    /* 8-bit floating point, value = element * scale of the key/value head */
};

/* Places for new tokens, built on the device from the requests' lengths.
 * Request b has seq_lens[b] tokens in the cache and gets new_lens[b] more.
 * Pages it needs beyond those it holds, ceil(seq_lens / page_size), are
 * taken from free_pages in request order, from entry *free_start on
 * (free_start NULL: 0), and entered into its row of block_table (rows
 * table_stride entries apart, max_pages entries each; other entries are left
 * as they were, so the same call made again gives the same result).
 *   slots[num_tokens], positions[num_tokens]: slot and position in its
 *     request of every new token, requests in order.  Rows past the last new
 *     token (a padded batch) get slot -1, position 0.
 *   cu_new[batch+1]: offsets of the requests' new tokens (the cu_q of a
 *     following fa_fwd_* call, which takes the same offsets on the host, too);  seq_lens_out[batch] = seq_lens + new_lens;
 *   free_next[1]: the first entry of free_pages not taken.
 * A token for which the table row or the free list has no page gets slot -1
 * (and the table entry -1); *free_next > num_free tells that the list ran
 * out, cu_new[batch] > num_tokens that slots was too short (tokens past it
 * get no slot and position here; their pages are taken and entered like the
 * others').  seq_lens_out must not overlap seq_lens or new_lens, and
 * free_next not free_start; no other output may overlap an input. */
int fa_kv_plan(int32_t* block_table, long long table_stride, int max_pages,
               const int32_t* seq_lens, const int32_t* new_lens,
               const int32_t* free_pages, int num_free, const int32_t* free_start,
               int page_size, int batch, int num_tokens,
               int64_t* slots, int32_t* positions, int32_t* cu_new,
               int32_t* seq_lens_out, int32_t* free_next, fa_stream_t stream);

/* Writes the new tokens' keys and values, k and v [num_tokens, Hkv, d] bf16
 * (rows k_row_stride / v_row_stride elements apart, multiples of 8: slices
 * of a fused projection need no copy), into the cache: row t goes to
 * slots[t]; rows whose slot is outside the cache (-1) are skipped and slots
 * that no row names are left as they were.  The slots of one call must
 * differ from one another (of rows with the same slot any one may remain, or
 * parts of several), and k and v must not overlap the cache.  kv_type FA_KV_E4M3 stores
 * e4m3(x / k_scale[head]) (v_scale for v; NULL: 1), round to nearest even,
 * saturating at +-448; NaN stays NaN.  Scales: [Hkv] float32 on the device,
 * positive; NULL with FA_KV_BF16. */
int fa_kv_append(const fa_bf16* k, const fa_bf16* v, long long k_row_stride, long long v_row_stride,
                 const int64_t* slots, int num_tokens,
                 void* k_cache, void* v_cache, int kv_type, const float* k_scale, const float* v_scale,
                 long long page_stride, long long slot_stride, long long head_stride,
                 int num_pages, int page_size, int heads_kv, int head_dim, fa_stream_t stream);

/* Bytes of device workspace fa_decode needs (an upper bound over all
 * lengths).  Returns 0 and sets fa_last_error() on bad arguments. */
size_t fa_decode_workspace_size(int batch, int heads, int heads_kv, int head_dim);

/* Attention of one new token per request over the cache: q [batch, H, d]
 * bf16 (rows q_row_stride elements apart, a multiple of 8), o [batch, H, d]
 * bf16 contiguous, lse [batch, H] float32 (may be NULL), the values
 * fa_fwd_lse gives for a query at position seq_lens[b] - 1 that sees keys
 * [max(0, seq_lens[b] - window), seq_lens[b]) (window 0: all).  The new
 * token's own key and value are in the cache already (fa_kv_append) and
 * count in seq_lens.  Lengths are clamped to max_pages * page_size.  Query
 * head h reads key/value head h / (H / Hkv), at most 1024 of them each.  A row that sees no key gets
 * o = 0, lse = -inf.  Contents of slots that are not seen do not matter
 * (NaN included); an infinite value that is seen gives an infinite element
 * (NaN beside one of the other sign, or where its weight underflows to 0).
 * o must not overlap q.  workspace: fa_decode_workspace_size() bytes, 16-byte
 * aligned, contents arbitrary; calls whose work overlaps on the GPU need one
 * each.  Results do not depend on timing: the same call gives the same bits. */
int fa_decode(const fa_bf16* q, long long q_row_stride,
              const void* k_cache, const void* v_cache, int kv_type, const float* k_scale, const float* v_scale,
              long long page_stride, long long slot_stride, long long head_stride,
              int num_pages, int page_size, const int32_t* block_table, long long table_stride, int max_pages,
              const int32_t* seq_lens, int batch, int heads, int heads_kv, int head_dim,
              int window, float scale, fa_bf16* o, float* lse,
              void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* Bytes of device workspace fa_extend needs, whatever the sizes.  Returns 0 and
 * sets fa_last_error() on bad arguments. */
size_t fa_extend_workspace_size(int head_dim);

/* Attention of several new tokens per request over the cache (a chunk of a
 * prompt, drafted tokens to be verified, single tokens, or a mixture): q
 * [num_tokens, H, d] bf16 (rows q_row_stride elements apart, a multiple of 8),
 * request b's rows are cu_new[b] to cu_new[b+1], cu_new [batch+1] int32 and
 * seq_lens [batch] int32 on the device as fa_kv_plan writes them: seq_lens[b]
 * keys with the new tokens' own, which are in the cache already
 * (fa_kv_append, fa_qk_rope_append).  Token i of n is at position
 * p = seq_lens[b] - n + i and sees the keys [max(0, p - window + 1), p] (window 0:
 * [0, p]).  o [num_tokens, H, d] bf16 contiguous, lse [num_tokens, H] float32
 * (may be NULL): for one new token per request, what fa_decode gives up to
 * rounding.  Lengths are clamped to max_pages * page_size, offsets to
 * num_tokens (a request cut off by num_tokens keeps its positions).  A row that
 * sees no key, and one that belongs to no request (from cu_new[batch] on; a
 * padded batch), gets o = 0, lse = -inf.  Contents of slots that no row of a
 * request sees do not matter (NaN included); a value that is not finite and that
 * some of a request's rows see may make NaN of others' outputs (0 times it), as
 * in fa_fwd_*.  The weights exp(x - r), where a row's r is at most 10.4 below its
 * largest x, are rounded to bf16 beside a bf16 cache (as in fa_fwd_*; fa_decode
 * keeps 16 bits of them), to fp16 beside an e4m3 one; sums are fp32, so
 * values up to 2^113 over the number of keys cannot overflow.  o must not
 * overlap q.  workspace: 16-byte aligned, contents arbitrary; calls whose work
 * overlaps on the GPU need one each.  Results do not depend on timing: the same
 * call gives the same bits.  Waits inside are bounded: fa_check_device_status
 * reports one that ran out. */
int fa_extend(const fa_bf16* q, long long q_row_stride,
              const void* k_cache, const void* v_cache, int kv_type, const float* k_scale, const float* v_scale,
              long long page_stride, long long slot_stride, long long head_stride,
              int num_pages, int page_size, const int32_t* block_table, long long table_stride, int max_pages,
              const int32_t* seq_lens, const int32_t* cu_new, int batch, int num_tokens,
              int heads, int heads_kv, int head_dim, int window, float scale, fa_bf16* o, float* lse,
              void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotation of queries and keys by their positions, with an optional norm per
 * head: what stands between a projection and fa_fwd_* or the cache.
 *
 * A head x of d values at position p becomes
 *   n = x / sqrt(mean(x^2) + eps) * weight     (n = x where the weight is NULL)
 *   y_a = mscale (n_a cos t_i - n_b sin t_i),  y_b = mscale (n_b cos t_i + n_a sin t_i)
 * for the pairs i of its first rotary_dim values, t_i = p * theta_i; the others
 * are n.  Computed in fp32, rounded once.
 *   rotary_dim  a multiple of 16 from 0 (the norm alone) to d
 *   positions   [num_tokens] int32 on the device (fa_kv_plan's), any value
 *   freqs       [rotary_dim / 2] on the device: theta_i / (2 pi) mod 1 as a
 *               64-bit fixed-point fraction of a turn (rounded times 2^64).  The
 *               product with a position loses nothing, whatever the position: an
 *               angle is off by the frequency's own rounding times the position
 *               and by 2^-32 turns.  Stretched positions are other frequencies; mscale carries
 *               a factor of the outputs that goes with them (1 otherwise).
 *   weights     [d] of weight_type on the device, or NULL: no norm of this tensor
 * q [num_tokens, H, d], k [num_tokens, Hkv, d] bf16, rows row_stride elements
 * apart (multiples of 8: slices of a fused projection need no copy), 16-byte
 * aligned; H or Hkv may be 0 (the tensor may then be NULL).  d 64, 128 or 256.
 * The gradient, and many rows into a cache, wait inside for copies, bounded:
 * fa_check_device_status reports a wait that ran out.
 * ------------------------------------------------------------------------ */
enum fa_rope_layout {
    FA_ROPE_HALF = 0,         /* pairs (i, i + rotary_dim / 2) */
    FA_ROPE_INTERLEAVED = 1   /* pairs (2i, 2i + 1) */
};
enum fa_weight_type {
    FA_WEIGHT_BF16 = 0,
    FA_WEIGHT_F32 = 1
};

/* q_out and k_out, shaped like q and k with row strides of their own.  q_out
 * may be q (same stride), k_out k; otherwise no output may overlap an input or
 * the other output. */
int fa_qk_rope(const fa_bf16* q, const fa_bf16* k, long long q_row_stride, long long k_row_stride,
               const int32_t* positions, const uint64_t* freqs, int rotary_dim, int layout, float mscale,
               const void* q_weight, const void* k_weight, int weight_type, float eps,
               int num_tokens, int heads, int heads_kv, int head_dim,
               fa_bf16* q_out, fa_bf16* k_out, long long q_out_row_stride, long long k_out_row_stride,
               fa_stream_t stream);

/* Bytes of device workspace fa_qk_rope_bwd needs where a weight is given.
 * Returns 0 and sets fa_last_error() on bad arguments. */
size_t fa_qk_rope_bwd_workspace_size(int head_dim);

/* Gradient of fa_qk_rope.  dq_out, dk_out: gradients of its outputs.  q, k: its
 * inputs, read only where the tensor has a weight (may be NULL otherwise).
 * Outputs: dq, dk (dq may be dq_out with the same stride, dk dk_out), and where
 * a weight is given its gradient dq_weight, dk_weight [d] float32 (whatever the
 * weight's type), overwritten.  The norm's factor is worked out again from q
 * and k.  Sums over rows go in a fixed order: same bits on every call.
 * workspace: needed with a weight, 16-byte aligned, contents arbitrary; calls
 * whose work overlaps on the GPU need one each. */
int fa_qk_rope_bwd(const fa_bf16* dq_out, const fa_bf16* dk_out, long long dq_out_row_stride,
                   long long dk_out_row_stride, const fa_bf16* q, const fa_bf16* k, long long q_row_stride,
                   long long k_row_stride, const int32_t* positions, const uint64_t* freqs, int rotary_dim,
                   int layout, float mscale, const void* q_weight, const void* k_weight, int weight_type, float eps,
                   int num_tokens, int heads, int heads_kv, int head_dim, fa_bf16* dq, fa_bf16* dk,
                   long long dq_row_stride, long long dk_row_stride, float* dq_weight, float* dk_weight,
                   void* workspace, size_t workspace_bytes, fa_stream_t stream);

/* fa_qk_rope and fa_kv_append in one pass: q is rotated (and normed) into
 * q_out, k likewise into the cache, v goes into the cache as it is.  Cache,
 * slots (rows whose slot is outside the cache are skipped in the cache, their
 * q_out row is written) and scales as in fa_kv_append.  To an e4m3 cache a
 * rotated key is rounded once, e4m3(y / k_scale[head]) of y in fp32, where y times
 * the scale's fp32 reciprocal stands for the quotient (next to the border of two
 * 8-bit values it may fall on the other side); values are stored as
 * fa_kv_append stores them.  q, k, v must not overlap the cache or q_out
 * (which may be q with the same stride). */
int fa_qk_rope_append(const fa_bf16* q, const fa_bf16* k, const fa_bf16* v, long long q_row_stride,
                      long long k_row_stride, long long v_row_stride, const int32_t* positions,
                      const uint64_t* freqs, int rotary_dim, int layout, float mscale, const void* q_weight,
                      const void* k_weight, int weight_type, float eps, int num_tokens, int heads,
                      fa_bf16* q_out, long long q_out_row_stride, const int64_t* slots,
                      void* k_cache, void* v_cache, int kv_type, const float* k_scale, const float* v_scale,
                      long long page_stride, long long slot_stride, long long head_stride,
                      int num_pages, int page_size, int heads_kv, int head_dim, fa_stream_t stream);

/* Diagnostic (the pages have no counterpart): launches a block for every
 * status word (the backward's, the forward's, fa_extend's, the rotation's) that
 * waits, through the same bounded mbarrier wait the kernels use, on a
 * barrier nothing arrives on.  After its own short limit (1 s; the
 * kernels' waits give up after 20 s) it records
 * FA_ERR_TIMEOUT in the status word and returns; nothing faults and
 * the context stays usable.  The next fa_check_device_status on `stream`
 * then returns FA_ERR_TIMEOUT.  Lets a caller test its handling of a timed
 * out kernel. */
int fa_selftest_wait_timeout(fa_stream_t stream);

/* Synchronises `stream`, then reads and clears the device status words
 * that bounded waits set.  Returns FA_OK, FA_ERR_TIMEOUT or FA_ERR_CUDA; the
 * message names every call whose word was set.
 * The outputs of the kernels launched before it are complete and valid
 * only when it returns FA_OK: after FA_ERR_TIMEOUT some CTAs stopped early
 * and their outputs (dq_acc, dk, dv; o, m, l; fa_extend's o and lse; dq, dk and
 * the weights' gradients of fa_qk_rope_bwd; q_out and the cache's slots of
 * fa_qk_rope_append) may be partial. */
int fa_check_device_status(fa_stream_t stream);

/* Message describing the last error returned on the calling thread
 * (empty string after success), in the manner of the argument validators
 * of the PyPTO block_attn_res_impl.py page (_validate_forward_inputs:
 * which argument, what was expected, what was given) and of the JAX
 * wrapper's check_layout.  The pointer stays valid until the next call on
 * the same thread. */
const char* fa_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FABWD_H */
