/*
 * verify_attn.h - C ABI of the GB300 (sm_103a) target-verify attention library.
 *
 * The operation (sglang PR 36330 digest, "Motivation" and "Key code excerpts"):
 * speculative decoding's target-verify step runs a short multi-token query
 * (1-4 draft tokens per sequence, a GQA group of query heads per KV head,
 * head_dim 256) causally over a long paged KV cache (page size 16, FP8 E4M3
 * with per-tensor k/v descale, or BF16). The work of each (sequence, KV head)
 * is split across KV segments and the per-segment partial results are merged
 * by a log-sum-exp segment reduction (same digest, "Implementation breakdown"
 * item 1: the main kernel plus its "reduce segments" kernel).
 *
 * For sequence b with L = cu_seqlens_q[b+1] - cu_seqlens_q[b] draft tokens and
 * S = seqused_k[b] cached tokens (S counts the draft tokens too: the digest's
 * call passes seq_lens + max_q_len), query head h of draft token t reads KV
 * head h / (Hq/Hkv) and sees keys [0, S - L + t]:
 *
 *   out[cu[b]+t, h, :] = softmax(softmax_scale * k_descale * q . K^T) (v_descale * V)
 *
 * A row whose token sees no key (S - L + t < 0) is written as 0.
 *
 * Conventions shared by every entry point
 *  - Every tensor argument is a va_tensor: a DEVICE pointer plus shape and
 *    strides counted in elements. The library never keeps a pointer after the
 *    call returns and never frees caller memory.
 *  - Launches are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream). No entry point synchronises, reads device memory from
 *    the host, or depends on device values for its launch shape: only the
 *    host integers max_seqlen_q / max_seqlen_k (upper bounds) size the grid.
 *  - Errors are returned as va_status before anything is launched; nothing
 *    aborts or throws across the ABI. VA_ERR_CUDA reports a failed launch or
 *    allocation (the CUDA error is left for cudaGetLastError to inspect).
 *  - Device-side preconditions (seqused_k[b] <= block_table width * 16,
 *    0 <= cu_seqlens_q deltas <= max_seqlen_q, cu_seqlens_q[B] <= total_q,
 *    block-table entries < num_blocks) are the caller's. Violations never
 *    cause an out-of-bounds access (lengths are clamped, bad page ids read as
 *    zeros) but the affected output rows are unspecified.
 */
#ifndef VERIFY_ATTN_H
#define VERIFY_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. FP8_E4M3 is OCP E4M3 "FN" (torch.float8_e4m3fn). */
typedef enum va_dtype {
  VA_BF16 = 0,
  VA_FP8_E4M3 = 1,
  VA_INT32 = 2,
  VA_FP32 = 3
} va_dtype;

/* A strided view of device memory. Strides are in elements. */
typedef struct va_tensor {
  void* data;
  int32_t dtype;      /* va_dtype */
  int32_t ndim;       /* 1..4 */
  int64_t shape[4];
  int64_t stride[4];
} va_tensor;

typedef enum va_status {
  VA_OK = 0,
  VA_ERR_NULL = 1,         /* a required pointer or descriptor is NULL */
  VA_ERR_SHAPE = 2,        /* shapes disagree with each other */
  VA_ERR_DTYPE = 3,        /* an element type is not the one required */
  VA_ERR_UNSUPPORTED = 4,  /* well-formed but outside what the kernels cover */
  VA_ERR_WORKSPACE = 5,    /* caller workspace missing or too small */
  VA_ERR_CUDA = 6,         /* a CUDA runtime call or launch failed */
  VA_ERR_LAYOUT = 7        /* a stride or alignment the kernels cannot read */
} va_status;

/* Launch plan chosen by the host heuristic (pure host arithmetic). */
typedef struct va_plan {
  int32_t tile_keys;       /* keys per pipeline tile of the main kernel */
  int32_t num_splits;      /* CTAs of the main kernel; each takes an equal share
                              of the batch's key tiles (its KV segments) */
  int32_t max_rows;        /* packed rows per (sequence, KV head) = G * max_seqlen_q */
  int32_t num_work;        /* B * Hkv (sequence, KV head) pairs */
  int32_t kernel;          /* main-kernel layout the launch will use: 1 = Q in
                              shared memory (BF16; FP8 batches of fewer than 16
                              tiles per CTA; any variant option), 2 = FP8 with
                              Q and P in tensor memory and a deeper K ring */
  int32_t reserved;
  int64_t workspace_bytes; /* scratch the split-KV partials need */
} va_plan;

/*
 * verify_attn - the operation described above.
 *
 * q            [total_q, Hq, 256] BF16; innermost stride 1, rows 16-byte aligned.
 * k_cache      [num_blocks, 16, Hkv, 256] FP8_E4M3 or BF16; innermost stride 1,
 * v_cache      the other strides multiples of 16 bytes. Same dtype and shape.
 *              Token-major pages with the heads of a token interleaved
 *              (sglang PR 36330 digest, unit test: key/value shape
 *              (num_blocks, block_size, num_kv_heads, head_size)).
 * block_table  [B, W] INT32, logical page -> physical page, W*16 >= max_seqlen_k.
 *              Only the first ceil(seqused_k[b]/16) entries of row b are read.
 * cu_seqlens_q [B+1] INT32 contiguous, prefix sums of the draft-token counts.
 * seqused_k    [B] INT32 contiguous, cached tokens per sequence incl. drafts.
 * max_seqlen_q host upper bound of the draft-token counts; 1 <= max_seqlen_q
 *              and (Hq/Hkv) * max_seqlen_q <= 64.
 * max_seqlen_k host upper bound of seqused_k (the digest passes
 *              page_table.shape[1] * page_size; sglang PR 30105 digest,
 *              "Key code excerpts").
 * softmax_scale  multiplies the logits (head_dim ** -0.5 in the pages).
 * k_descale, v_descale  [1] FP32 device scalars or NULL (= 1.0): the
 *              dequantised value is stored value * descale (sglang PR 34517
 *              digest, "Key code excerpts": qk *= sm_scale * k_scale).
 * out          [total_q, Hq, 256] BF16, written in place (round to nearest
 *              even from fp32); may not alias any input.
 * stream       cudaStream_t.
 *
 * Scratch: a per-device workspace owned by the library, grown (cudaMalloc) on
 * demand and kept until process exit. Because growing allocates, make the
 * first call with the largest shape before capturing a CUDA graph, or use
 * verify_attn_ex with a caller workspace. Calls that share the library
 * workspace must be ordered on one stream (concurrent streams race on it).
 * verify_attn_last_device_error(NULL, ...) reports a bounded wait that ran
 * out in a call made with it.
 */
va_status verify_attn(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                      const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                      const va_tensor* seqused_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                      float softmax_scale, const va_tensor* k_descale,
                      const va_tensor* v_descale, va_tensor* out, void* stream);

/*
 * verify_attn_ex - verify_attn with a caller-owned workspace and an optional
 * forced split count. Not on the pages: it exists so a caller can own all
 * memory (graph capture, allocator integration) and so tests can force the
 * number of KV segments.
 *
 * workspace        device pointer, 256-byte aligned, at least
 *                  verify_attn_workspace_size(...) bytes for the same shapes
 *                  and num_splits; NULL with workspace_bytes == 0 is valid only
 *                  when that size is 0.
 * num_splits       0 = the heuristic's choice; > 0 forces the main kernel's
 *                  CTA count (clamped to the number of key tiles it could have).
 * event_after_main NULL, or a cudaEvent_t recorded on `stream` between the
 *                  main and the merge kernel (lets a caller time the main
 *                  kernel alone with CUDA events on the launching stream).
 * The workspace holds no state between calls, except its status word (the
 * first 4 bytes; zero it before first use), which a bounded wait that runs out
 * sets and verify_attn_last_device_error reads and clears.
 */
va_status verify_attn_ex(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                         const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                         const va_tensor* seqused_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                         float softmax_scale, const va_tensor* k_descale,
                         const va_tensor* v_descale, va_tensor* out, void* workspace,
                         size_t workspace_bytes, int32_t num_splits, void* event_after_main,
                         void* stream);

/*
 * verify_attn_check - validation only: the same checks verify_attn runs before
 * launching, as a pure host function (no CUDA call; device pointers are only
 * tested for NULL and alignment). Turns the shape gate of sglang PR 36330
 * digest ("Key code excerpts", aiter_backend.py) and the rejections of sglang
 * PR 34517 digest ("Implementation breakdown": can_handle) into status codes.
 */
va_status verify_attn_check(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                            const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                            const va_tensor* seqused_k, int32_t max_seqlen_q,
                            int32_t max_seqlen_k, const va_tensor* k_descale,
                            const va_tensor* v_descale, const va_tensor* out);

/*
 * verify_attn_plan - the host launch heuristic as a pure function (no CUDA
 * call). Picks the tile size and the number of KV segments (main-kernel CTAs)
 * from the batch, the KV-length bound and the SM count, so that short-query
 * batches fill every SM (sglang PR 36330 digest, "Implementation breakdown"
 * item 1: 8-64 segments for CU parallelism; sglang PR 30105 digest,
 * "Implementation breakdown" item 3: split-KV restores occupancy for short
 * queries).
 *
 * num_sms        SMs of the target device (> 0).
 * force_splits   0 = heuristic; > 0 = this many (clamped as in verify_attn_ex).
 * Returns VA_ERR_NULL if plan is NULL, VA_ERR_UNSUPPORTED for arguments out
 * of range.
 */
va_status verify_attn_plan(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads,
                           int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t kv_dtype,
                           int32_t num_sms, int32_t force_splits, va_plan* plan);

/*
 * verify_attn_workspace_size - bytes of workspace verify_attn_ex needs for
 * these shapes on the current device with num_splits (0 = heuristic). Queries
 * the current device's SM count (a CUDA call); returns 0 on error.
 */
size_t verify_attn_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t num_q_heads,
                                  int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t kv_dtype,
                                  int32_t num_splits);

/*
 * va_options - variants of the generic attention that the pages pass through
 * (sglang PR 30105 digest, "Key code excerpts": unified_attention(...,
 * window_size, softcap, sinks)). All off is window_left = -1, softcap = 0,
 * sinks = NULL.
 *  window_left  sliding window: the draft token at position i = S - L + t
 *               sees keys [i - window_left, i] (the pages' window_size =
 *               (sliding_window_size - 1, 0)); -1 = no window. Block-table
 *               pages holding only keys before every token's window are never
 *               read, so a sliding-window page table need not map them.
 *  softcap      > 0: each logit s = softmax_scale * k_descale * q.k becomes
 *               softcap * tanh(s / softcap) before masking; 0 = off.
 *  sinks        [Hq] fp32, contiguous, or NULL: a per-query-head logit
 *               (natural-log units) that joins that head's softmax normaliser
 *               with a zero value vector. A row that sees no key is still 0.
 */
typedef struct va_options {
  int32_t window_left;
  float softcap;
  const va_tensor* sinks;
} va_options;

/*
 * verify_attn_opt - verify_attn with the variants above.
 *  opts       NULL means all variants off (then this is verify_attn_ex).
 *  workspace  a caller workspace as for verify_attn_ex, or NULL to use the
 *             library's own per-device workspace as verify_attn does (which
 *             may then allocate, so not during stream capture).
 * Other arguments, layouts and results are those of verify_attn_ex; num_splits
 * 0 lets the heuristic pick (with a window it counts only the window's tiles).
 * Returns VA_ERR_SHAPE / VA_ERR_DTYPE / VA_ERR_NULL / VA_ERR_UNSUPPORTED for
 * bad options before launching (window_left < -1, softcap negative or not
 * finite, sinks not fp32 [Hq] contiguous).
 */
va_status verify_attn_opt(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                          const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                          const va_tensor* seqused_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                          float softmax_scale, const va_tensor* k_descale,
                          const va_tensor* v_descale, va_tensor* out, const va_options* opts,
                          void* workspace, size_t workspace_bytes, int32_t num_splits,
                          void* stream);

/*
 * verify_attn_noalloc - verify_attn for callers that cannot allocate device
 * memory. The pages have no counterpart; this is a library addition.
 *
 * Who needs it: code that must not call cudaMalloc when it runs attention,
 * e.g. a serving runtime that sized its GPU memory pool at start-up and
 * forbids later allocations (cudaMalloc synchronises the device and
 * fragments the pool), or an allocator callback that must not re-enter the
 * allocator. verify_attn would grow its workspace with cudaMalloc;
 * verify_attn_ex needs the caller to allocate one.
 *
 * Arguments, layouts, results and errors are those of verify_attn. The
 * split-KV partials go to a fixed array of VERIFY_ATTN_NOALLOC_SCRATCH_BYTES
 * compiled into the library; every GPU that loads the library holds that
 * array until the process exits. Nothing is allocated or freed by this call.
 *  - Returns VA_ERR_WORKSPACE, before launching anything, when the shapes
 *    need more partial storage than the array holds (it needs about
 *    (B*Hkv + SMs) * (Hq/Hkv) * max_seqlen_q KiB).
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress, with that device current) and keeps it; make
 *    that first call before any stream capture.
 *  - Every call on a device shares the one array and leaves its contents
 *    behind. Nothing in it needs to start at zero, but calls that overlap on
 *    the GPU (different streams, or different host threads) race on it:
 *    order them on one stream.
 *  - The array's first word is the status word of the kernels' bounded
 *    waits, shared by every call on the device. This call never clears it;
 *    verify_attn_last_device_error(NULL, ...) reads and clears it (and
 *    synchronises the stream it is given, so call it between batches).
 */
#define VERIFY_ATTN_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

va_status verify_attn_noalloc(const va_tensor* q, const va_tensor* k_cache,
                              const va_tensor* v_cache, const va_tensor* block_table,
                              const va_tensor* cu_seqlens_q, const va_tensor* seqused_k,
                              int32_t max_seqlen_q, int32_t max_seqlen_k, float softmax_scale,
                              const va_tensor* k_descale, const va_tensor* v_descale,
                              va_tensor* out, void* stream);

/*
 * verify_attn_block_table_from_indptr - the block table and KV lengths of a
 * batch given in flat token-slot form. This is the draft-extend pass of the
 * sglang PR 30105 digest ("Fix 2: draft_extend_v2 re-routed to
 * unified_attention"): it builds a 2D page table from its flat metadata, takes
 * each sequence's KV length as the difference of consecutive kv_indptr
 * entries, and then runs the same split-KV attention as target verify. After
 * this call, verify_attn on (block_table, seqused_k) with
 * max_seqlen_k = width * 16 is that attention.
 *
 * Arguments (all device memory, all int32):
 *  kv_indptr    [B+1], contiguous. Sequence b's tokens are kv_indices
 *               [kv_indptr[b], kv_indptr[b+1]).
 *  kv_indices   [nnz], contiguous. The KV-cache token slot of every token,
 *               slot = page * 16 + position in the page.
 *  block_table  [B, width], any non-negative strides; written. Entry p of
 *               row b is the page holding sequence b's tokens [16p, 16p + 16),
 *               i.e. the page of the first of those slots. Entries past the
 *               sequence's last page are set to pad_page.
 *  seqused_k    [B], any stride; written with kv_indptr[b+1] - kv_indptr[b].
 *  status       optional (NULL: not reported), one int32. The kernel ORs in:
 *                 1  a page's slots are not one page in order: the first slot
 *                    is not a multiple of 16, or the next ones are not
 *                    consecutive. The entry still names the first slot's page.
 *                 2  a sequence has more than width pages; its row keeps the
 *                    first width pages.
 *                 4  kv_indptr[b] is negative, decreases, or passes nnz; that
 *                    row is all pad_page and its length 0.
 *               The kernel never clears it.
 *
 * Behaviour:
 *  - One launch, asynchronous on stream.
 *  - Returns before launching: VA_ERR_NULL, VA_ERR_DTYPE, VA_ERR_SHAPE; VA_ERR_LAYOUT
 *    for a strided kv_indptr / kv_indices; VA_ERR_UNSUPPORTED for more than 65535
 *    sequences.
 *  - Returns VA_ERR_CUDA if the launch fails.
 */
va_status verify_attn_block_table_from_indptr(const va_tensor* kv_indptr,
                                              const va_tensor* kv_indices, va_tensor* block_table,
                                              va_tensor* seqused_k, int32_t pad_page,
                                              int32_t* status, void* stream);

/*
 * verify_attn_mla - target-verify attention over an absorbed-MLA latent cache.
 *
 * The grouped-head shared-KV verify kernel of the sglang PR 34517 digest
 * ("Implementation breakdown" item 1, the verify_mla.py excerpt) also serves
 * an absorbed-MLA layout: the single TP-local KV head is the MLA latent,
 * NOPE_DIM latent columns plus PE_DIM = 64 RoPE columns, and the logits are
 * (q_nope . k_nope + q_pe . k_pe) * softmax_scale * k_scale. The values are
 * the latent columns of the same cache rows. The latent width is not on the
 * pages; this library takes NOPE_DIM = 512 (the DeepSeek-V3 / Kimi-K2 MLA
 * family). For sequence b (L draft tokens, S = seqused_k[b]) and query head h
 * of draft token t, with cache row j = [c_j | r_j] (decoded e4m3 or bf16):
 *
 *   out[cu[b]+t, h, :] = sum_j softmax_j(softmax_scale * k_descale *
 *                          (q[.., :512] . c_j + q[.., 512:] . r_j)) * v_descale * c_j
 *
 * over keys j in [0, S - L + t]; a row that sees no key is 0.
 *
 * Arguments (device memory unless stated):
 *  q            [total_q, Hq, 576] bf16: [q_nope (absorbed, 512) | q_pe (64)].
 *  kv_cache     [num_blocks, 16, 1, 576] FP8 E4M3 (OCP FN) or BF16: [latent |
 *               rope key] (the digest's tests cover both cache types, same
 *               digest, "Implementation breakdown" item 4).
 *  block_table, cu_seqlens_q, seqused_k, max_seqlen_q, max_seqlen_k,
 *  softmax_scale, k_descale, v_descale: as for verify_attn (Hkv = 1, so the
 *               group is Hq and Hq * max_seqlen_q <= 64). A cache with one
 *               scale passes it as both descales.
 *  out          [total_q, Hq, 512] bf16, written.
 *  workspace    device memory of at least verify_attn_mla_workspace_size()
 *               bytes, 256-byte aligned; NULL uses the library's per-device
 *               workspace (grown with cudaMalloc as needed).
 *  num_splits   0 = the library's choice (one CTA per SM, fewer for small
 *               batches); > 0 forces that many CTAs.
 *  event_after_main  optional cudaEvent_t (NULL: none) recorded on stream
 *               between the main kernel and the merge kernel, as in
 *               verify_attn_ex.
 *
 * Layout: innermost strides 1 and every other stride a multiple of 16 bytes;
 * q, out, kv_cache 16-byte aligned.
 * Errors (before any launch): VA_ERR_NULL, VA_ERR_SHAPE, VA_ERR_DTYPE,
 * VA_ERR_LAYOUT as for verify_attn (VA_ERR_DTYPE for a cache that is neither
 * FP8 E4M3 nor BF16); VA_ERR_UNSUPPORTED for more than one KV head, other row
 * widths or Hq * max_seqlen_q > 64;
 * VA_ERR_WORKSPACE for a short or misaligned workspace; VA_ERR_CUDA for a
 * failed launch or allocation. Device-side timeouts set the workspace
 * status word as for verify_attn_ex.
 */
va_status verify_attn_mla(const va_tensor* q, const va_tensor* kv_cache, const va_tensor* block_table,
                          const va_tensor* cu_seqlens_q, const va_tensor* seqused_k,
                          int32_t max_seqlen_q, int32_t max_seqlen_k, float softmax_scale,
                          const va_tensor* k_descale, const va_tensor* v_descale, va_tensor* out,
                          void* workspace, size_t workspace_bytes, int32_t num_splits,
                          void* event_after_main, void* stream);

/* Workspace bytes verify_attn_mla needs for these shapes on the current
 * device, for either cache type (0 if they are unsupported). */
size_t verify_attn_mla_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t max_seqlen_q,
                                      int32_t max_seqlen_k, int32_t num_splits);

/*
 * verify_attn_partial - verify attention over one shard of each sequence's
 * keys, for splitting a sequence's KV over several parts (context
 * parallelism across ranks; a shared prefix in one cache and per-sequence
 * suffixes in another). The pages name a decode-context-parallel degree
 * (sglang PR 34517 digest, attn_dcp_size) and merge split-KV segments by log-sum-exp
 * (sglang PR 36330 digest, "reduce segments"); this entry computes one
 * shard's result and verify_attn_merge_partials combines shards. The
 * exchange of shard results between GPUs is the caller's.
 *
 * A shard holds the keys of global positions [o_b, o_b + S_b) of sequence b,
 * reached through its own block_table row (S_b = seqused_k[b]). With
 * E_b = kv_extent[b] = (the sequence's total keys) - o_b, draft token t of L
 * sees the shard's local keys j <= E_b - L + t (and j < S_b). NULL kv_extent
 * means E_b = S_b, the last shard (or the whole sequence).
 *
 * Arguments as verify_attn_ex, except:
 *  kv_extent  [B] int32 (nullable), contiguous; values below S_b count as S_b.
 *  o          [total_q, Hq, 256] fp32, written: the shard's attention output,
 *             normalised over the shard's visible keys, times v_descale.
 *  lse        [total_q, Hq] fp32, written: ln(sum over the visible keys of
 *             exp(softmax_scale * k_descale * q . k)); -inf (and o = 0) for a
 *             row that sees no key of the shard.
 *  workspace  as verify_attn_ex; NULL uses the library's per-device workspace.
 * The variants of verify_attn_opt are not available here. Errors as
 * verify_attn_ex (o and lse: VA_ERR_DTYPE unless fp32, VA_ERR_SHAPE, and
 * VA_ERR_LAYOUT for o rows that are not 16-byte aligned).
 */
va_status verify_attn_partial(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                              const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                              const va_tensor* seqused_k, const va_tensor* kv_extent,
                              int32_t max_seqlen_q, int32_t max_seqlen_k, float softmax_scale,
                              const va_tensor* k_descale, const va_tensor* v_descale, va_tensor* o,
                              va_tensor* lse, void* workspace, size_t workspace_bytes,
                              int32_t num_splits, void* stream);

/*
 * verify_attn_merge_partials - combines n (1..16) shard results of
 * verify_attn_partial: out = sum_i exp(lse_i - LSE) o_i with
 * LSE = ln sum_i exp(lse_i), rounded to bf16; a row whose lse are all -inf
 * is 0. o_parts and lse_parts are HOST arrays of n descriptors (fp32
 * [total_q, Hq, 256] and [total_q, Hq], device memory); out is bf16
 * [total_q, Hq, 256]. One launch on stream. Returns VA_ERR_UNSUPPORTED for n
 * outside 1..16, and the usual shape / dtype / layout errors.
 */
va_status verify_attn_merge_partials(int32_t n, const va_tensor* o_parts, const va_tensor* lse_parts,
                                     va_tensor* out, void* stream);

/*
 * va_rope - rotary position embedding of the append entry points.
 *  cos_sin      [P, rot] fp32, row p: cos of the rot / 2 angles of position p,
 *               then their sin; rot a multiple of 8, 8 <= rot <= 256 (64 on
 *               the latent path). Rows 16-byte aligned. Only a head's first
 *               rot columns turn.
 *  positions    [total_q] int32, contiguous, or NULL: each token's position
 *               is the one it is stored at, S - L + t. A position outside
 *               [0, P) is read as the nearest inside.
 *  interleaved  0: column i turns with column i + rot / 2; 1: column 2 i turns
 *               with column 2 i + 1.
 * A pair (x1, x2) becomes (x1 cos - x2 sin, x2 cos + x1 sin) in fp32, each
 * product and the sum rounded by itself.
 */
typedef struct va_rope {
  const va_tensor* cos_sin;
  const va_tensor* positions;
  int32_t interleaved;
} va_rope;

/*
 * verify_attn_append_kv - rotates a batch's new queries and keys and stores
 * its new keys and values in the paged cache: what runs before verify_attn.
 * With L = cu_seqlens_q[b+1] - cu_seqlens_q[b] new tokens of sequence b and
 * S = seqused_k[b] cached tokens (the new ones counted, as verify_attn's),
 * new token t is stored at position S - L + t, i.e. in slot (S - L + t) % 16
 * of page block_table[b, (S - L + t) / 16]. The two calls take the same
 * block_table, cu_seqlens_q and seqused_k.
 *
 *  q, q_out     [total_q, Hq, 256] bf16, or both NULL. q_out is written with
 *               the rotated q; it may be q itself (same address and strides),
 *               and may not overlap any input otherwise.
 *  k, v         [total_q, Hkv, 256] bf16; v is not rotated. q, k and v may be
 *               views of one projection's output (innermost stride 1, rows
 *               16-byte aligned).
 *  rope         NULL: k is stored as it is (then q and q_out are NULL).
 *  k_cache, v_cache  [num_blocks, 16, Hkv, 256] FP8_E4M3 or BF16, as verify_attn
 *               reads them; written in place.
 *  k_descale, v_descale  [1] fp32 or NULL (= 1.0): the stored value is
 *               value / descale, rounded once from fp32 to nearest even (e4m3:
 *               saturating at 448; NaN stays NaN).
 *  k_scales, v_scales  [num_blocks, Hkv] fp32, any positive strides, or both
 *               NULL: the cache is page-scaled (FP8_E4M3 only, no descales), as
 *               verify_attn_scaled reads it: value = code * scales[page, head].
 *               Written in place. Per page and KV head that gets new tokens:
 *               need = the smallest 2^e, -64 <= e <= 64, with max|new| <=
 *               448 * 2^e (NaN ignored). If the page's slot 0 is among the new
 *               tokens its scale becomes need; otherwise the page holds older
 *               tokens, its scale (read as clamped to [2^-64, 2^64]) becomes the
 *               larger of itself and need, and where it grows the older tokens'
 *               codes are rounded to it (exact between powers of two, except
 *               below e4m3's normal range). Slots behind the new tokens are
 *               left as they are.
 *
 * What is written (q_out, the caches, the scales) has a place of its own for
 * every element: in some order of the dimensions each stride is at least what the
 * inner ones span (else VA_ERR_LAYOUT). k_cache and v_cache (k_scales and
 * v_scales) may be interleaved views of one tensor, not the same view
 * (VA_ERR_LAYOUT), and share no element.
 * Tokens at negative positions (L > S) are neither stored nor rotated. Rows of
 * q_out behind the last sequence are left as they were. Block-table entries
 * outside [0, num_blocks) and positions past the table's width store nothing.
 * Two sequences of a call may not append to the same page.
 *
 * One launch, asynchronous on stream; no workspace, no allocation, capturable.
 * Errors before launching: VA_ERR_NULL (also one of q / q_out, or of k_scales /
 * v_scales, without the other, or q without rope), VA_ERR_SHAPE, VA_ERR_DTYPE (also page scales
 * over a BF16 cache), VA_ERR_LAYOUT, VA_ERR_UNSUPPORTED (head_dim other than
 * 256, pages other than 16, rot out of range, descales beside page scales,
 * more heads than a grid holds: 2 Hkv + Hq / 4 > 65535); VA_ERR_CUDA for a failed
 * launch.
 */
va_status verify_attn_append_kv(const va_tensor* q, const va_tensor* k, const va_tensor* v,
                                const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                const va_tensor* seqused_k, const va_rope* rope,
                                const va_tensor* k_descale, const va_tensor* v_descale,
                                va_tensor* k_scales, va_tensor* v_scales, va_tensor* q_out,
                                va_tensor* k_cache, va_tensor* v_cache, void* stream);

/*
 * va_norm - norms of queries and keys over each head's 256 columns, ahead of the
 * rotation: x becomes x / sqrt(mean(x^2) + eps) * (weight + offset), in fp32, not
 * rounded before the rotation.
 *  q_weight, k_weight  [256] bf16 or fp32, contiguous, 16-byte aligned; NULL: queries
 *               (keys) are not normalised.
 *  eps          >= 0, finite.   offset  finite: 1 for weights stored as their
 *               difference from 1, else 0.
 */
typedef struct va_norm {
  const va_tensor* q_weight;
  const va_tensor* k_weight;
  float eps;
  float offset;
} va_norm;

/*
 * verify_attn_append_kv_norm - verify_attn_append_kv with norms of the queries and
 * keys in the same pass: q_out, the keys stored and a page's scale of keys are those of
 * the normalised and rotated values. norm NULL: verify_attn_append_kv. With a q_weight,
 * rope may be NULL (queries normalised only); a q_weight without q is VA_ERR_NULL. Errors
 * of the weights: VA_ERR_DTYPE, VA_ERR_SHAPE, VA_ERR_LAYOUT, VA_ERR_NULL; VA_ERR_UNSUPPORTED
 * for eps or offset out of range. Otherwise as verify_attn_append_kv, in one launch.
 */
va_status verify_attn_append_kv_norm(const va_tensor* q, const va_tensor* k, const va_tensor* v,
                                     const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                     const va_tensor* seqused_k, const va_norm* norm, const va_rope* rope,
                                     const va_tensor* k_descale, const va_tensor* v_descale, va_tensor* k_scales,
                                     va_tensor* v_scales, va_tensor* q_out, va_tensor* k_cache,
                                     va_tensor* v_cache, void* stream);

/*
 * verify_attn_append_mla - the same for a latent cache (verify_attn_mla): new
 * token t's row is [latent | rotated k_pe].
 *
 *  q_pe, q_pe_out  [total_q, Hq, 64] bf16, or both NULL: the queries' rope
 *               parts. q_pe_out is usually the columns [512, 576) of the q that
 *               verify_attn_mla takes, and q_pe may be that same view.
 *  latent       [total_q, 512] bf16;  k_pe  [total_q, 64] bf16 (views of one
 *               projection's output are fine).
 *  rope         cos_sin [P, 64]; NULL: k_pe is stored as it is.
 *  kv_cache     [num_blocks, 16, 1, 576] FP8_E4M3 or BF16, written in place.
 *  descale      [1] fp32 or NULL: stored value = value / descale.
 *  scales       [num_blocks, 1] fp32 or NULL: one scale a page for the whole
 *               row, by the rule of verify_attn_append_kv; read by
 *               verify_attn_mla_scaled.
 * Otherwise as verify_attn_append_kv.
 */
va_status verify_attn_append_mla(const va_tensor* q_pe, const va_tensor* latent, const va_tensor* k_pe,
                                 const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                 const va_tensor* seqused_k, const va_rope* rope,
                                 const va_tensor* descale, va_tensor* scales, va_tensor* q_pe_out,
                                 va_tensor* kv_cache, void* stream);

/* num_splits of the page-scaled calls: see verify_attn_scaled. */
#define VA_LIBRARY_STATUS (1 << 30)

/*
 * verify_attn_scaled - verify attention over a page-scaled e4m3 cache: a key's
 * stored codes stand for code * k_scales[page, head], a value's for
 * code * v_scales[page, head] (verify_attn_append_kv writes such a cache).
 * Otherwise the operation of verify_attn_opt:
 *
 *   s_j = softmax_scale * k_scales[p_j, h] * q . K_j   (then soft cap, mask, window)
 *   out = sum_j softmax(s)_j * v_scales[p_j, h] * V_j,  p_j = key j's page
 *
 *  k_cache, v_cache  [num_blocks, 16, Hkv, 256] FP8_E4M3.
 *  k_scales, v_scales  [num_blocks, Hkv] fp32, any positive strides; interleaved
 *               ([num_blocks, Hkv, 2]) a page's two lie in one sector. Read as
 *               clamped to [2^-64, 2^64] (NaN as 2^-64), so a scale of 0 makes
 *               values of at most 448 * 2^-64. Only the scales of pages that
 *               are read for their keys are read.
 *  opts         NULL: no window, soft cap or sinks.
 *  workspace    as verify_attn_ex (same size: verify_attn_workspace_size with
 *               VA_FP8_E4M3), or NULL to use the library's own per-device workspace,
 *               whose calls must be ordered on one stream; during stream
 *               capture NULL is refused (VA_ERR_WORKSPACE).
 *  num_splits   0: the library's choice, which for small batches is one cluster of
 *               up to 8 CTAs per (sequence, KV head) that joins its partial results
 *               on chip, without a merge kernel; > 0 forces the split over that many
 *               CTAs. The choice goes by max_seqlen_k, the lengths being on the
 *               device: with a bound far above them (the capacity, 32K and more for
 *               two sequences of 1K keys) it is the split, 42 us where clusters take
 *               8.2 (latent 45 and 10). With VA_LIBRARY_STATUS added a wait that runs out is reported
 *               by verify_attn_last_device_error(NULL, ...) instead of the
 *               workspace's status word: for a workspace that is given back behind
 *               the call.
 *  event_after_main  as verify_attn_ex; with clusters, behind the only kernel.
 * Accuracy, with w a key's softmax weight times its page's V scale:
 *  - The keys of a sequence are taken in blocks of 32 from its start on. w enters
 *    the product with V to 8 bits while it is within 2^-14 of its block's largest,
 *    and in steps of at most 2^-21 of that one below. Blocks do not limit each other while
 *    their largest w lie within 2^-115 of the row's.
 *  - The normaliser is a sum in fp32; it counts a key while its w is within
 *    2^-126 of the row's largest.
 *  - Q enters the logits as two e4m3 terms, scaled by the row's largest |q|: 8
 *    bits, in steps of at most 2^-16 of that one.
 *  - Logits below 2^20 in magnitude (fp32 holds them to 2^-4 there).
 * verify_attn, its variants and verify_attn_mla over e4m3 caches are the same, with
 * one V scale for all pages.
 * Page-scaled caches are read by these two entry points and verify_attn_chunk: not by
 * verify_attn_partial (and so not over context-parallel shards),
 * verify_attn_noalloc or the draft-extend pass.
 * Errors as verify_attn_opt; VA_ERR_NULL without scales, VA_ERR_DTYPE for a
 * BF16 cache or scales that are not fp32, VA_ERR_SHAPE for scales of another
 * shape, VA_ERR_LAYOUT for a zero stride or an address off 4 bytes.
 */
va_status verify_attn_scaled(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                             const va_tensor* k_scales, const va_tensor* v_scales,
                             const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                             const va_tensor* seqused_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                             float softmax_scale, va_tensor* out, const va_options* opts,
                             void* workspace, size_t workspace_bytes, int32_t num_splits,
                             void* event_after_main, void* stream);

/*
 * verify_attn_mla_scaled - verify_attn_mla over a page-scaled e4m3 latent
 * cache: scales [num_blocks, 1] fp32, one scale a page for its whole rows, as
 * key and as value (verify_attn_append_mla writes such a cache). Workspace as
 * verify_attn_mla (NULL is refused during stream capture); scales, num_splits and
 * accuracy as verify_attn_scaled.
 */
va_status verify_attn_mla_scaled(const va_tensor* q, const va_tensor* kv_cache, const va_tensor* scales,
                                 const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                 const va_tensor* seqused_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                 float softmax_scale, va_tensor* out, void* workspace,
                                 size_t workspace_bytes, int32_t num_splits, void* event_after_main,
                                 void* stream);

/*
 * The page pool: sequences that share pages of their caches (a prompt's pages under
 * several candidates). Beside the block table [B, W] and seqused_k [B], both as the
 * attention calls take them, two int32 arrays in device memory:
 *  page_count  [B]: pages that row b holds, entries [0, page_count[b]) of its row; at
 *              least ceil(seqused_k[b] / 16), more where room was reserved.
 *  refs        [num_blocks]: rows that hold the page; 0: it is free. A page that no row
 *              may get (a padding page) has any other count.
 * All caches of a model share one pool: the table's calls run once, verify_attn_copy_pages
 * once a cache. The calls below are asynchronous on stream, capturable, one launch each,
 * without a workspace or host reads; they decide from the arrays as they are when the
 * call starts, and their results depend on nothing else. Lists are contiguous int32
 * device tensors. `status` (nullable): one int32 that VA_PG_* bits are ORed into, never
 * cleared. What a bit reports is left undone, for that sequence or entry alone:
 *  VA_PG_BAD_SEQ    a listed index outside [0, B); a child listed twice (the first counts)
 *                   or listed as a parent too
 *  VA_PG_IN_USE     a child whose row holds pages (free it first)
 *  VA_PG_NO_PAGES   not enough free pages
 *  VA_PG_ROW_FULL   more tokens than a row of the table has places for
 *  VA_PG_BAD_TABLE  a count below its tokens or past the row, a page outside the pool, or
 *                   one freed more often than it was held (its count stays 0)
 * Errors before launching: VA_ERR_NULL, VA_ERR_SHAPE, VA_ERR_DTYPE (all int32),
 * VA_ERR_LAYOUT (strided vectors; a block table whose entries overlap; a vector that is
 * written over another one).
 */
#define VA_PG_BAD_SEQ 1
#define VA_PG_IN_USE 2
#define VA_PG_NO_PAGES 4
#define VA_PG_ROW_FULL 8
#define VA_PG_BAD_TABLE 16

/*
 * verify_attn_free_pages - takes the rows of the listed sequences out of the pool: their
 * pages' refs fall by one, page_count and seqused_k become 0 (the row's entries stay as
 * they were). A sequence listed twice is freed once.
 */
va_status verify_attn_free_pages(const va_tensor* block_table, va_tensor* seqused_k, va_tensor* page_count,
                                 va_tensor* refs, const va_tensor* seqs, int32_t* status, void* stream);

/*
 * verify_attn_fork_pages - children[i], whose row holds no page, becomes a copy of
 * parents[i]: seqused_k and the pages that hold its tokens, whose refs grow by one (the
 * parent's reserved room is not shared). Nothing is copied until one of them writes: see
 * verify_attn_reserve_pages. A parent may be listed any number of times.
 */
va_status verify_attn_fork_pages(va_tensor* block_table, va_tensor* seqused_k, va_tensor* page_count,
                                 va_tensor* refs, const va_tensor* parents, const va_tensor* children,
                                 int32_t* status, void* stream);

/*
 * verify_attn_reserve_pages - pages of its own for the next new_tokens[b] tokens of every
 * sequence (0 or less: none): what runs before append. With S = seqused_k[b] and want =
 * ceil((S + new_tokens[b]) / 16), the places [S / 16, want) of row b end up holding
 * pages with refs 1: one that other rows held too is replaced (its refs fall by one, also
 * where every one of its rows replaces it), places behind page_count[b] are filled, and
 * page_count[b] becomes want if that is more. The k-th page that the call needs, in the
 * order of sequences and of places, is the k-th page with refs 0 (VA_PG_NO_PAGES: a sequence
 * gets all or none of its pages, and none if the sum up to it exceeds the free ones).
 *  src, dst   [B], written: the page whose contents sequence b's caches need copied
 *             (verify_attn_copy_pages takes the two lists), -1 for none.
 *  room       [B], written: tokens that row b has places for now, 16 * page_count[b].
 * VA_ERR_UNSUPPORTED for more than 8,192 sequences or 4,194,304 pages.
 */
va_status verify_attn_reserve_pages(va_tensor* block_table, const va_tensor* seqused_k, va_tensor* page_count,
                                    va_tensor* refs, const va_tensor* new_tokens, va_tensor* src, va_tensor* dst,
                                    va_tensor* room, int32_t* status, void* stream);

/*
 * verify_attn_copy_pages - page dst[i] of a cache becomes a copy of page src[i], for K and V,
 * with their page scales.
 *  k_cache, v_cache  [num_blocks, 16, H, D] BF16 or FP8_E4M3, D a multiple of 16 bytes,
 *               strides as verify_attn; v_cache NULL: one cache (a latent one).
 *  k_scales, v_scales  [num_blocks, H] fp32 of e4m3 caches, or NULL.
 *  src, dst     [n]. A pair with an index outside [0, num_blocks) (-1), or of one page
 *               twice, copies nothing. A page may be copied any number of times; one that is
 *               written twice, or written and read, has unspecified contents.
 * Errors: VA_ERR_NULL, VA_ERR_SHAPE, VA_ERR_DTYPE (scales over a BF16 cache), VA_ERR_LAYOUT
 * (elements on top of each other, K and V in one place), VA_ERR_UNSUPPORTED (pages other
 * than 16, other widths, token rows of more than 65,535 * 512 bytes).
 */
va_status verify_attn_copy_pages(va_tensor* k_cache, va_tensor* v_cache, va_tensor* k_scales, va_tensor* v_scales,
                                 const va_tensor* src, const va_tensor* dst, void* stream);

/*
 * verify_attn_chunk - attention of chunks of new tokens over the paged cache:
 * whole prompts, pieces of prompts behind cached tokens, single tokens, mixed in
 * a batch. The operation of verify_attn and of its variants for any number of
 * new tokens and query heads a KV head: with L = cu_seqlens_q[b+1] -
 * cu_seqlens_q[b] new tokens of sequence b and S = seqused_k[b] cached ones (the
 * new ones counted, stored before), token t is at position i = S - L + t and
 * head h of it reads KV head h / (Hq/Hkv):
 *
 *   s_j = softmax_scale * k_descale * q . K_j        (then the soft cap)
 *   out[cu[b]+t, h, :] = v_descale * sum_j softmax(s)_j V_j  over j in [0, i], or
 *                        with a window over j in [i - window_left, i] and
 *                        j < min(first_tokens, i + 1)
 *
 *  q, out       [total_q, Hq, 256] BF16; out is written (rows of sequences; rows
 *               behind the last sequence are left as they were) and may not
 *               overlap an input or itself. A row that sees no key is 0.
 *  k_cache, v_cache  [num_blocks, 16, Hkv, 256] FP8_E4M3 or BF16, as verify_attn.
 *  k_scales, v_scales  [num_blocks, Hkv] fp32: a page-scaled e4m3 cache, as
 *               verify_attn_scaled reads it (no descales); or both NULL.
 *  block_table, cu_seqlens_q, seqused_k, k_descale, v_descale  as verify_attn.
 *               A page none of whose keys is seen is not read, so a
 *               sliding-window page table need not map it. Lengths past the
 *               table's width are read as the width, page ids outside
 *               [0, num_blocks) as pages of zeros.
 *  opts         NULL: no window, soft cap or sinks (verify_attn_opt).
 *  first_tokens with a window: the sequence's first tokens that stay visible
 *               (attention sinks that are tokens); without one they are anyhow.
 *  workspace    verify_attn_chunk_workspace_size() bytes of device memory,
 *               256-byte aligned, first 4 bytes its status word, as
 *               verify_attn_ex; or NULL to use the library's own, whose calls
 *               must be ordered on one stream (refused during stream capture,
 *               VA_ERR_WORKSPACE).
 *  num_splits   0: the library's choice; > 0: the CTA pairs that share the work
 *               (at most what the device holds). VA_LIBRARY_STATUS as
 *               verify_attn_scaled.
 *
 * Two launches (the second one joins what pairs shared), asynchronous on
 * stream, capturable; nothing depends on host bounds of the lengths.
 * Accuracy: Q K^T and P V on the tensor cores in 16 bits with fp32 sums. BF16
 * caches: P is rounded to bf16. E4M3 caches: Q enters as two e4m3 terms, bf16's 8
 * bits in steps of at most 2^-16 of the row's largest; V's codes are taken as f16
 * (exact) and P is rounded to f16, in steps of 2^-31 below 2^-21 of the row's
 * reference (within 2^8 of its largest weight). Beside a key whose value is 0, weights 2^-24
 * of its own keep 7 bits, 2^-28 three, and below 2^-32 they are gone (the normaliser counts
 * them); verify_attn_scaled and the other verify calls scale P by blocks of 32 keys and
 * keep them.
 * The normaliser, the references and the joined sums are fp32. With page scales a weight
 * is taken times its page's V scale, in the steps above too: the normaliser counts a key
 * while that product is within 2^-126 of the row's largest.
 * A value that is NaN or infinite at a key in [0, S) may reach rows of the same
 * sequence that do not see the key; keys may be anything where they are not seen.
 * Errors before launching, as verify_attn_append_kv; VA_ERR_UNSUPPORTED also for
 * first_tokens < 0, descales beside page scales, total_q * Hq / Hkv past 2^31, or
 * num_seqs * Hq * (total_q * Hq / Hkv / 256 + 1) * (16 * table width + total_q) past about 2^62.
 */
va_status verify_attn_chunk(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                            const va_tensor* k_scales, const va_tensor* v_scales, const va_tensor* block_table,
                            const va_tensor* cu_seqlens_q, const va_tensor* seqused_k, float softmax_scale,
                            const va_tensor* k_descale, const va_tensor* v_descale, va_tensor* out,
                            const va_options* opts, int32_t first_tokens, void* workspace, size_t workspace_bytes,
                            int32_t num_splits, void* stream);

/* Workspace bytes of verify_attn_chunk on the current device, for any shapes (0
 * on error). */
size_t verify_attn_chunk_workspace_size(void);

/*
 * verify_attn_last_device_error - reads and clears the device status word of
 * a workspace. This turns the pages' gates and asserts (sglang PR 36330 digest,
 * "Key code excerpts") into something a caller can check after launch: a
 * condition found on the device, when no host check could see it.
 *
 * Every wait of the main kernels (a ring slot, a TMA copy landing, an MMA
 * finishing) is bounded in time (2 s unless verify_attn_set_wait_limit says
 * otherwise). A wait that runs out makes the kernel stop issuing work, let
 * its copies and MMAs in flight finish, free its tensor memory and return;
 * it ORs a nonzero code into the status word of the call's workspace. The
 * outputs of that call are then unspecified. The status word is sticky:
 * kernels only ever set bits in it.
 *
 *  workspace  the 256-byte-aligned workspace pointer that was passed to
 *             verify_attn_ex, verify_attn_opt, verify_attn_mla,
 *             verify_attn_partial, verify_attn_chunk or a page-scaled call; or NULL for the library's own scratch on
 *             the current device: the workspace of calls made without one
 *             (verify_attn, and the others with a NULL workspace), the
 *             built-in array of verify_attn_noalloc, and the word of page-scaled
 *             and chunk calls with VA_LIBRARY_STATUS. The library's workspace
 *             is replaced when it grows; its word then starts at 0 again.
 *  bits       host int32, written: the OR of the words read (0 = no bounded
 *             wait ran out since the last read and clear). Nonzero bits name
 *             the wait that gave up; they are diagnostic, not an API.
 *  stream     the words are read after the work queued on `stream` (this
 *             call synchronises it), then cleared on it. Calls on other
 *             streams that use the same scratch must be ordered by the caller.
 * Returns VA_ERR_NULL for a NULL bits, VA_ERR_WORKSPACE for a misaligned
 * workspace, VA_ERR_CUDA if a copy or the synchronisation fails.
 */
va_status verify_attn_last_device_error(const void* workspace, int32_t* bits, void* stream);

/*
 * verify_attn_set_wait_limit - the time limit, in nanoseconds, of the main
 * kernels' bounded waits for launches made after this call, process-wide; 0
 * restores the default of 2 s. A hook for tests of the timeout path: a limit
 * of a few nanoseconds makes waits run out on any input, so that a test can
 * check that the call still returns, the status word is set and the next
 * call is correct. Not for production use (any limit shorter than the
 * kernels' normal waits makes every call fail). Always returns VA_OK.
 */
va_status verify_attn_set_wait_limit(uint64_t limit_ns);

/* Static, NUL-terminated name of a status code. */
const char* verify_attn_status_string(int32_t status);

#ifdef __cplusplus
}
#endif

#endif /* VERIFY_ATTN_H */
