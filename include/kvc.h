/*
 * kvc.h -- C ABI of the GB300 persistent KV-cache library (libkvc.so).
 *
 * One step of the hot path appends new key/value rows to a persistent cache
 * and runs grouped-query attention (GQA) over it:
 *
 *     kvc_seq_lengths      lengths derived on the device from seqlens_k
 *     kvc_window_append    append (contiguous cache), in-place compaction +
 *                          append (windowed cache, one token), or C + S
 *                          staging seed / copy-back (windowed, several tokens)
 *     kvc_gqa_decode       one-token GQA attention over the cache
 *     kvc_gqa_decode_ring  the same over a ring of C slots (circular addressing)
 *     kvc_window_append_inplace  the staging step with the stage in the cache's rows
 *     kvc_paged_append, kvc_gqa_decode_paged  append and decode on a paged cache
 *     kvc_quantize_pages, kvc_gqa_decode_paged_q  int8 pages and decode over
 *                          a cache of 16-bit and int8 pages
 *     kvc_decode_step      lengths + append + decode in one launch (contiguous
 *                          cache or ring)
 *     kvc_window_decode_step  the same for a windowed cache
 *     kvc_gqa_prefill_chunk  multi-token GQA attention over staged rows
 *     kvc_window_prefill_step  a windowed multi-token step that stages only
 *                          the rows whose eviction its chunk would see
 *     kvc_tensor_scatter   the ONNX TensorScatter cache update (linear/circular)
 *     kvc_quant_append, kvc_dequant_rows, kvc_gqa_decode_quant  a cache whose
 *                          rows are quantised as they are written, read back
 *                          in 16 bits or attended over as codes
 *     kvc_tree_mask, kvc_tree_append, kvc_gqa_tree, kvc_tree_commit  a tree of
 *                          drafted tokens verified over the cache
 *     kvc_page_bounds, kvc_gqa_decode_sparse  one-token attention over the
 *                          pages that a cheap score selects
 *     kvc_page_release, kvc_ragged_plan, kvc_rope_tables, kvc_ragged_append,
 *     kvc_gqa_ragged       a step whose requests bring different numbers of new
 *                          tokens: pages and places, tables, append, attention
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  * Ownership: the caller owns every buffer.  The library allocates nothing,
 *    keeps no state between calls (apart from cached device attributes and
 *    the scratch array of kvc_gqa_decode_noalloc) and never reads device
 *    memory on the host, so the calls listed above can be captured in a CUDA
 *    graph.  Pointers marked "device" must be device (or managed)
 *    memory of the current device; pointers marked "host" are read during
 *    the call only.
 *  * Streams: `stream` is a cudaStream_t (NULL = legacy default stream).  Work
 *    is enqueued, never waited for.
 *  * Threads: calls may come from several host threads at once, a new thread's
 *    first CUDA call among them; what they write is theirs to keep apart.
 *  * Layout: caches and staging buffers are BNSH: [batch, kv_heads, rows, D],
 *    row-major, rows of D contiguous elements.  Queries and outputs are
 *    [batch, q_heads, new_tokens, D].  Query head h reads KV head
 *    h / (q_heads / kv_heads).
 *  * Errors: arguments are validated on the host before any launch and a
 *    non-zero kvc_status is returned with nothing enqueued.  Errors that
 *    depend on device data (an index out of range, a bad seqlens_k, a RoPE
 *    position beyond the cos/sin cache) are OR-ed into the caller's device
 *    word `dev_status` (may be NULL) as KVC_DEV_* bits, and the offending
 *    batch row writes nothing.  A failed launch returns KVC_ERR_CUDA.
 *  * Element types: KVC_F32, KVC_BF16, KVC_F16.  Attention accumulates in
 *    fp32 and rounds the output to nearest-even in the input type.
 *
 * Sources (page title, section):
 *   "TensorScatter" operator page (ai.onnx, since version 24): spec,
 *     pseudocode, examples.
 *   "GQA support sliding_window_cache" (onnxruntime pull request 29904):
 *     section "Design" (windowed invariant, append formula, device-side
 *     lengths, C + S staging) and the follow-up commits (int64 widening,
 *     RoPE bounded by the cos/sin cache length, not by the capacity).
 *   "Persistent KV Cache and Decode Performance Roadmap", section "Phase 1"
 *     (streaming decode with online softmax, GQA heads sharing a KV block,
 *     split of one query row across workers with an (m, l, o) merge).
 *   "Stateful decode & KV cache", section "Sliding-window ring buffer"
 *     (RoPE baked into K at write time; the mask depends on positions only).
 *   "Persistent KV Cache and Decode Performance Roadmap", "Phase 2" and the
 *     CPU backend's "fixed-size paged blocks and a page-table iterator
 *     consumed directly by Attention" (the paged calls).
 */
#ifndef KVC_H
#define KVC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVC_ABI_VERSION 7

typedef enum {
    KVC_OK = 0,
    KVC_ERR_NULL = 1,        /* a required pointer is NULL                       */
    KVC_ERR_SHAPE = 2,       /* a size is out of range or buffers overlap badly  */
    KVC_ERR_DTYPE = 3,       /* element type not supported by this entry point   */
    KVC_ERR_ALIGN = 4,       /* a buffer is not 16-byte aligned where required   */
    KVC_ERR_UNSUPPORTED = 5, /* a valid combination the library does not cover   */
    KVC_ERR_CAPACITY = 6,    /* capacity < 1 or too small for the request        */
    KVC_ERR_WINDOW = 7,      /* windowed cache needs 0 < local_window_size <= C  */
    KVC_ERR_WORKSPACE = 8,   /* workspace NULL or smaller than required          */
    KVC_ERR_CUDA = 9         /* a CUDA call failed (launch or driver)            */
} kvc_status;

typedef enum { KVC_F32 = 0, KVC_BF16 = 1, KVC_F16 = 2 } kvc_dtype;
/* 8-bit codes of a quantised row (code * scale is the value) */
typedef enum { KVC_INT8 = 0, KVC_E4M3 = 1 } kvc_quant_format;
/* how rotation frequencies are stretched for contexts longer than those trained on */
typedef enum {
    KVC_ROPE_PLAIN = 0,  /* as trained                                           */
    KVC_ROPE_LINEAR = 1, /* positions divided by a factor                        */
    KVC_ROPE_BASE = 2,   /* a larger base: the slowest pair is slowed by it      */
    KVC_ROPE_PARTS = 3   /* slow pairs slowed, fast ones kept, a ramp between    */
} kvc_rope_scaling;
typedef enum { KVC_LINEAR = 0, KVC_CIRCULAR = 1 } kvc_mode;
typedef enum { KVC_APPEND = 0, KVC_COPY_BACK = 1 } kvc_phase;
/* How the resident rows of a cache follow the absolute length T (the
 * `windowed` argument of the calls below). */
typedef enum {
    KVC_CONTIGUOUS = 0, /* every token stays: rows [0, T), T <= C               */
    KVC_WINDOWED = 1,   /* the last min(T, C) tokens; compaction on every step
                           once the cache is full                              */
    KVC_DRIFTING = 2,   /* the last end(T) tokens, W <= end(T) <= C: compaction
                           reclaims C - W + 1 rows at once, every C - W + 1
                           one-token steps                                     */
    KVC_RING = 3        /* a ring of C slots: token p lives in slot p mod C and
                           nothing ever moves ("Stateful decode & KV cache",
                           "Sliding-window ring buffer")                       */
} kvc_cache_policy;

/* device status bits (OR-ed into *dev_status) */
#define KVC_DEV_INDEX_OOB 1u    /* TensorScatter linear: wi < 0 or wi + S > max_seq    */
#define KVC_DEV_SEQLEN_RANGE 2u /* seqlens_k + 1 < new_tokens, or >= 2^31             */
#define KVC_DEV_CAPACITY 4u     /* contiguous cache: seqlens_k + 1 > capacity          */
#define KVC_DEV_ROPE_RANGE 8u   /* an absolute position >= rope_max_pos                */
#define KVC_DEV_TIMEOUT 16u     /* a bounded wait inside a kernel gave up              */

/*
 * Per-batch lengths, five device int32 arrays of [batch] each, written by
 * kvc_seq_lengths and read by the other calls ("GQA support
 * sliding_window_cache", "Design": absolute lengths for RoPE, cache-relative
 * lengths for addressing, and the evict count).  A rejected row holds -1 in
 * all five.
 *   past_abs    P  = T - S        absolute tokens before this step
 *   total_abs   T  = seqlens_k+1  absolute tokens after this step
 *   cache_past  Lp                rows resident before the step
 *   cache_total L                 rows resident after the step
 *   evict       E                 rows evicted by the step
 */
typedef struct {
    int32_t *past_abs;
    int32_t *total_abs;
    int32_t *cache_past;
    int32_t *cache_total;
    int32_t *evict;
} kvc_lengths;

/*
 * kvc_tensor_scatter -- ONNX TensorScatter ("TensorScatter" operator page,
 * opset 24: spec and pseudocode).
 *
 * present_cache  device, shape cache_shape, elem_bytes per element.
 * past_cache     device, same shape.  present_cache == past_cache runs in
 *                place (only the updated rows move); distinct buffers run the
 *                functional form (every row of present is written once, from
 *                update or from past).  Partially overlapping buffers ->
 *                KVC_ERR_SHAPE.
 * update         device, cache_shape with dimension `axis` = update_seq_len.
 * write_indices  device int64 [cache_shape[0]], or NULL (all zeros).
 * rank           2..8; cache_shape is a HOST array of `rank` sizes.
 * axis           sequence axis, != 0 (negative counts from the end; the
 *                operator's default is -2).
 * mode           KVC_LINEAR: row b writes [wi, wi + S); wi < 0 or
 *                wi + S > max_seq sets KVC_DEV_INDEX_OOB and leaves row b of
 *                present equal to past.  KVC_CIRCULAR: index mod max_seq
 *                (floor modulo, so negative wi wraps).
 * update_seq_len 0..max_seq (a longer update is a shape error).
 * elem_bytes     1, 2, 4 or 8: rows are copied as bytes, any element type.
 */
kvc_status kvc_tensor_scatter(void *present_cache, const void *past_cache, const void *update,
                              const int64_t *write_indices, int rank, const int64_t *cache_shape,
                              int64_t update_seq_len, int axis, int mode, int elem_bytes,
                              int32_t *dev_status, void *stream);

/*
 * kvc_seq_lengths -- derive the five length arrays on the device ("GQA
 * support sliding_window_cache", "Design"; int64 arithmetic per the PR's
 * widening commit).  T = seqlens_k[b] + 1 computed in 64 bits, P = T - S.
 *   KVC_WINDOWED, KVC_RING:
 *                   Lp = min(P, C), E = max(0, Lp + S - C), L = Lp - E + S
 *                   (for a ring: slots holding a token before / after the
 *                   step, and old tokens the step overwrites)
 *   KVC_DRIFTING:   Lp = end(P), L = end(T), E = Lp + S - L, where (the PR's
 *                   CPU commit, "drifting layout") gap = C - W + 1 and
 *                   end(T) = T for T <= C, else T - gap * ceil((T - C) / gap)
 *   KVC_CONTIGUOUS: Lp = P, E = 0, L = T; T > C sets KVC_DEV_CAPACITY.
 * T < S or T >= 2^31 sets KVC_DEV_SEQLEN_RANGE.  A rejected row gets -1 in
 * every array.
 * seqlens_k        device int32 [batch].
 * new_tokens       S >= 1.
 * capacity         C >= 1 rows per head.
 * windowed         a kvc_cache_policy (other values: KVC_ERR_UNSUPPORTED).
 * local_window_size  windowed, drifting or ring cache: must satisfy 0 < W <= C
 *                  (KVC_ERR_WINDOW otherwise); ignored for a contiguous cache.
 */
kvc_status kvc_seq_lengths(const int32_t *seqlens_k, int batch, int new_tokens, int64_t capacity,
                           int windowed, int local_window_size, kvc_lengths out,
                           int32_t *dev_status, void *stream);

/*
 * kvc_window_append -- write S new K/V rows per (batch, kv head) ("GQA
 * support sliding_window_cache", "Design").  K rows are rotated (RoPE,
 * rotate-half pairs (i, i + D/2), float32 with every product and sum
 * rounded separately) at their ABSOLUTE position P + i before they are
 * stored; V rows are stored as given.
 *
 * k_cache, v_cache  device [batch, kv_heads, capacity, head_dim].
 * new_k, new_v      device [batch, kv_heads, new_tokens, head_dim].
 * k_stage, v_stage  device [batch, kv_heads, capacity + new_tokens, head_dim]
 *                   for a windowed cache with S > 1, else ignored (may be NULL).
 * len               outputs of kvc_seq_lengths for the same S and C.
 * windowed          a kvc_cache_policy; KVC_WINDOWED and KVC_DRIFTING append
 *                   alike (what differs is in `len`) and are called
 *                   "windowed" below.  KVC_RING: row i goes to slot
 *                   (P + i) mod C for any S, nothing moves and no stage is
 *                   used (when S > C only the last C rows are written, the
 *                   ones that would survive); phase must be KVC_APPEND.
 * phase = KVC_APPEND:
 *   contiguous cache:      rows [P, P + S) of the cache.
 *   windowed, S == 1:      in place: rows [E, Lp) move to [0, Lp - E)
 *                          (E <= 1 for KVC_WINDOWED, 0 or C - W + 1 for
 *                          KVC_DRIFTING), then the new row goes to Lp - E.
 *   windowed, S > 1:       seeds the stage: stage[0, Lp) = cache[0, Lp),
 *                          stage[Lp + i] = new row i.  Attention then runs on
 *                          the stage (kvc_gqa_prefill_chunk).
 * phase = KVC_COPY_BACK (windowed, S > 1 only):
 *                          cache[0, L) = stage[E, Lp + S).
 * rope_cos, rope_sin  device float32 [rope_max_pos, head_dim / 2] indexed by
 *                   absolute position, or both NULL for no rotation.  A row
 *                   with P + S > rope_max_pos sets KVC_DEV_ROPE_RANGE and is
 *                   not written.
 * head_dim          even, 2..1024; dtype KVC_F32/KVC_BF16/KVC_F16.
 */
kvc_status kvc_window_append(void *k_cache, void *v_cache, const void *new_k, const void *new_v,
                             void *k_stage, void *v_stage, kvc_lengths len, int batch,
                             int kv_heads, int new_tokens, int64_t capacity, int head_dim,
                             int dtype, int windowed, int phase, const float *rope_cos,
                             const float *rope_sin, int64_t rope_max_pos, int32_t *dev_status,
                             void *stream);

/*
 * kvc_window_append_inplace -- the C + S staging step of a windowed cache
 * with the stage held in the cache's own rows ("GQA support
 * sliding_window_cache", "Design": a step with S new tokens attends over the
 * cached rows and the new ones, then keeps the last positions; here the stage
 * is not a second buffer).  The cache lives in rows [0, Lp) of a buffer with
 * rows_per_head >= capacity + new_tokens rows per head, so the rows a stage
 * would hold are already in place and no seed copy is made.
 *
 * k_rows, v_rows  device [batch, kv_heads, rows_per_head, head_dim]; rows
 *                 [0, Lp) hold the cache (Lp = len.cache_past).  Other calls
 *                 that read this cache take rows_per_head as their row pitch
 *                 (their `capacity` argument), while kvc_seq_lengths takes the
 *                 cache's capacity C.
 * new_k, new_v    device [batch, kv_heads, new_tokens, head_dim].
 * len             outputs of kvc_seq_lengths for the same S and C.
 * windowed        KVC_WINDOWED or KVC_DRIFTING.
 * phase = KVC_APPEND:     rows [Lp, Lp + S) <- the new rows (K rotated at
 *                         P + i, as kvc_window_append).  Attention then runs
 *                         on these rows (kvc_gqa_prefill_chunk with this
 *                         rows_per_head).
 * phase = KVC_COPY_BACK:  rows [0, L) <- rows [E, Lp + S), moved in place
 *                         (one CTA per (batch, kv head, K/V) walks the range
 *                         in ascending chunks, so every row is read before it
 *                         is overwritten).  Rows [0, L) are then byte for byte
 *                         what kvc_window_append's staged pair leaves in a
 *                         cache of `capacity` rows; rows past L are scratch.
 * A row rejected by kvc_seq_lengths (lengths -1) or for its RoPE range is left
 * untouched by both phases (KVC_DEV_ROPE_RANGE as kvc_window_append).
 * head_dim * element size a multiple of 16 bytes (KVC_ERR_UNSUPPORTED);
 * buffers 16-byte aligned; rows_per_head < capacity + new_tokens ->
 * KVC_ERR_CAPACITY.
 */
kvc_status kvc_window_append_inplace(void *k_rows, void *v_rows, const void *new_k,
                                     const void *new_v, kvc_lengths len, int batch, int kv_heads,
                                     int new_tokens, int64_t capacity, int64_t rows_per_head,
                                     int head_dim, int dtype, int windowed, int phase,
                                     const float *rope_cos, const float *rope_sin,
                                     int64_t rope_max_pos, int32_t *dev_status, void *stream);

/*
 * kvc_gqa_decode -- one-token grouped-query attention over the cache after
 * the append ("Persistent KV Cache and Decode Performance Roadmap", Phase 1:
 * streaming online softmax, a KV block read once per query-head group, a
 * split of long rows across CTAs merged by (m, l, o); masks from "GQA support
 * sliding_window_cache").
 *
 * For batch row b: rows [0, L) of each head (L = len.cache_total[b]) hold
 * absolute positions T - L + r (T = len.total_abs[b]); the query is at
 * T - 1 and is rotated there when rope tables are given.  Row r is visible
 * iff local_window_size <= 0 or (T - 1) - pos(r) < local_window_size.
 *
 * out, q        device [batch, q_heads, 1, head_dim], same dtype as the cache.
 * k_cache/v_cache device [batch, kv_heads, capacity, head_dim].
 * scale         0 -> 1/sqrt(head_dim).
 * workspace     device scratch of kvc_gqa_decode_workspace_size(...) bytes
 *               (holds per-split partial (m, l, o)); 256-byte aligned.
 * Supported: KVC_BF16/KVC_F16 with head_dim in {64, 128, 256} and
 * q_heads / kv_heads <= 16 (tensor-core path); KVC_F32 with head_dim <= 256.
 * All buffers 16-byte aligned (KVC_ERR_ALIGN).
 */
kvc_status kvc_gqa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                          kvc_lengths len, int batch, int q_heads, int kv_heads, int64_t capacity,
                          int head_dim, int dtype, int local_window_size, float scale,
                          const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                          void *workspace, size_t workspace_bytes, int32_t *dev_status,
                          void *stream);

/* Bytes of workspace kvc_gqa_decode needs for these sizes (0 on bad sizes). */
size_t kvc_gqa_decode_workspace_size(int batch, int q_heads, int kv_heads, int64_t capacity,
                                     int head_dim, int dtype);

/* Size of the library's own decode scratch array (see kvc_gqa_decode_noalloc). */
#define KVC_DECODE_STATIC_SCRATCH_BYTES (16u << 20)

/*
 * kvc_gqa_decode_noalloc -- kvc_gqa_decode for callers that cannot allocate
 * device memory.  The source pages have no counterpart of this call; it is a
 * convenience of this library.
 *
 * Who needs it: code that runs where it has no device allocator to call, or
 * is not allowed to use one -- for example a plugin or operator inside a host
 * framework that owns all device memory through its own pool and gives its
 * kernels no way to request scratch, or a caller that has sized its memory
 * up front and must not grow it while serving.  Such a caller still owns and
 * passes every input and output; only the decode's split partials (the
 * workspace of kvc_gqa_decode) move into memory the library provides.
 *
 * The scratch is one file-scope device array of
 * KVC_DECODE_STATIC_SCRATCH_BYTES (16 MiB) that every device loading the
 * library keeps until the process exits.  Sizes whose workspace
 * (kvc_gqa_decode_workspace_size) exceeds it are rejected with
 * KVC_ERR_WORKSPACE before anything is enqueued.  The call itself allocates
 * nothing: no cudaMalloc, cudaFree or allocating library routine.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  All calls share the one array and it keeps the
 * previous call's contents: nothing in it needs to start at zero (every
 * partial is written before it is read within a call), but two calls whose
 * kernels overlap on the GPU -- on different streams, or different threads
 * -- race on it and may return wrong results.  Serialise them (one stream,
 * or events).
 *
 * Arguments, layouts, supported sizes and errors are those of
 * kvc_gqa_decode without the workspace pair.
 */
kvc_status kvc_gqa_decode_noalloc(void *out, const void *q, const void *k_cache,
                                  const void *v_cache, kvc_lengths len, int batch, int q_heads,
                                  int kv_heads, int64_t capacity, int head_dim, int dtype,
                                  int local_window_size, float scale, const float *rope_cos,
                                  const float *rope_sin, int64_t rope_max_pos,
                                  int32_t *dev_status, void *stream);

/*
 * kvc_gqa_decode_ring -- kvc_gqa_decode over a ring of C slots ("Stateful
 * decode & KV cache", "Sliding-window ring buffer"; the ring written by
 * kvc_window_append(KVC_RING) or by kvc_tensor_scatter in KVC_CIRCULAR mode
 * at write index P): slot r holds position T - 1 - ((T - 1 - r) mod C).  The
 * query at T - 1 sees the newest n = min(L, W) positions (n = L when
 * local_window_size <= 0), where L = len.cache_total[b] (min(T, C) from
 * kvc_seq_lengths) and T = len.total_abs[b]; they occupy slots
 * (T - n) mod C onwards, wrapping at C.  Equal to kvc_gqa_decode over the
 * full history whenever W <= C.  Arguments, layouts, supported sizes,
 * workspace and errors are those of kvc_gqa_decode.
 */
kvc_status kvc_gqa_decode_ring(void *out, const void *q, const void *k_cache, const void *v_cache,
                               kvc_lengths len, int batch, int q_heads, int kv_heads,
                               int64_t capacity, int head_dim, int dtype, int local_window_size,
                               float scale, const float *rope_cos, const float *rope_sin,
                               int64_t rope_max_pos, void *workspace, size_t workspace_bytes,
                               int32_t *dev_status, void *stream);

/*
 * Paged cache ("Persistent KV Cache and Decode Performance Roadmap", Phase 2:
 * fixed-size pages read through a page table, never gathered into one
 * contiguous cache).  K and V live in page pools [n_pool_pages, kv_heads,
 * page_size, head_dim] (one page holds page_size consecutive tokens of every
 * KV head).  block_table is device int32 [batch, max_pages]: logical row r of
 * batch row b is slot r % page_size of page block_table[b * max_pages +
 * r / page_size].  The caller allocates the pages (the table entries a step
 * touches must name pages of the pool); the lengths are those of a
 * contiguous cache of capacity max_pages * page_size (kvc_seq_lengths with
 * KVC_CONTIGUOUS).
 *
 * kvc_paged_append -- write the S new rows (K rotated at P + i as in
 * kvc_window_append) at logical rows [P, P + S).  A row whose new tokens
 * would land in a page id outside [0, n_pool_pages) sets KVC_DEV_INDEX_OOB
 * and writes nothing.  Any even head_dim <= 1024; all dtypes.
 */
kvc_status kvc_paged_append(void *k_pool, void *v_pool, const void *new_k, const void *new_v,
                            const int32_t *block_table, int max_pages, int64_t n_pool_pages,
                            int page_size, kvc_lengths len, int batch, int kv_heads,
                            int new_tokens, int head_dim, int dtype, const float *rope_cos,
                            const float *rope_sin, int64_t rope_max_pos, int32_t *dev_status,
                            void *stream);

/*
 * kvc_gqa_decode_paged -- kvc_gqa_decode over a paged cache: the split
 * kernel streams 64-row tiles straight from the pages (page_size must be a
 * positive multiple of 64, so that no tile straddles two pages).  A page id
 * outside the pool sets KVC_DEV_INDEX_OOB; that row's output is then
 * undefined.  Workspace: kvc_gqa_decode_workspace_size(batch, q_heads,
 * kv_heads, max_pages * page_size, head_dim, dtype).  Supported:
 * KVC_BF16/KVC_F16, head_dim in {64, 128, 256}, q_heads / kv_heads <= 16.
 */
kvc_status kvc_gqa_decode_paged(void *out, const void *q, const void *k_pool,
                                const void *v_pool, const int32_t *block_table, int max_pages,
                                int64_t n_pool_pages, int page_size, kvc_lengths len, int batch,
                                int q_heads, int kv_heads, int head_dim, int dtype,
                                int local_window_size, float scale, const float *rope_cos,
                                const float *rope_sin, int64_t rope_max_pos, void *workspace,
                                size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * Quantized pages ("Persistent input/output feedback", "Optional
 * heterogeneous paged KV": selected-block affine quantization; "Persistent
 * KV Cache and Decode Performance Roadmap", "Phase 3": cold pages to INT8,
 * recent tokens kept in the native type).  Int8 pages live in pools
 * qk_pool, qv_pool [n_qpool_pages, kv_heads, page_size, head_dim] of bytes; a
 * block-table entry with KVC_PAGE_QUANT set names page
 * (entry & ~KVC_PAGE_QUANT) of these pools.  qparams is device float
 * [n_qpool_pages][4] = (k_scale, k_zp, v_scale, v_zp) per int8 page, so that
 * a stored byte u (unsigned) reconstructs as (u - zp) * scale.
 *
 * Payload order (the MMA fragment order of the decode): the page_size rows of
 * a (page, kv head) are cut into groups of 16; group G is 16 * head_dim
 * bytes at G * 16 * head_dim.  Within a group, with D = head_dim:
 *   K element (row j, column d):  nb = j / 8, g = j % 8, kk = d / 16,
 *     dd = d % 16, lane = 4 g + (dd % 8) / 2,
 *     f = (2 kk + dd / 8) * 4 + 2 nb + dd % 2
 *   V element (row j, column c):  mb = c / 16, cc = c % 16,
 *     lane = 4 (cc % 8) + (j % 8) / 2, f = (2 mb + j / 8) * 4 + 2 (cc / 8) + j % 2
 *   byte = (f / 16) * 512 + lane * 16 + f % 16
 * (lane l's D / 2 bytes are the A fragments of its mma.m16n8k16 steps --
 * the 16 rows are the MMA's M dimension, K as it is and V transposed --
 * stored as 16-byte pieces interleaved across the 32 lanes).
 */
#define KVC_PAGE_QUANT 0x40000000

/*
 * kvc_quantize_pages -- page src_pages[i] of the 16-bit pools (every row and
 * KV head) becomes int8 page dst_pages[i], for i < n_pages:
 *     code = saturate(round_half_even(x / scale) + zero_point)
 * with x / scale in float32, saturated to [-128, 127] (INT8) or [0, 255]
 * (UINT8: *_unsigned != 0); the stored byte is the unsigned code + 128 - bias
 * (bias 0 for INT8, 128 for UINT8: an INT8 code c is stored as c + 128, a
 * UINT8 code as itself) and qparams[dst] = (k_scale, k_zero_point + 128 -
 * k_bias, v_scale, v_zero_point + 128 - v_bias).  K and V may use different
 * formats.
 * k_pool, v_pool     device [n_pool_pages, kv_heads, page_size, head_dim],
 *                    KVC_BF16 or KVC_F16.
 * src_pages, dst_pages  device int32 [n_pages]; a pair with an id outside its
 *                    pool sets KVC_DEV_INDEX_OOB and is skipped.  Destinations
 *                    must be distinct.  The block table is not touched: the
 *                    caller points its entries at (dst | KVC_PAGE_QUANT).
 * Scales positive and finite, zero points inside the code range
 * (KVC_ERR_SHAPE otherwise); page_size a multiple of 16; head_dim a multiple
 * of 32.
 */
kvc_status kvc_quantize_pages(const void *k_pool, const void *v_pool, void *qk_pool,
                              void *qv_pool, const int32_t *src_pages, const int32_t *dst_pages,
                              int n_pages, int64_t n_pool_pages, int64_t n_qpool_pages,
                              int page_size, int kv_heads, int head_dim, int dtype, float k_scale,
                              int k_zero_point, int k_unsigned, float v_scale, int v_zero_point,
                              int v_unsigned, float *qparams, int32_t *dev_status, void *stream);

/*
 * kvc_gqa_decode_paged_q -- kvc_gqa_decode_paged over a cache whose pages are
 * 16-bit (entries naming the k_pool / v_pool pages) or int8 (entries with
 * KVC_PAGE_QUANT).  An int8 tile is read at half the bytes and its
 * reconstruction (u - zp) * scale enters the attention with the page's
 * scale applied in float32 after the products: scores = k_scale * q . (u - zp),
 * values = v_scale * sum p (u - zp).  An entry outside its pool sets
 * KVC_DEV_INDEX_OOB (that row's output is undefined).  Same arguments and
 * limits as kvc_gqa_decode_paged plus the int8 pools, qparams (16-byte
 * aligned) and n_qpool_pages.
 */
kvc_status kvc_gqa_decode_paged_q(void *out, const void *q, const void *k_pool,
                                  const void *v_pool, const void *qk_pool, const void *qv_pool,
                                  const float *qparams, int64_t n_qpool_pages,
                                  const int32_t *block_table, int max_pages, int64_t n_pool_pages,
                                  int page_size, kvc_lengths len, int batch, int q_heads,
                                  int kv_heads, int head_dim, int dtype, int local_window_size,
                                  float scale, const float *rope_cos, const float *rope_sin,
                                  int64_t rope_max_pos, void *workspace, size_t workspace_bytes,
                                  int32_t *dev_status, void *stream);

/*
 * kvc_decode_step -- one fused one-token step on a contiguous cache or a
 * ring: kvc_seq_lengths + kvc_window_append (S = 1) + kvc_gqa_decode (or
 * kvc_gqa_decode_ring) with the same results, the lengths, the append and
 * the attention in one launch ("Persistent KV Cache and Decode Performance
 * Roadmap", Phase 1; "GQA support sliding_window_cache", "Design";
 * "Stateful decode & KV cache", "Sliding-window ring buffer").  The CTA that
 * holds the newest position rotates the new K row at T - 1 and stores it and
 * the V row to the cache (row T - 1, or slot (T - 1) mod C) while its first
 * tiles are in flight, then places both in its last tile on chip.  Rows long
 * enough for several splits are merged by a second launch, as in
 * kvc_gqa_decode.
 *
 * out, q          device [batch, q_heads, 1, head_dim].
 * k_cache/v_cache device [batch, kv_heads, capacity, head_dim], updated in place.
 * new_k, new_v    device [batch, kv_heads, 1, head_dim].
 * seqlens_k       device int32 [batch] (total after this token, minus one).
 * len             the five length arrays to fill (as kvc_seq_lengths would,
 *                 same policy, S = 1), or all five NULL.
 * windowed        KVC_CONTIGUOUS (T > C sets KVC_DEV_CAPACITY) or KVC_RING;
 *                 else KVC_ERR_UNSUPPORTED.
 * local_window_size, scale, rope_*: as kvc_gqa_decode.
 * workspace       device, kvc_decode_step_workspace_size(...) bytes (the same
 *                 as kvc_gqa_decode_workspace_size), 256-byte aligned.
 * Supported: KVC_BF16/KVC_F16, head_dim in {64, 128, 256}, q_heads / kv_heads
 * <= 16 (KVC_ERR_UNSUPPORTED otherwise).
 * Device errors as kvc_seq_lengths / kvc_window_append / kvc_gqa_decode.
 */
kvc_status kvc_decode_step(void *out, const void *q, void *k_cache, void *v_cache,
                           const void *new_k, const void *new_v, const int32_t *seqlens_k,
                           kvc_lengths len, int batch, int q_heads, int kv_heads, int64_t capacity,
                           int head_dim, int dtype, int windowed, int local_window_size,
                           float scale, const float *rope_cos, const float *rope_sin,
                           int64_t rope_max_pos, void *workspace, size_t workspace_bytes,
                           int32_t *dev_status, void *stream);

/* Bytes of workspace kvc_decode_step needs for these sizes (0 on bad sizes). */
size_t kvc_decode_step_workspace_size(int batch, int q_heads, int kv_heads, int64_t capacity,
                                      int head_dim, int dtype);

/*
 * kvc_window_decode_step -- one one-token step on a windowed cache:
 * kvc_seq_lengths + kvc_window_append (S = 1) + kvc_gqa_decode with the same
 * results ("GQA support sliding_window_cache", "Design": rows [E, Lp) move
 * to [0, Lp - E), the new row goes to Lp - E; attention over the window that
 * results).
 *   Small windows, capacity * head_dim <= 32768 (C <= 512 at D = 64, 256 at
 *   D = 128, 128 at D = 256): a single launch.  One CTA owns a (batch row, kv
 *   head) slice and reads it once: the resident rows are loaded into shared
 *   memory (when nothing is evicted, only those the window can see), written
 *   back E rows lower when rows were evicted (else only the new row is
 *   stored), and attended over from there.  No workspace is used.
 *   Larger windows: a ring runs as kvc_decode_step(KVC_RING); a windowed or
 *   drifting cache runs as kvc_seq_lengths, kvc_window_append (the in-place
 *   compaction of large slices runs as a cluster of CTAs per slice) and
 *   kvc_gqa_decode.  The workspace holds the split partials, and the lengths
 *   when `len` is all NULL.
 *
 * out, q          device [batch, q_heads, 1, head_dim].
 * k_cache/v_cache device [batch, kv_heads, capacity, head_dim], updated in place.
 * new_k, new_v    device [batch, kv_heads, 1, head_dim].
 * seqlens_k       device int32 [batch] (total after this token, minus one).
 * len             the five length arrays to fill (as kvc_seq_lengths would,
 *                 same policy, S = 1), or all five NULL.
 * windowed        KVC_WINDOWED, KVC_DRIFTING or KVC_RING (else
 *                 KVC_ERR_UNSUPPORTED).  For a ring the new row goes to slot
 *                 (T - 1) mod C, nothing else is written, and attention
 *                 reads the slots as kvc_gqa_decode_ring does.
 * workspace       device, kvc_window_decode_step_workspace_size(...) bytes,
 *                 256-byte aligned (0 bytes, NULL allowed, for small windows).
 * Requires 0 < local_window_size <= capacity (KVC_ERR_WINDOW).  Supported:
 * KVC_BF16/KVC_F16, head_dim in {64, 128, 256}, q_heads / kv_heads <= 16.
 * Device errors as kvc_seq_lengths / kvc_window_append / kvc_gqa_decode.
 */
kvc_status kvc_window_decode_step(void *out, const void *q, void *k_cache, void *v_cache,
                                  const void *new_k, const void *new_v, const int32_t *seqlens_k,
                                  kvc_lengths len, int batch, int q_heads, int kv_heads,
                                  int64_t capacity, int head_dim, int dtype, int windowed,
                                  int local_window_size, float scale, const float *rope_cos,
                                  const float *rope_sin, int64_t rope_max_pos, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Bytes of workspace kvc_window_decode_step needs for these sizes (0 for a
 * window held on chip, or on bad sizes). */
size_t kvc_window_decode_step_workspace_size(int batch, int q_heads, int kv_heads,
                                             int64_t capacity, int head_dim, int dtype);

/*
 * kvc_gqa_prefill_chunk -- attention of an S-token chunk over staged rows
 * ("GQA support sliding_window_cache", "Design": multi-token steps run
 * against the C + S staging cache; causal plus local-window mask).
 *
 * For batch row b with Lp = len.cache_past[b], P = len.past_abs[b]: rows
 * [0, Lp + S) of each head of k_rows/v_rows hold positions P - Lp + r (the
 * stage after kvc_window_append(KVC_APPEND), or a contiguous cache after its
 * append, where Lp = P).  Query i is at P + i and sees row r iff
 * pos(r) <= P + i and (local_window_size <= 0 or P + i - pos(r) <
 * local_window_size).  Queries are rotated at P + i when rope tables are
 * given.
 *
 * out, q          device [batch, q_heads, new_tokens, head_dim].
 * k_rows, v_rows  device [batch, kv_heads, rows_per_head, head_dim],
 *                 rows_per_head >= Lp + S for every row (C + S for a stage).
 * workspace       device scratch of kvc_gqa_prefill_workspace_size(...) bytes,
 *                 256-byte aligned, or NULL.  When the launch would not fill
 *                 the GPU (few query blocks), each block's key range is split
 *                 over several CTAs whose (o, m, l) partials go to the
 *                 workspace and are merged by a second launch; with NULL (or
 *                 too small a workspace) the call runs unsplit, with the same
 *                 results up to floating-point rounding order.
 * Supported: KVC_BF16/KVC_F16 with head_dim in {64, 128, 256} and
 * q_heads / kv_heads in {1, 2, 4, 8, 16} (tcgen05 tensor-core path);
 * KVC_F32 with head_dim <= 256 (no workspace used).  Buffers, the rope
 * tables included, 16-byte aligned (KVC_ERR_ALIGN).
 */
kvc_status kvc_gqa_prefill_chunk(void *out, const void *q, const void *k_rows, const void *v_rows,
                                 int64_t rows_per_head, kvc_lengths len, int batch, int q_heads,
                                 int kv_heads, int new_tokens, int head_dim, int dtype,
                                 int local_window_size, float scale, const float *rope_cos,
                                 const float *rope_sin, int64_t rope_max_pos, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_status, void *stream);

/*
 * kvc_window_prefill_step -- one whole step of S new tokens on a windowed or
 * drifting cache of C rows: append, chunk attention and row movement, with
 * the C + S stage used only for the rows that need it ("GQA support
 * sliding_window_cache", CPU commit: "Staging for hazardous steps"; the
 * decision is taken per batch row on the device, from the lengths).
 *
 * Batch row b with Lp = len.cache_past[b], E = len.evict[b] is hazardous
 * when E > 0 and E > Lp - W + 1: the rows [0, E) that the step evicts
 * include one that its first query (at stage row Lp) still sees.
 *   hazardous rows:  the new rows go to stage[Lp, Lp + S) and the 127 old
 *                    rows below them to stage[Lp - 127, Lp) (fewer when Lp <
 *                    127); the attention reads its 128-key tiles that lie
 *                    below Lp from the cache and the others from the stage;
 *                    then cache rows [E, Lp) move to [0, Lp - E) in place
 *                    and stage rows [max(E, Lp), Lp + S) follow them -- the
 *                    rows and results of kvc_window_append's staged pair at
 *                    about half its row traffic (the seed and copy-back of
 *                    the whole window become one move of it);
 *   the other rows:  cache rows [E, Lp) move to [0, Lp - E) in place, the new
 *                    rows go to [Lp - E, L), and the attention reads the
 *                    cache; no stage traffic (E = 0: only the new rows).
 * Either way the cache ends byte for byte as kvc_window_append leaves it and
 * the output is the attention of kvc_gqa_prefill_chunk over the stage (up to
 * floating-point summation order).  A row rejected by kvc_seq_lengths
 * (lengths -1) or for its RoPE range is left as kvc_window_append leaves it.
 *
 * out, q          device [batch, q_heads, new_tokens, head_dim].
 * k_cache, v_cache  device [batch, kv_heads, capacity, head_dim].
 * new_k, new_v    device [batch, kv_heads, new_tokens, head_dim].
 * k_stage, v_stage  device [batch, kv_heads, capacity + new_tokens, head_dim]
 *                 for S > 1, rows indexed as the cache's (only hazardous rows
 *                 write or read them, at most 127 + S rows each); may be NULL
 *                 for S = 1, which never stages.
 * len             kvc_seq_lengths outputs for this S, C, policy and window.
 * windowed        KVC_WINDOWED or KVC_DRIFTING; 0 < local_window_size <= C
 *                 (KVC_ERR_WINDOW).
 * workspace       kvc_gqa_prefill_workspace_size(batch, q_heads, kv_heads,
 *                 new_tokens, capacity, head_dim, dtype, local_window_size)
 *                 bytes, or NULL (as kvc_gqa_prefill_chunk).
 * Supported: KVC_BF16/KVC_F16 with head_dim in {64, 128, 256} and
 * q_heads / kv_heads in {1, 2, 4, 8, 16}; KVC_F32 with head_dim <= 256
 * (there every row of an S > 1 step is staged).  head_dim * element size a
 * multiple of 16 bytes (KVC_ERR_UNSUPPORTED); buffers 16-byte aligned.
 * Launches: the row movement before the attention (stage seed, in-place
 * move, new rows), the attention (+ its merge), and the copy-back.
 */
kvc_status kvc_window_prefill_step(void *out, const void *q, void *k_cache, void *v_cache,
                                   const void *new_k, const void *new_v, void *k_stage,
                                   void *v_stage, kvc_lengths len, int batch, int q_heads,
                                   int kv_heads, int new_tokens, int64_t capacity, int head_dim,
                                   int dtype, int windowed, int local_window_size, float scale,
                                   const float *rope_cos, const float *rope_sin,
                                   int64_t rope_max_pos, void *workspace, size_t workspace_bytes,
                                   int32_t *dev_status, void *stream);

/* Bytes of workspace kvc_gqa_prefill_chunk uses for these sizes on the
 * current device (0: it would not split). */
size_t kvc_gqa_prefill_workspace_size(int batch, int q_heads, int kv_heads, int new_tokens,
                                      int64_t rows_per_head, int head_dim, int dtype,
                                      int local_window_size);

/*
 * A cache quantised as it is written ("Persistent KV Cache and Decode
 * Performance Roadmap", "Phase 3: cache quantization and fusion").  A row x of
 * head_dim values is held as head_dim 8-bit codes and one float32 scale:
 *     KVC_INT8:  scale = max|x| / 127, code = clamp(rint(x / scale), -127, 127)
 *     KVC_E4M3:  scale = max|x| / 448, code = x / scale to e4m3 (nearest even,
 *                saturated)
 * with both divisions in float32; code * scale is the value read back.  A row
 * of zeros (or one so small that its scale is 0) has scale 0 and codes 0; a
 * row with a NaN or an infinity has scale NaN and codes 0, so it reads back
 * as NaN.  The cache of B x kv_heads x capacity rows is four arrays:
 *   kq_cache, vq_cache  device [batch, kv_heads, capacity, head_dim] bytes
 *   k_scale, v_scale    device float32 [batch, kv_heads, capacity]
 * (16-byte aligned, not overlapping).  `windowed` is KVC_CONTIGUOUS or KVC_RING
 * in all three calls (other policies move rows and are KVC_ERR_UNSUPPORTED);
 * `format` is a kvc_quant_format (KVC_ERR_DTYPE otherwise).
 *
 * kvc_quant_append -- write the S new rows of each (batch, kv head): K rotated
 * at P + i in float32 and quantised without a rounding in between, V as given.
 * Row P + i of a contiguous cache, slot (P + i) mod C of a ring (of S > C rows
 * only the last C).  A row past rope_max_pos sets KVC_DEV_ROPE_RANGE, lengths
 * that do not fit the capacity KVC_DEV_CAPACITY; that batch row writes nothing.
 * new_k, new_v  device [batch, kv_heads, new_tokens, head_dim], any kvc_dtype.
 * len           outputs of kvc_seq_lengths for the same S, C and policy.
 * head_dim      a multiple of 16, at most 256 (KVC_ERR_UNSUPPORTED);
 * batch * kv_heads <= 65535 (KVC_ERR_SHAPE).
 */
kvc_status kvc_quant_append(void *kq_cache, void *vq_cache, float *k_scale, float *v_scale,
                            const void *new_k, const void *new_v, kvc_lengths len, int batch,
                            int kv_heads, int new_tokens, int64_t capacity, int head_dim, int dtype,
                            int format, int windowed, const float *rope_cos,
                            const float *rope_sin, int64_t rope_max_pos, int32_t *dev_status,
                            void *stream);

/*
 * kvc_dequant_rows -- rows [0, L) of k_out, v_out <- the L resident rows
 * (L = len.cache_total), oldest first, as code * scale rounded to `dtype`: for
 * a ring, row r is position T - L + r.  Rows past L are left as they were, so
 * kvc_gqa_prefill_chunk can run a chunk over the rows of a contiguous cache
 * right after kvc_quant_append (rows_per_head = rows_out).
 * k_out, v_out  device [batch, kv_heads, rows_out, head_dim]; a batch row with
 *               L > rows_out sets KVC_DEV_CAPACITY and is left as it was.
 * head_dim as kvc_quant_append; batch * kv_heads <= 65535 (KVC_ERR_SHAPE).
 */
kvc_status kvc_dequant_rows(void *k_out, void *v_out, const void *kq_cache, const void *vq_cache,
                            const float *k_scale, const float *v_scale, kvc_lengths len, int batch,
                            int kv_heads, int64_t capacity, int64_t rows_out, int head_dim,
                            int dtype, int format, int windowed, int32_t *dev_status, void *stream);

/*
 * kvc_gqa_decode_quant -- kvc_gqa_decode (contiguous) or kvc_gqa_decode_ring
 * (ring) over a quantised cache, without a 16-bit copy of it: the codes go to
 * the tensor cores as halves (exactly) and the rows' scales enter in float32.
 * Masks, lengths, rope and errors as those calls: row r of the L rows of a
 * contiguous cache is position T - L + r, for any T >= L (a windowed cache's
 * lengths too).  A NaN scale of a visible row makes the output NaN.  Rejected batch rows keep their output.
 * out, q     device [batch, q_heads, 1, head_dim], KVC_BF16 or KVC_F16.
 * head_dim 64, 128 or 256, q_heads / kv_heads <= 16 (KVC_ERR_UNSUPPORTED).
 * workspace  device, kvc_gqa_decode_quant_workspace_size(...) bytes on the
 *            current device, 256-byte aligned (0 bytes: may be NULL).  Calls
 *            that may overlap on the GPU need workspaces of their own.
 * Every CTA takes the same share of the batch's visible rows, whatever the
 * lengths; rows that several CTAs worked on are joined by a second launch, in
 * a fixed order.
 * Beside the result, the rotated query (over a power of two) and the weights are
 * rounded to halves for KVC_BF16; for KVC_F16 they enter with the digits of two.
 * Query values up to 2^120 and scores (q . k times scale) up to 1e30 in magnitude;
 * beyond, the output may be NaN.
 */
kvc_status kvc_gqa_decode_quant(void *out, const void *q, const void *kq_cache,
                                const void *vq_cache, const float *k_scale, const float *v_scale,
                                kvc_lengths len, int batch, int q_heads, int kv_heads,
                                int64_t capacity, int head_dim, int dtype, int format, int windowed,
                                int local_window_size, float scale, const float *rope_cos,
                                const float *rope_sin, int64_t rope_max_pos, void *workspace,
                                size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Bytes of workspace kvc_gqa_decode_quant needs for these sizes (0 on bad sizes). */
size_t kvc_gqa_decode_quant_workspace_size(int batch, int q_heads, int kv_heads, int64_t capacity,
                                           int head_dim);

/*
 * One-token attention over selected pages of a paged cache ("Persistent KV
 * Cache and Decode Performance Roadmap", "Phase 2").  Every full page holds,
 * for each kv head, 8-bit bounds of its keys (as stored, K rotated):
 *     s = max|k| / 127,  hi_d = ceil(max_r k[r][d] / s),  lo_d = floor(min_r k[r][d] / s)
 * (float32 divisions; s = 0 for a page of zeros, s = infinity and zero codes
 * for a page with a NaN or an infinity, which is then always taken before
 * others).
 *   bounds       device int8 [n_pool_pages, kv_heads, 2, head_dim] (hi, lo)
 *   bound_scale  device float32 [n_pool_pages, kv_heads]
 *
 * kvc_page_bounds -- write the bounds of the pages that the step of S tokens
 * filled: logical pages [P / page_size, T / page_size) of each batch row
 * (after kvc_paged_append; a one-token step that fills no page writes
 * nothing).  Other pages' bounds are left as they were.  A page id outside the
 * pool sets KVC_DEV_INDEX_OOB and is skipped.  KVC_BF16/KVC_F16, head_dim 64,
 * 128 or 256 (KVC_ERR_UNSUPPORTED); bounds, bound_scale, k_pool 16-byte aligned.
 */
kvc_status kvc_page_bounds(void *bounds, float *bound_scale, const void *k_pool,
                           const int32_t *block_table, int max_pages, int64_t n_pool_pages,
                           int page_size, kvc_lengths len, int batch, int kv_heads, int new_tokens,
                           int head_dim, int dtype, int32_t *dev_status, void *stream);

/*
 * kvc_gqa_decode_sparse -- kvc_gqa_decode_paged over min(n_select, pages) of the
 * ceil(T / page_size) pages of each (batch row, kv head): the first sink_pages,
 * the last recent_pages (that of the newest token among them), and of the
 * others those with the largest scores, ties to the lower page.  With q the
 * rotated queries of the group (float32; -q when scale is negative, whose weights
 * grow with -q . k),
 *     u_d = sum_h max(q_hd, 0), w_d = sum_h min(q_hd, 0), rounded to float32,
 *     sq = max(|u|, |w|) / 127, both rounded to codes rint(. / sq),
 *     score = s * float(sum_d code(u_d) hi_d + code(w_d) lo_d)
 * the 8-bit form of sum_d max(q_d hi_d, q_d lo_d), which no key of the page
 * exceeds.  The sum is of whole numbers, so the choice is the same on every run.
 * Every page but the last recent_pages must have had its bounds written.
 * selected     device int32 [batch, kv_heads, n_select]: the logical pages taken,
 *              ascending, then -1.  A batch row that kvc_seq_lengths rejected, or
 *              whose position is past rope_max_pos (KVC_DEV_ROPE_RANGE) or beyond
 *              the table (KVC_DEV_CAPACITY), leaves its part of it and of out
 *              as they were.  A page id outside the pool sets KVC_DEV_INDEX_OOB
 *              (that row's output is then undefined, as in kvc_gqa_decode_paged).
 * sink_pages >= 0, recent_pages >= 1, their sum at most n_select (KVC_ERR_SHAPE);
 * max_pages <= 49152 (KVC_ERR_CAPACITY); batch * kv_heads <= 65535.
 * Types and sizes as kvc_gqa_decode_paged; the rotated query and the weights
 * enter with the digits of two 16-bit numbers, and only the result is rounded.
 * A NaN or an infinity in a column of a V row that is read makes that column of
 * the output NaN (rows behind the newest token may hold anything).
 * Scores (q . k times scale) up to 1e30 in magnitude; beyond, it may be NaN.
 * workspace    device, kvc_gqa_decode_sparse_workspace_size(...) bytes, 256-byte
 *              aligned.  Calls that may overlap on the GPU need their own.
 */
kvc_status kvc_gqa_decode_sparse(void *out, const void *q, const void *k_pool, const void *v_pool,
                                 const void *bounds, const float *bound_scale,
                                 const int32_t *block_table, int max_pages, int64_t n_pool_pages,
                                 int page_size, kvc_lengths len, int batch, int q_heads,
                                 int kv_heads, int head_dim, int dtype, int n_select,
                                 int sink_pages, int recent_pages, int32_t *selected, float scale,
                                 const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                                 void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                 void *stream);

/* Bytes of workspace kvc_gqa_decode_sparse needs for these sizes (0 on bad sizes). */
size_t kvc_gqa_decode_sparse_workspace_size(int batch, int q_heads, int kv_heads, int page_size,
                                            int n_select, int head_dim, int dtype);

/*
 * A tree of drafted tokens over a cache ("Persistent KV Cache and Decode
 * Performance Roadmap", "Phase 1", "Phase 2").  N nodes follow the P tokens of
 * each batch row (kvc_seq_lengths with new_tokens = N and KVC_CONTIGUOUS, so
 * P = T - N).  Node i continues the line of its parent: it stands at position
 * P + depth_i, its K and V rows lie at row P + i, and it sees every row of the
 * cache, its ancestors and itself (with a local window W only what is less than
 * W positions back).  The cache is contiguous, [batch, kv_heads, capacity,
 * head_dim] with block_table NULL, or paged as above (block_table, max_pages,
 * n_pool_pages and a page_size that is a multiple of 64; capacity is then
 * ignored).  KVC_BF16/KVC_F16, head_dim 64, 128 or 256, N <= 256
 * (KVC_ERR_UNSUPPORTED).
 *
 * kvc_tree_mask -- what the other calls read of the tree:
 *   parents  device int32 [batch, nodes]: the index of an earlier node, -1 (the
 *            node follows the cache), or -2 (no node: trees of a batch may
 *            differ in size).  Other values set KVC_DEV_INDEX_OOB and count as -2.
 *   mask     device uint32 [batch, nodes, ceil(nodes / 32)]: bit j % 32 of word
 *            j / 32 of node i is set when j is i or an ancestor of i.
 *   depth    device int32 [batch, nodes]: ancestors of the node, -1 for an
 *            absent node or one below it (its mask is zero).
 * mask and depth may also be written by the caller: any set of drafts may be
 * visible to a node (not only a line), at any depth in [0, nodes); a node whose
 * depth is outside is absent (KVC_DEV_INDEX_OOB when it is nodes or more), and
 * no node sees it whatever its mask says.
 */
kvc_status kvc_tree_mask(const int32_t *parents, int batch, int nodes, uint32_t *mask,
                         int32_t *depth, int32_t *dev_status, void *stream);

/*
 * kvc_tree_append -- rows P + i <- the nodes' K (rotated at P + depth_i) and V;
 * rows of absent nodes are left as they were.  A batch row with P + nodes past
 * the capacity (KVC_DEV_CAPACITY) or rope_max_pos (KVC_DEV_ROPE_RANGE), or with a
 * page id outside the pool among its new rows' (KVC_DEV_INDEX_OOB), writes
 * nothing.
 * new_k, new_v  device [batch, kv_heads, nodes, head_dim].
 */
kvc_status kvc_tree_append(void *k_cache, void *v_cache, const void *new_k, const void *new_v,
                           const int32_t *depth, const int32_t *block_table, int max_pages,
                           int64_t n_pool_pages, int page_size, kvc_lengths len, int batch,
                           int kv_heads, int nodes, int64_t capacity, int head_dim, int dtype,
                           const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                           int32_t *dev_status, void *stream);

/*
 * kvc_gqa_tree -- the attention of the nodes after kvc_tree_append: queries
 * rotated at P + depth_i; an absent node, or one that sees nothing, gives zeros.
 * A NaN or an infinity in a column of a V row that a node sees makes that column
 * of its output NaN, whatever the row's weight; a NaN in a K row that it sees
 * makes all of them NaN.  What it does not see may hold anything.
 * A batch row that kvc_seq_lengths rejected, or with P + nodes past the capacity
 * (KVC_DEV_CAPACITY) or rope_max_pos (KVC_DEV_ROPE_RANGE), keeps its output; a page
 * id outside the pool among the rows read, the nodes' own among them, sets
 * KVC_DEV_INDEX_OOB (that row's output is then undefined).
 * Beside the result, one of two numbers is rounded to the cache's type: the
 * weights (head_dim 64 and 128) or the rotated query (256); the other enters with
 * the digits of two 16-bit numbers.
 * out, q     device [batch, q_heads, nodes, head_dim]; q_heads / kv_heads <= 16,
 *            any whole number.
 * workspace  device, kvc_gqa_tree_workspace_size(...) bytes on the current device,
 *            256-byte aligned.  Calls that may overlap on the GPU need their own.
 */
kvc_status kvc_gqa_tree(void *out, const void *q, const void *k_cache, const void *v_cache,
                        const uint32_t *mask, const int32_t *depth, const int32_t *block_table,
                        int max_pages, int64_t n_pool_pages, int page_size, kvc_lengths len,
                        int batch, int q_heads, int kv_heads, int nodes, int64_t capacity,
                        int head_dim, int dtype, int local_window_size, float scale,
                        const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                        void *workspace, size_t workspace_bytes, int32_t *dev_status,
                        void *stream);

/* Bytes of workspace kvc_gqa_tree needs for these sizes (0 on bad sizes). */
size_t kvc_gqa_tree_workspace_size(int batch, int q_heads, int kv_heads, int nodes, int head_dim);

/*
 * kvc_tree_commit -- keep one line of the tree: rows P + path[j] move to P + j for
 * j < accepted, in place (K was rotated at its depth, so a line from the root on
 * is then as one-token steps would have left it), and seqlens_k <- P + accepted - 1,
 * the value from which the next step's starts.  The rows behind are scratch.
 * path       device int32 [batch, path_len], ascending nodes (path[j] >= j).
 * accepted   device int32 [batch], 0 <= accepted <= min(path_len, nodes).
 * seqlens_k  device int32 [batch], written (may be the step's own input).
 * A batch row whose path or count is not such, or whose pages [P, P + nodes) are
 * not all in the pool, sets KVC_DEV_INDEX_OOB and is left as it was, seqlens_k
 * too (KVC_DEV_CAPACITY when P + nodes is past the capacity).
 */
kvc_status kvc_tree_commit(void *k_cache, void *v_cache, const int32_t *path,
                           const int32_t *accepted, int path_len, const int32_t *block_table,
                           int max_pages, int64_t n_pool_pages, int page_size, kvc_lengths len,
                           int32_t *seqlens_k, int batch, int kv_heads, int nodes, int64_t capacity,
                           int head_dim, int dtype, int32_t *dev_status, void *stream);

/*
 * A ragged step over a paged cache ("Persistent KV Cache and Decode Performance
 * Roadmap", "Phase 2").  The calls above take the same number of new tokens for
 * every batch row; here request b (a row of the block table) brings n_b >= 0 of
 * its own -- one while it decodes, many while its prompt is read, none while it
 * waits -- and the new tokens lie packed, request behind request, in buffers of
 * `tokens` rows of which the last ones may be unused:
 *     offsets    device int32 [batch + 1]: request b's tokens are rows
 *                [offsets[b], offsets[b + 1])
 *     positions  device int32 [tokens]: a token's position in its request
 *     slots      device int32 [tokens]: page * page_size + row of the pool, where
 *                its K and V go
 * (positions and slots -1 for a row that is unused or whose request was rejected).
 * Pools, tables and pages are those of kvc_paged_append; page_size >= 1, at most
 * 16384 requests (KVC_ERR_UNSUPPORTED), max_pages * page_size and n_pool_pages *
 * page_size below 2^31, `tokens` up to 2^31 - 1024 (KVC_ERR_CAPACITY).  What a call
 * writes may not overlap what it reads (KVC_ERR_SHAPE); in particular a step's
 * `cached` is not an array of the `len` that it writes: copy it.
 *
 * Free pages are a stack: free_pages device int32 [n_pool_pages], its first
 * *free_count entries (device int32) the ids of the free pages.  Both calls read
 * *free_count and write *free_left, which must be another word: a loop that uses
 * both calls passes (a, b) to one and (b, a) to the other.  A count outside
 * [0, n_pool_pages] sets KVC_DEV_INDEX_OOB and counts as 0.
 *
 * kvc_page_release -- the pages of the first released[b] tokens of each row
 * (device int32 [batch], 0: keeps all) are pushed, row by row, lower pages first.
 * The table's entries stay as they are.  A negative count or one past the table
 * sets KVC_DEV_SEQLEN_RANGE and releases nothing of that row; rows that the stack
 * has no room for release nothing (KVC_DEV_CAPACITY); an id outside the pool is
 * pushed as it is and sets KVC_DEV_INDEX_OOB.
 */
kvc_status kvc_page_release(const int32_t *released, const int32_t *block_table, int max_pages,
                            int page_size, int32_t *free_pages, int64_t n_pool_pages,
                            const int32_t *free_count, int32_t *free_left, int batch,
                            int32_t *dev_status, void *stream);

/*
 * kvc_ragged_plan -- a step's places.  Request b holds cached[b] tokens in the
 * ceil(cached[b] / page_size) first pages of its table row and brings
 * new_tokens[b]; the pages that it lacks are popped off the stack, request by
 * request, lower pages first, and written into the table.  offsets, positions and
 * slots as above; len as kvc_seq_lengths(KVC_CONTIGUOUS) would: past_abs =
 * cache_past = cached, total_abs = cache_total = cached + new_tokens, evict = 0,
 * for use with the other calls of a paged cache.
 * A rejected request has lengths -1, takes no page, and its rows of positions and
 * slots are -1 (they keep their place in the buffer):
 *   cached or new_tokens negative, or their sum past 2^31 - 1: KVC_DEV_SEQLEN_RANGE
 *   (it takes no place); tokens past the table's row, past `tokens` rows, or pages
 *   that the stack has not left (a request that wants pages after it is then
 *   rejected too): KVC_DEV_CAPACITY; new tokens that would go on in a page whose id
 *   is outside the pool: KVC_DEV_INDEX_OOB.
 * A popped id outside the pool sets KVC_DEV_INDEX_OOB; its entry and slots are -1.
 * offsets never exceed `tokens`.  positions, slots 16-byte aligned.
 */
kvc_status kvc_ragged_plan(const int32_t *cached, const int32_t *new_tokens, int32_t *block_table,
                           int max_pages, int page_size, const int32_t *free_pages,
                           int64_t n_pool_pages, const int32_t *free_count, int32_t *free_left,
                           int batch, int tokens, int32_t *offsets, kvc_lengths len,
                           int32_t *positions, int32_t *slots, int32_t *dev_status, void *stream);

/*
 * kvc_rope_tables -- the cos and sin tables that the calls here take, for
 * positions first, first + 1, ...: cos_table[p][i] = magnitude * cos((first + p) *
 * speed_i), sin likewise, i < rotary_dim / 2.  With speed = base^(-2 i / rotary_dim)
 *   KVC_ROPE_PLAIN   speed_i = speed
 *   KVC_ROPE_LINEAR  speed_i = speed / factor
 *   KVC_ROPE_BASE    speed_i = speed with base * factor^(rotary_dim / (rotary_dim - 2))
 *   KVC_ROPE_PARTS   a pair that goes round `high` times or more within `trained`
 *                    positions keeps its speed, one that goes round `low` times or
 *                    less has speed / factor, and between them g = (trained * speed /
 *                    2 pi - low) / (high - low): g * speed + (1 - g) * speed / factor
 *                    (a ramp over the rounds, not over a pair's index between two
 *                    indices rounded to whole numbers: a model that was extended by
 *                    the latter wants tables of its own)
 * Speeds are float64; the angle that a speed has at a position is reduced in whole
 * numbers, to 2^-32 of a turn at any position, so that far positions are as exact as
 * near ones: off by a float32 rounding or two, beside the few 2^-53 of itself that the
 * speed, and with it the angle, is off (up to positions of 2^27 that is less).
 * cos_table, sin_table  device float32 [positions, rotary_dim / 2] (4-byte aligned; the
 *             calls that read them want 16).
 * positions   up to 2^31 - 1; first >= 0, first + positions up to 2^31 (KVC_ERR_SHAPE).
 * rotary_dim  even, 2..256 (KVC_ERR_UNSUPPORTED above).  base > 0; factor > 0
 *             (ignored by KVC_ROPE_PLAIN); KVC_ROPE_PARTS: trained >= 1, low < high;
 *             all finite, magnitude also as a float32 (KVC_ERR_SHAPE).
 */
kvc_status kvc_rope_tables(float *cos_table, float *sin_table, int64_t first, int64_t positions,
                           int rotary_dim, double base, int scaling, double factor,
                           int64_t trained, double low, double high, double magnitude,
                           void *stream);

/*
 * kvc_ragged_append -- from the projections of a packed batch to attention: each
 * head's query and key is normed (x / sqrt(mean x^2 + eps) * weight, over the
 * head's head_dim values; not where the weight is NULL) and its first rotary_dim
 * columns rotated at the token's position, in float32 with one rounding at the
 * end; queries go to q_out, K and V rows (V as given) to the token's slot.
 * Pairs are (i, i + rotary_dim / 2), or with interleaved != 0 (2 i, 2 i + 1), with
 * entry i of the tables; the other columns stay.  Products and sums of the rotation
 * are rounded separately, so that without a norm and with rotary_dim = head_dim a
 * row is bit for bit that of kvc_paged_append.
 * q, k, v    device [tokens, heads, head_dim], the heads of a token dense, tokens
 *            q_stride, k_stride, v_stride elements apart (slices of one projection's
 *            output): multiples of 8, 16-byte aligned.
 * q_out      device [tokens, q_heads, head_dim]; may be q where that is dense.
 * q_weight, k_weight  device [head_dim] of `dtype`, or NULL.
 * rope_cos, rope_sin  device float32 [rope_max_pos, rotary_dim / 2], or NULL (no
 *            rotation; rotary_dim is then ignored).
 * A token with slot < 0 is skipped: its row of q_out stays as it was.  So is one
 * with a slot outside the pool (KVC_DEV_INDEX_OOB) or a position outside the tables
 * (KVC_DEV_ROPE_RANGE).  Two tokens with one slot leave parts of either there.
 * KVC_BF16/KVC_F16; head_dim a multiple of 16 up to 256, rotary_dim a multiple of 16
 * up to head_dim, q_heads and kv_heads up to 32767 (KVC_ERR_UNSUPPORTED).  q_out and the pools may not overlap what is
 * read (KVC_ERR_SHAPE).
 */
kvc_status kvc_ragged_append(void *q_out, void *k_pool, void *v_pool, const void *q, const void *k,
                             const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             const void *q_weight, const void *k_weight, float eps,
                             const int32_t *positions, const int32_t *slots, int tokens,
                             int q_heads, int kv_heads, int64_t n_pool_pages, int page_size,
                             int head_dim, int dtype, int rotary_dim, int interleaved,
                             const float *rope_cos, const float *rope_sin, int64_t rope_max_pos,
                             int32_t *dev_status, void *stream);

/*
 * kvc_gqa_ragged -- the attention of the new tokens of a packed batch after their
 * K and V are in the cache (kvc_ragged_append): the token at position p of request
 * b sees the rows of that request's positions 0..p, with a local window W > 0 those
 * less than W positions back.  Prompts, chunks of prompts over what is cached and
 * single tokens go together in one call.
 * out, q     device [tokens, q_heads, head_dim], q rotated; out may not overlap
 *            what is read (KVC_ERR_SHAPE).
 * offsets, len  as kvc_ragged_plan wrote them.  A request with lengths -1 keeps its
 *            rows of `out`, as do rows behind the last request's.  So does one whose
 *            offsets are outside [0, tokens] or not total_abs - past_abs apart
 *            (KVC_DEV_SEQLEN_RANGE), or with more tokens than its row of the table
 *            has room for, or than 2^31 - 512 (KVC_DEV_CAPACITY).  A page id outside the pool among the
 *            rows that are read sets KVC_DEV_INDEX_OOB (that request's output is then
 *            undefined).
 * page_size  a multiple of 16 (KVC_ERR_SHAPE).
 * KVC_BF16/KVC_F16, head_dim 64, 128 or 256, q_heads / kv_heads any whole number up
 * to 16, kv_heads <= 32767, batch <= 65535 (KVC_ERR_UNSUPPORTED); n_pool_pages *
 * page_size * kv_heads and tokens * q_heads below 2^31 (KVC_ERR_CAPACITY); scale 0 ->
 * 1 / sqrt(head_dim).
 * Beside the result, the softmax weights are rounded to the cache's type.  Scores
 * (q . k times scale) up to 1e30 in magnitude; beyond, the output may be NaN.
 * A NaN or an infinity in a column of a V row that a token sees makes that column of
 * its output NaN, whatever the row's weight; a NaN in a K row that it sees makes all
 * of them NaN.  What it does not see may hold anything; table entries before the page of
 * the first row that a request's first token sees are not read (pages that a window has
 * left behind may be given back).
 * workspace  device, kvc_gqa_ragged_workspace_size(...) bytes on the current device,
 *            256-byte aligned, apart from every other argument (KVC_ERR_SHAPE).
 *            Calls that may overlap on the GPU need their own.
 */
kvc_status kvc_gqa_ragged(void *out, const void *q, const void *k_pool, const void *v_pool,
                          const int32_t *offsets, const int32_t *block_table, int max_pages,
                          int64_t n_pool_pages, int page_size, kvc_lengths len, int batch,
                          int tokens, int q_heads, int kv_heads, int head_dim, int dtype,
                          int local_window_size, float scale, void *workspace,
                          size_t workspace_bytes, int32_t *dev_status, void *stream);

/* Bytes of workspace kvc_gqa_ragged needs for these sizes (0 on bad sizes). */
size_t kvc_gqa_ragged_workspace_size(int batch, int tokens, int q_heads, int kv_heads,
                                     int head_dim);

/* Human-readable name of a status code (static storage). */
const char *kvc_status_string(kvc_status status);

/* KVC_ABI_VERSION of the loaded library. */
int kvc_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KVC_H */
