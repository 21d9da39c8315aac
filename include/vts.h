/*
 * vts.h -- exact batched variable-length top-K selection and the operators
 * that follow it in a decode step (C ABI).
 *
 * The selections, asynchronous on the caller's HIP stream, exact with ties
 * interchangeable:
 *
 *   vts_topk_varlen                 decode-step top-k with per-request lengths
 *   vts_topk_varlen_ordered         the same in canonical order with a tie-break
 *   vts_topk_page_table_transform   top-k over row windows, fused with a
 *                                   page-table translation of the indices
 *
 * The decode-step operators over a paged KV cache (further down):
 *
 *   vts_tree_attention              attention of drafted tokens
 *   vts_attention_weight_add        attention weight per cached entry
 *   vts_evict_cache                 eviction by that weight
 *   vts_verify_draft                acceptance of drafted tokens
 *
 * and what brings a request that far:
 *
 *   vts_write_cache                 head norms, positions, keys and values into
 *                                   the cache, in 16, 8 or 4 bits
 *   vts_read_cache                  cached rows of listed slots
 *   vts_prompt_attention            attention of packed prompts
 *   vts_tree_attention_microscaled  vts_tree_attention over 8- or 4-bit caches
 *
 * The unprefixed names topk_varlen and topk_page_table_transform are exported
 * as aliases of the two entry points.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are HIP device memory (or memory the device can
 *     read/write directly); the caller owns all of it.  The library allocates
 *     nothing during a call and reads no device memory from the host, so a call
 *     may be captured into a HIP graph.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  The
 *     call only enqueues work; results are ready when the stream reaches it.
 *   - Integers in device arrays (lengths, starts, hints) may hold any value: the
 *     kernels clamp them as described and never read out of bounds because of
 *     them.
 *   - Return value: a vts_status.  Argument errors are detected on the host
 *     before any HIP call, so nothing is enqueued when a call fails.
 */
#ifndef VTS_H
#define VTS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of the score rows. */
typedef enum { VTS_F32 = 0, VTS_BF16 = 1, VTS_F16 = 2 } vts_dtype;

typedef enum {
    VTS_OK = 0,
    /* pre_idx was not usable (misaligned); it was ignored and the call ran
     * without a hint.  Results are unaffected.  (FlashInfer top_k_varlen doc,
     * `pre_idx`: a malformed hint is discarded with a warning.) */
    VTS_WARN_HINT_DISCARDED = 1,
    /* a shape, pointer, alignment or grouping argument breaks the contract
     * (FlashInfer top_k_varlen doc, "raises ValueError"). */
    VTS_ERR_INVALID = -1,
    /* the request is valid but outside what this library implements:
     * top_k above 16384 (above 2048 in the deterministic mode), a row of
     * width columns taking 2^31 bytes or more, or a device other than
     * gfx950. */
    VTS_ERR_UNSUPPORTED = -2,
    /* workspace pointer null or smaller than the matching *_workspace_bytes(). */
    VTS_ERR_WORKSPACE = -3,
    /* a HIP runtime call failed (no device, launch failure). */
    VTS_ERR_HIP = -4,
    /* vts_topk_varlen_noalloc: the shape needs more scratch than its fixed
     * device array holds. */
    VTS_ERR_TOO_LARGE = -5
} vts_status;

/* Workspace: device scratch used by rows that several workgroups share and by
 * candidate overflow.  Query its size with the matching *_workspace_bytes()
 * (a pure host function of the shape and element type), allocate it, fill it with zeros ONCE
 * (vts_workspace_init or any memset), then pass it to every call of that
 * shape.  Each call leaves it as it found it apart from the event counters of
 * vts_workspace_stats, so it never needs clearing again.  One workspace must
 * not be used by two calls that can run at the same time (for example on two
 * streams): give each stream its own.  (FlashInfer top_k_varlen doc,
 * `workspace`: a zero-initialised, self-restoring slab, one per stream.) */
size_t vts_topk_varlen_workspace_bytes(int64_t num_rows, int64_t width, int32_t top_k,
                                       int32_t dtype);
size_t vts_page_transform_workspace_bytes(int64_t num_rows, int64_t width, int32_t top_k,
                                          int32_t dtype);

/* Fills `bytes` bytes of `workspace` with zeros on `stream`. */
int vts_workspace_init(void* workspace, size_t bytes, void* stream);

/*
 * vts_topk_varlen -- FlashInfer "flashinfer.top_k_varlen" documentation
 * (signature, `seq_lens`, `compress_ratio`, `next_n`, `pre_idx`,
 * `return_values`, `out_indices`, `out_values`).
 *
 * logits      device, dtype elements, num_rows rows of `width` columns with
 *             consecutive rows `row_stride` elements apart (row_stride >=
 *             width); the base must be aligned to the element size.
 * seq_lens    device int32[num_rows / next_n]: KV-cache length of each request
 *             in KV-token units.  Row r belongs to request i = r / next_n as its
 *             t = r % next_n-th row and ranks its first
 *               n = max(0, (seq_lens[i] - next_n + t + 1) / compress_ratio)
 *             columns (integer division), clamped to `width`.
 * top_k       1 <= top_k <= 16384 (the range of FlashInfer's radix_filter
 *             backend, same page, `backend`).  Above 2048 the candidate
 *             lists live in LDS and the workspace (a larger workspace, see
 *             vts_topk_varlen_workspace_bytes) instead of registers.
 * next_n      >= 1, must divide num_rows.
 * compress_ratio >= 1.
 * pre_idx     device int32[num_rows / next_n, top_k] or NULL: the previous
 *             step's selection for each request, a sampling anchor only
 *             (FlashInfer top_k_varlen doc, `pre_idx`).  It is validated
 *             (16-byte aligned, else ignored with VTS_WARN_HINT_DISCARDED).
 *             The default path does not read it: its threshold comes from a
 *             strided sample of the row, which measured faster than also
 *             bounding it by the hint (the VTS_TUNE_HINT_RUNG switch turns
 *             that on; it reads the row at every hinted column and the next
 *             one).  Results never depend on it.
 * out_indices device int32[num_rows, top_k], 16-byte aligned.  Row r receives
 *             the column indices of its top-k (in no particular order) when
 *             n > top_k; the indices 0..n-1 followed by -1 when n <= top_k (all
 *             -1 when n == 0).
 * out_values  device dtype[num_rows, top_k], 16-byte aligned, or NULL (values
 *             not returned).  Bit copies of the selected elements, aligned
 *             with out_indices; slots holding -1 get the lowest finite value
 *             of the dtype (-FLT_MAX for fp32, 0xFF7F bf16, 0xFBFF fp16).
 * workspace   device, >= vts_topk_varlen_workspace_bytes(num_rows, width,
 *             top_k, dtype) bytes, 16-byte aligned, zeroed once (see above).
 *
 * Ties: all elements that compare equal are interchangeable; -0 and +0 are
 * ties.  +inf, -inf and subnormals rank exactly.  NaN is ordered above +inf
 * (sign clear) or below -inf (sign set).
 */
int vts_topk_varlen(const void* logits, int32_t dtype, int64_t num_rows, int64_t width,
                    int64_t row_stride, const int32_t* seq_lens, int32_t top_k, int32_t next_n,
                    int32_t compress_ratio, const int32_t* pre_idx, int32_t* out_indices,
                    void* out_values, void* workspace, size_t workspace_bytes, void* stream);

/*
 * vts_topk_varlen_noalloc -- vts_topk_varlen for callers that cannot allocate
 * device memory (code being captured into a HIP graph, tight serving loops,
 * harnesses that forbid allocation): the same arguments, results and errors,
 * without the workspace.  Its scratch is a fixed 32 MiB device array of the
 * library (one per device, held from the library's first use of that device
 * until the process ends); the call allocates nothing and frees nothing.
 *
 * Limit: the shape's workspace must fit the array with at least 3776
 * candidate slots per workgroup; otherwise VTS_ERR_TOO_LARGE and nothing is
 * enqueued.  That admits up to about 1100 row units (rows times workgroups
 * per row; e.g. 1024 rows of 262144 columns, or 64 rows split in four),
 * with fewer spill slots per unit than the workspace entry point when it is
 * near the limit (a spill beyond them takes the slower, still exact,
 * re-filtering path).
 *
 * Each call first clears the array's counters and row tickets on `stream`
 * (a small kernel), then runs the selection.  Every call on one device shares
 * that device's array: calls that can overlap on one device (two streams, two
 * threads) race and must be serialised by the caller.
 */
int vts_topk_varlen_noalloc(const void* logits, int32_t dtype, int64_t num_rows, int64_t width,
                            int64_t row_stride, const int32_t* seq_lens, int32_t top_k,
                            int32_t next_n, int32_t compress_ratio, const int32_t* pre_idx,
                            int32_t* out_indices, void* out_values, void* stream);

/* Tie-breaks of the deterministic mode (the *_ordered entry points). */
enum vts_tie_break {
    VTS_TIE_SMALL = 1,   /* of the values equal to the k-th, the smallest columns */
    VTS_TIE_LARGE = 2,   /* of the values equal to the k-th, the largest columns */
    /* added to SMALL or LARGE: the same selected set, written in no particular
     * order (no canonical sort); a row with n <= top_k is then the identity
     * 0..n-1 followed by -1, as in the unordered entry points */
    VTS_TIE_UNSORTED = 4
};

/*
 * vts_topk_varlen_ordered -- vts_topk_varlen in deterministic mode (the
 * FlashInfer page-size PR body on the SGLang PR #33237 page, "Description" and
 * "Performance": a deterministic post-sort of each row's outputs and a SMALL /
 * LARGE choice among tied values).  The order itself is not spelled out there;
 * value descending, then column ascending, is the reading taken here.
 *
 * Arguments, windows, errors and workspace are those of vts_topk_varlen,
 * except that top_k is at most 2048 (VTS_ERR_UNSUPPORTED above);
 * tie_break is VTS_TIE_SMALL or VTS_TIE_LARGE, optionally plus
 * VTS_TIE_UNSORTED (anything else: VTS_ERR_INVALID).  The selected set is
 * unique: every value above the k-th largest, then, of the values equal to
 * it, those at the smallest (SMALL) or largest (LARGE) columns.  Values
 * compare as numbers: -0 and +0 are equal (TensorRT-LLM PR #17821, "Test
 * coverage": signed zeros normalised), every NaN with the sign clear is
 * above +inf and equal to every other such NaN, every NaN with the sign set
 * below -inf and equal to every other such NaN.  Each row's outputs are in
 * canonical order: value descending, then column ascending; a row with
 * n <= top_k lists all n columns in that order, then -1.  The output is a
 * function of the inputs alone (bit-identical from run to run); out_values
 * are bit copies of the selected elements, as for vts_topk_varlen.  The sort
 * adds an epilogue per row (about 66 LDS compare-exchange rounds at top_k
 * 2048); VTS_TIE_UNSORTED skips it.
 */
int vts_topk_varlen_ordered(const void* logits, int32_t dtype, int64_t num_rows, int64_t width,
                            int64_t row_stride, const int32_t* seq_lens, int32_t top_k,
                            int32_t next_n, int32_t compress_ratio, const int32_t* pre_idx,
                            int32_t* out_indices, void* out_values, void* workspace,
                            size_t workspace_bytes, void* stream, int32_t tie_break);

/*
 * vts_topk_page_table_transform -- top-k over row windows with the compact
 * page-table transform (FlashInfer page-size PR body quoted on the SGLang
 * PR #33237 page, "Description"; `lengths` / `row_starts` as in SGLang's
 * fast_topk_v2, TopK_Ops page, I/O contract).
 *
 * scores       device, dtype, num_rows rows, `width` columns, `row_stride`
 *              elements apart (row_stride >= width).
 * lengths      device int32[num_rows]: valid length of each row's window.
 * row_starts   device int32[num_rows] or NULL (all 0): first column of each
 *              row's window, in score elements.  The window is
 *              [row_start, row_start + n) with n = clamp(length, 0,
 *              width - row_start); a start outside [0, width] gives n = 0.
 * src_page_table device int32, num_rows rows of page_table_width entries,
 *              page_table_stride entries apart.
 * page_table_row_starts device int32[num_rows] or NULL: first page-table entry
 *              of each row, in page-table entries.  NULL means the row start
 *              (row_starts, or 0); when page_size > 1 and row_starts is given
 *              it is required.
 * page_size    1 <= page_size <= 2^30.
 * top_k        1 <= top_k <= 16384.
 * out          device int32[num_rows, top_k], 16-byte aligned: for each
 *              selected window-relative index idx,
 *                src_page_table[r, pt_start + idx / page_size] * page_size
 *                  + idx % page_size,
 *              and -1 in unused slots.  A page-table entry outside
 *              [0, page_table_width) also yields -1.
 * out_raw_indices device int32[num_rows, top_k] or NULL: the window-relative
 *              indices themselves, positionally aligned with `out`, -1 in
 *              unused slots.  Must not overlap `out`.
 * workspace    as for vts_topk_varlen, sized by vts_page_transform_workspace_bytes.
 */
int vts_topk_page_table_transform(const void* scores, int32_t dtype, int64_t num_rows,
                                  int64_t width, int64_t row_stride, const int32_t* lengths,
                                  const int32_t* row_starts, const int32_t* src_page_table,
                                  int64_t page_table_stride, int64_t page_table_width,
                                  const int32_t* page_table_row_starts, int32_t page_size,
                                  int32_t top_k, int32_t* out, int32_t* out_raw_indices,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * vts_topk_page_table_transform_ordered -- vts_topk_page_table_transform in
 * the deterministic mode of vts_topk_varlen_ordered (same page, "Description":
 * `out_raw_indices` stays positionally aligned with `out` through the
 * deterministic post-sort).  The selection over each window, its order and
 * tie_break are those of vts_topk_varlen_ordered, on window-relative indices;
 * `out` holds their translations slot by slot.
 */
int vts_topk_page_table_transform_ordered(
    const void* scores, int32_t dtype, int64_t num_rows, int64_t width, int64_t row_stride,
    const int32_t* lengths, const int32_t* row_starts, const int32_t* src_page_table,
    int64_t page_table_stride, int64_t page_table_width, const int32_t* page_table_row_starts,
    int32_t page_size, int32_t top_k, int32_t* out, int32_t* out_raw_indices, void* workspace,
    size_t workspace_bytes, void* stream, int32_t tie_break);

/*
 * vts_topk_transform_ragged -- top-k over row windows with the ragged-KV index
 * transform (SGLang TopK_Ops page, fast_topk_transform_ragged_fused: the
 * offset of each row's top-k indices in a ragged KV buffer).
 *
 * scores, lengths, row_starts, top_k, workspace: as for
 *              vts_topk_page_table_transform (workspace sized by
 *              vts_page_transform_workspace_bytes).
 * topk_indices_offset device int32[num_rows]: added to every selected
 *              window-relative index of the row (int32 arithmetic; keeping
 *              the sums in range is the caller's contract).
 * out          device int32[num_rows, top_k], 16-byte aligned: idx +
 *              topk_indices_offset[r] for each selected window-relative
 *              index idx, -1 in unused slots.
 * out_raw_indices device int32[num_rows, top_k] or NULL: the window-relative
 *              indices, positionally aligned with `out`, -1 in unused slots.
 *              Must not overlap `out`.
 */
int vts_topk_transform_ragged(const void* scores, int32_t dtype, int64_t num_rows, int64_t width,
                              int64_t row_stride, const int32_t* lengths,
                              const int32_t* row_starts, const int32_t* topk_indices_offset,
                              int32_t top_k, int32_t* out, int32_t* out_raw_indices,
                              void* workspace, size_t workspace_bytes, void* stream);

/* vts_topk_transform_ragged in the deterministic mode (see
 * vts_topk_page_table_transform_ordered). */
int vts_topk_transform_ragged_ordered(const void* scores, int32_t dtype, int64_t num_rows,
                                      int64_t width, int64_t row_stride, const int32_t* lengths,
                                      const int32_t* row_starts,
                                      const int32_t* topk_indices_offset, int32_t top_k,
                                      int32_t* out, int32_t* out_raw_indices, void* workspace,
                                      size_t workspace_bytes, void* stream, int32_t tie_break);

/*
 * vts_topk_transform_page1 -- top-k over row windows with the page-size-1
 * transform of SGLang's fast_topk_transform_fused (TopK_Ops page): each row
 * is a query of one request, found through `cu_seqlens_q`, and each selected
 * window-relative index (a KV position of that request) is replaced by the
 * request's page-table entry for it.
 *
 * scores, lengths, row_starts, top_k: as for vts_topk_page_table_transform.
 * page_table   device int32, num_batches rows of page_table_width entries,
 *              page_table_stride entries apart: row b maps KV positions of
 *              request b to physical KV slots.
 * cu_seqlens_q device int32[num_batches + 1], non-decreasing: rows
 *              [cu_seqlens_q[b], cu_seqlens_q[b + 1]) belong to request b.
 * out          device int32[num_rows, top_k], 16-byte aligned:
 *              page_table[b(r), idx] for each selected index idx, -1 in
 *              unused slots, where idx >= page_table_width, and in every slot
 *              of a row outside [cu_seqlens_q[0], cu_seqlens_q[num_batches]).
 * out_raw_indices device int32[num_rows, top_k] or NULL: the window-relative
 *              indices, positionally aligned with `out`; must not overlap it.
 * workspace    as for vts_topk_varlen, sized by vts_page_transform_workspace_bytes;
 *              the call also writes a row-to-request map into it (a small
 *              kernel on `stream` before the selection).
 */
int vts_topk_transform_page1(const void* scores, int32_t dtype, int64_t num_rows, int64_t width,
                             int64_t row_stride, const int32_t* lengths, const int32_t* row_starts,
                             const int32_t* page_table, int64_t page_table_stride,
                             int64_t page_table_width, const int32_t* cu_seqlens_q,
                             int64_t num_batches, int32_t top_k, int32_t* out,
                             int32_t* out_raw_indices, void* workspace, size_t workspace_bytes,
                             void* stream);

/* vts_topk_transform_page1 in the deterministic mode (see
 * vts_topk_page_table_transform_ordered). */
int vts_topk_transform_page1_ordered(const void* scores, int32_t dtype, int64_t num_rows,
                                     int64_t width, int64_t row_stride, const int32_t* lengths,
                                     const int32_t* row_starts, const int32_t* page_table,
                                     int64_t page_table_stride, int64_t page_table_width,
                                     const int32_t* cu_seqlens_q, int64_t num_batches,
                                     int32_t top_k, int32_t* out, int32_t* out_raw_indices,
                                     void* workspace, size_t workspace_bytes, void* stream,
                                     int32_t tie_break);

/* Aliases with the operation names of the pages. */
int topk_varlen(const void* logits, int32_t dtype, int64_t num_rows, int64_t width,
                int64_t row_stride, const int32_t* seq_lens, int32_t top_k, int32_t next_n,
                int32_t compress_ratio, const int32_t* pre_idx, int32_t* out_indices,
                void* out_values, void* workspace, size_t workspace_bytes, void* stream);
int topk_page_table_transform(const void* scores, int32_t dtype, int64_t num_rows, int64_t width,
                              int64_t row_stride, const int32_t* lengths,
                              const int32_t* row_starts, const int32_t* src_page_table,
                              int64_t page_table_stride, int64_t page_table_width,
                              const int32_t* page_table_row_starts, int32_t page_size,
                              int32_t top_k, int32_t* out, int32_t* out_raw_indices,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Decode-step operators over a paged KV cache.
 *
 * The four calls below are what a decode step with drafted tokens does after
 * the selection: attention of the drafted tokens, verification of them,
 * attention weight accumulated per cached entry, and eviction by it.  They
 * share one description of the cache.  A length counts the drafted tokens, as
 * in vts_topk_varlen (next_n): of a request with length n and `draft` drafted
 * tokens, positions [0, n - draft) are the prefix and position n - draft + i is
 * drafted token i.  Lengths are clamped to [0, page_table_width * page_size].
 *
 * A page-table entry outside [0, num_pages) means that its positions are not
 * there: they are skipped, whatever the length says.
 *
 * k, v       device, dtype (VTS_BF16 or VTS_F16), 16-byte aligned: num_pages
 *            pages of page_size positions of kv_heads rows of head_dim (64 or
 *            128) consecutive elements.
 * k_strides, v_strides  elements between pages, positions of a page, and
 *            heads, multiples of 8 (ignored for a dimension of one): any order
 *            of the three dimensions is possible.  A cache spans at most 2^32
 *            16-byte vectors and 2^31 - 1 positions.
 * page_table device int32[batch, page_table_width], rows page_table_stride
 *            entries apart.
 * seq_lens   device int32[batch].
 */
typedef struct {
    const void* k;
    const void* v;
    int64_t k_strides[3];
    int64_t v_strides[3];
    const int32_t* page_table;
    int64_t page_table_stride;
    int64_t page_table_width;
    const int32_t* seq_lens;
    int64_t num_pages;
    int32_t page_size;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t batch;
    int32_t dtype;
} vts_paged_cache;

/*
 * vts_tree_attention -- attention of drafted tokens over the cache.
 *
 *   out[b, t, h] = sum_j p_j v_j,   p = softmax_j(scale * q[b, t, h] . k_j)
 *   lse[b, t, h] = log sum_j exp(scale * q . k_j)
 *
 * over the places j that row (b, t) sees; query head h uses KV head
 * h / (heads / kv_heads).  Without `slots` these are the prefix and the drafted
 * tokens i with bit i of tree_mask[b, t] set (tree_mask NULL: i <= t, a chain).
 * With `slots` they are the row's listed slots (page * page_size + position in
 * the page, as vts_topk_page_table_transform writes them; slots outside the
 * cache, such as the -1 of unused entries, are skipped) and, if tree_mask is
 * given, the drafted tokens it names.  A row that sees nothing, or nothing of
 * weight, gets zeros and an lse of -inf.  Values in places that a row does not
 * see never reach it, infinities and NaN among them; in those that it sees they
 * count as the weight says, so that with a score of -inf they give NaN.  A row with
 * a score that is NaN or +inf gets NaN, its lse too.
 *
 * q          device, the cache's dtype, 16-byte aligned; q_strides: elements
 *            between requests, drafted tokens and heads, multiples of 8.
 * draft      1..64 drafted tokens per request (1 for plain decoding).
 * heads      a multiple of kv_heads, at most 8192.
 * tree_mask  device int64[batch, draft] or NULL.
 * slots      device int32[batch, draft, top_k] or NULL (then top_k is 0).
 * out        device, dtype[batch, draft, heads, head_dim], 16-byte aligned; must
 *            not overlap q or the caches.
 * lse        device float[batch, draft, heads] or NULL.
 * workspace  device, 16-byte aligned, at least
 *            vts_tree_attention_workspace_bytes(...) bytes, zeroed once.  The
 *            calls of this section leave their workspaces fit for each
 *            other, of any shape, but not for the selections.
 *
 * Sums are 32-bit; the probabilities are rounded to dtype for the product with
 * V, fp16's in a range that keeps their precision down to 2^-25 of the row's
 * greatest.  The result depends on the shape and the lengths but not on timing.
 * Work is shared in units of 32 to 128 places over the batch's real lengths, so
 * ragged batches cost what their lengths say.
 */
size_t vts_tree_attention_workspace_bytes(int32_t batch, int32_t draft, int32_t heads,
                                          int32_t kv_heads, int32_t head_dim, int32_t top_k);
int vts_tree_attention(const vts_paged_cache* cache, const void* q, const int64_t* q_strides,
                       int32_t draft, int32_t heads, const int64_t* tree_mask,
                       const int32_t* slots, int32_t top_k, float scale, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * vts_attention_weight_add -- attention weight accumulated per cached entry:
 *
 *   weights[b, hk, j] += sum over t with row_keep[b, t] != 0 and the query
 *       heads h of KV head hk of exp(scale * q[b, t, h] . k_j - lse[b, t, h])
 *
 * for every position j < width that row (b, t) sees (as vts_tree_attention
 * without slots).  Rows whose lse is -inf add nothing.  cache->v is not read
 * and may be NULL.  The sum over rows is in a fixed order.
 *
 * lse        device float[batch, draft, heads], of vts_tree_attention.
 * row_keep   device uint8[batch, draft] or NULL (all rows): for instance the
 *            drafted tokens that were accepted.
 * weights    device float, `width` consecutive per request and KV head, at
 *            the strides given (elements); no two of these rows may have an
 *            element in common.
 */
int vts_attention_weight_add(const vts_paged_cache* cache, const void* q,
                             const int64_t* q_strides, int32_t draft, int32_t heads,
                             const int64_t* tree_mask, const float* lse, const uint8_t* row_keep,
                             float scale, float* weights, int64_t weights_batch_stride,
                             int64_t weights_head_stride, int64_t width, void* stream);

/*
 * vts_evict_cache -- shrinks every request to at most `keep` entries.
 *
 * Of a request's n entries (its length, at most `width`) and each KV head by
 * itself: if n <= keep all stay; else the first `sinks`, the last `recent`, and
 * the entries of largest weight among the others stay, keep in all; of
 * equal weights the lower positions stay, and weights order as in
 * vts_topk_varlen_ordered (-0 equals +0, a NaN ranks by its sign beyond the
 * infinities).  The kept entries' K and V rows go, in the order of their
 * positions, to the pages of out_page_table, which must not be pages that are
 * read (k_out may be the cache itself, with fresh pages); their positions to
 * kept[b, hk, 0..] (-1 in unused entries) and their weights to
 * out_weights[b, hk, 0..] (0 in unused entries); min(n, keep) to out_lens[b].
 * An entry whose page is not there is moved as zeros; a row whose out_page_table
 * entry is outside [0, out_pages) is not written.
 *
 * sinks + recent <= keep; out_page_table_width >= ceil(keep / page_size).  At most
 * 2^21 pairs of request and KV head, and 2^23 blocks of 64 kept entries in all.
 */
int vts_evict_cache(const vts_paged_cache* cache, const float* weights,
                    int64_t weights_batch_stride, int64_t weights_head_stride, int64_t width,
                    int32_t keep, int32_t sinks, int32_t recent, void* k_out,
                    const int64_t* k_out_strides, void* v_out, const int64_t* v_out_strides,
                    int64_t out_pages, const int32_t* out_page_table,
                    int64_t out_page_table_stride, int64_t out_page_table_width, int32_t* kept,
                    int32_t* out_lens, float* out_weights, void* stream);

/*
 * vts_verify_draft -- verification of drafted tokens against the target's
 * probabilities from given random numbers; the accepted tokens and the next one
 * are distributed as the target's own.
 *
 * Node t of a request is drafted token draft_tokens[b, t], hung from node
 * parents[b, t] < t (-1: the context; parents NULL: a chain).  Row n + 1 of
 * target_probs[b] is the target's distribution after node n (row 0: after the
 * context), row n + 1 of draft_probs[b] the distribution that the children of
 * node n were drawn from (never read for the last node, so `draft` rows).
 * From the context on, a node's children are tried in index order: the child
 * of token x is accepted if u q(x) < r(x), u = uniforms[b, t], where r begins
 * as the target's row p and turns into max(r - q, 0), normalised, at each
 * rejection.  draft_probs NULL: the tokens were chosen, not drawn, and q is 1
 * at x and 0 elsewhere.  Where no child is accepted, the next token is the
 * first v whose running sum of r passes uniforms[b, draft] times r's whole sum
 * (if r has no mass, p's; if p has none, -1).
 *
 * At most 64 drafted tokens, 2^21 requests and 2^31 - 2^16 - 1 tokens of vocabulary.
 * Probabilities are used as they are given; NaN and negative values count as
 * 0.  A token outside [0, vocab) or a parent outside [-1, t) makes a node that
 * is not there: it is neither accepted nor rejected, and takes nothing from r (a
 * request with fewer drafts is padded with tokens of -1).  Sums and comparisons
 * are in 64 bits.
 *
 * path       device int32[batch, draft]: the accepted nodes in order, then -1.
 * count      device int32[batch]: how many.
 * next_token device int32[batch].
 * workspace  as for vts_tree_attention, sized by
 *            vts_verify_draft_workspace_bytes.
 */
size_t vts_verify_draft_workspace_bytes(int64_t batch, int64_t vocab);
int vts_verify_draft(const void* target_probs, int32_t dtype, int64_t target_batch_stride,
                     int64_t target_row_stride, const void* draft_probs,
                     int64_t draft_batch_stride, int64_t draft_row_stride,
                     const int32_t* draft_tokens, const int32_t* parents, const float* uniforms,
                     int64_t batch, int32_t draft, int64_t vocab, int32_t* path, int32_t* count,
                     int32_t* next_token, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Filling a paged cache, microscaled caches, and prompts.
 *
 * A microscaled cache holds its rows in 8 or 4 bits to an element and one power
 * of two to 32 consecutive ones.  Its vts_paged_cache has the dtype of the queries
 * and outputs; k and v point to bytes, rows of head_dim (bits 8) or head_dim / 2
 * (bits 4) of them, 16-byte aligned, k_strides and v_strides in bytes, multiples of
 * 16.  Elements are E4M3 numbers (bits 8: sign, 4 bits of exponent with bias 7, 3 of
 * mantissa; 0x7F and 0xFF are NaN) or E2M1 (bits 4: 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a
 * sign, the first of two in a byte's low half).  A scale is one byte, E8M0: 2^(x - 127), NaN
 * for 255.  Values are rounded to the queries' dtype where they are used: bf16 holds
 * every number of the format from 2^-133 to its own largest, fp16 those of its own
 * range, and what lies past it is an infinity.  So are values next to the dtype's
 * largest that the format rounds up to the next power of two: written with 4 bits from
 * 1.75 times its largest power of two on (57344 in fp16), with 8 from 1.9375 (63488).
 *
 * k, v       device: head_dim / 32 bytes per row, aligned to that.
 * k_strides, v_strides  bytes between pages, positions of a page, and heads,
 *            multiples of head_dim / 32 (ignored for a dimension of one).
 */
typedef struct {
    const uint8_t* k;
    const uint8_t* v;
    int64_t k_strides[3];
    int64_t v_strides[3];
    int32_t bits;
} vts_microscales;

/*
 * vts_tree_attention_microscaled -- vts_tree_attention over a microscaled cache,
 * with the same arguments, masks, sums and guarantees; the workspace serves caches of
 * 8 and of 4 bits.
 */
size_t vts_tree_attention_microscaled_workspace_bytes(int32_t batch, int32_t draft, int32_t heads,
                                                      int32_t kv_heads, int32_t head_dim, int32_t top_k);
int vts_tree_attention_microscaled(const vts_paged_cache* cache, const vts_microscales* scales, const void* q,
                                   const int64_t* q_strides, int32_t draft, int32_t heads,
                                   const int64_t* tree_mask, const int32_t* slots, int32_t top_k, float scale,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * vts_write_cache -- new tokens' queries made ready and their keys and values put
 * into the cache:
 *
 *   x'    = x / sqrt(mean(x^2) + eps) * norm          (q and k, per head; norm NULL:
 *                                                      x' = x)
 *   (a, b) -> (a c - b s, b c + a s)                  (q and k, per pair of x';
 *                                                      rotary NULL: not turned)
 *
 * where pair i of a row is elements i and i + rot / 2 (interleaved: 2 i and 2 i + 1),
 * i < rot / 2, and c = rotary[position][i], s = rotary[position][rot / 2 + i];
 * elements from rot on are not turned.  q goes to q_out, k (and to k_out, if given) and
 * v to the slot's rows of the cache.  Rows are computed in 32 bits and rounded once.
 * For a microscaled cache k is computed in 64: each block of 32 elements gets the least
 * power of two (from 2^-127) with which its largest magnitude rounds to a number of the
 * format, and its elements, divided by that, are rounded to nearest, ties to even; a block
 * that holds an infinity or NaN gets the scale NaN.
 *
 * A slot outside the cache (-1 for padding) is not written; the token's q_out and
 * k_out are.  A token whose position is outside [0, max_position) gets zeros in q_out
 * and k_out and is not written.  The slots inside the cache have to be distinct: the
 * entry of one named twice holds parts of either token.  So do rows of the caches, and
 * of their scales, that overlap each other.  Nothing else of the cache changes.  page_table, seq_lens and batch of `cache` are not looked at.
 *
 * q, k, v    device, the cache's dtype, 16-byte aligned rows of head_dim elements;
 *            strides: elements between tokens and heads, multiples of 8.
 * q_norm, k_norm  device [head_dim], 16-byte aligned, of norm_dtype (VTS_F32 or the
 *            cache's dtype), or NULL.
 * rotary     device float[max_position, rot], 16-byte aligned, or NULL (then rot is
 *            0); rot: a multiple of 16, at most head_dim.
 * positions  device int32[tokens] (not read without rotary).
 * slots      device int32[tokens].
 * q_out      device, dtype[tokens, heads, head_dim], 16-byte aligned; k_out: the same
 *            with kv_heads, or NULL.  They must not overlap each other, the inputs
 *            or the caches.
 * At most 2^25 tokens.
 */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_strides[2];
    int64_t k_strides[2];
    int64_t v_strides[2];
    const void* q_norm;
    const void* k_norm;
    double eps;
    const float* rotary;
    int64_t max_position;
    const int32_t* positions;
    const int32_t* slots;
    int64_t tokens;
    void* q_out;
    void* k_out;
    int32_t heads;
    int32_t norm_dtype;
    int32_t rot;
    int32_t interleaved;
} vts_new_tokens;
int vts_write_cache(const vts_paged_cache* cache, const vts_microscales* scales, const vts_new_tokens* tokens,
                    void* stream);

/*
 * vts_read_cache -- the cached rows of listed slots, as rows of the cache's dtype:
 * k_out[i], v_out[i] = rows of all KV heads of slots[i], zeros for a slot outside the
 * cache.  A slot may be listed more than once.
 *
 * scales     of a microscaled cache, or NULL.
 * slots      device int32[count].
 * k_out, v_out  device, dtype[count, kv_heads, head_dim], 16-byte aligned; they must
 *            not overlap each other or the caches.
 * At most 2^33 / (kv_heads * head_dim / 8) slots.  page_table, seq_lens and batch of
 * `cache` are not looked at.
 */
int vts_read_cache(const vts_paged_cache* cache, const vts_microscales* scales, const int32_t* slots,
                   int64_t count, void* k_out, void* v_out, void* stream);

/*
 * vts_prompt_attention -- attention of packed prompts.
 *
 *   out[i, h] = sum_j p_j v_j,   p = softmax_j(scale * q[i, h] . k_j)
 *   lse[i, h] = log sum_j exp(scale * q . k_j)
 *
 * Sequence b has query rows [cu_q[b], cu_q[b + 1]) and key rows [cu_k[b], cu_k[b + 1]);
 * query head h uses KV head h / (heads / kv_heads).  causal: its queries are the last of
 * its keys, so of nq queries and nk keys query i sees the keys j <= i + nk - nq; else
 * all.  A row that sees nothing, or nothing of weight, gets zeros and an lse of
 * -inf.  Values of keys that a row does not see never reach it, infinities and NaN
 * among them; of keys that it sees they count as the weight says, so that with a score
 * of -inf they give NaN (0 times infinity).  A row with a score that is NaN or +inf gets
 * NaN, its lse too.  Rows of no sequence (before cu_q[0], from cu_q[batch] on) are left as
 * they were, or with `clear` get zeros and -inf.
 *
 * Entries of cu_q and cu_k are clamped to the rows there are; one below its
 * predecessor makes an empty sequence, after which what later sequences' rows get is
 * not defined (nothing outside the outputs is touched).
 *
 * Scores, maxima, sums and outputs are 32-bit; the probabilities are rounded to dtype
 * for the product with V, as in vts_tree_attention, and the sum takes them unrounded.
 *
 * q, k, v    device, dtype (VTS_BF16 or VTS_F16), 16-byte aligned rows of head_dim
 *            (64 or 128) elements, total_q of heads, total_k of kv_heads; strides:
 *            elements between tokens and heads, multiples of 8.
 * cu_q, cu_k device int32[batch + 1], ascending.
 * out        device, dtype[total_q, heads, head_dim], 16-byte aligned; must not
 *            overlap the inputs.
 * lse        device float[total_q, heads] or NULL.
 * workspace  device, 16-byte aligned, at least vts_prompt_attention_workspace_bytes(...)
 *            bytes, of any contents (NULL where that is 0: only few queries behind long
 *            contexts take any).
 *
 * total_q * heads, total_k and batch are below 2^31 - 1024, and kv_heads *
 * (total_q * (heads / kv_heads) / 128 + batch) below 2^24 - 64.
 */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_strides[2];
    int64_t k_strides[2];
    int64_t v_strides[2];
    const int32_t* cu_q;
    const int32_t* cu_k;
    int64_t batch;
    int64_t total_q;
    int64_t total_k;
    int32_t heads;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t dtype;
} vts_prompts;
size_t vts_prompt_attention_workspace_bytes(int64_t batch, int64_t total_q, int64_t total_k, int32_t heads,
                                            int32_t kv_heads, int32_t head_dim);
int vts_prompt_attention(const vts_prompts* prompts, int32_t causal, float scale, void* out, float* lse,
                         int32_t clear, void* workspace, size_t workspace_bytes, void* stream);

/* Human-readable text of a vts_status. */
const char* vts_status_string(int status);

/* Event counters kept in a workspace, copied to `out` (host, `count` <= 4
 * entries)
 * with a synchronous copy on `stream`, then cleared:
 *   out[0]  workgroups whose candidates overflowed and were re-filtered
 *   out[1]  rows whose sampled threshold kept fewer than top_k candidates
 *           and that were re-selected over the whole row
 *   out[2]  rows whose candidates outgrew on-chip memory (selected over the
 *           spilled workspace slots too)
 *   out[3]  rows with fewer than top_k keys at or above the likely threshold,
 *           so that the whole candidate list (keys at or above the safe
 *           threshold) was ranked */
int vts_workspace_stats(void* workspace, uint32_t* out, int32_t count, void* stream);

/* Plan log: with VTS_LOG=1 in the environment (read once per process), every
 * call prints one line to stderr naming the entry point, the shape, the
 * kernels (any-order, ordered, wide or hinted), the units per row, the row
 * placement and the device's compute units.  Results never depend on it. */

/* Diagnostic and test switches.  Each applies to the calls (and workspace-size
 * queries) of the thread that set it, nowhere else.  None of them changes
 * results, only which internal path computes them.
 *   VTS_TUNE_NSPLIT       workgroups per long row (0 = automatic, 1..32)
 *   VTS_TUNE_FORCE_PATH   0 normal, 1 every chunk uses the compaction filter,
 *                         2 every row is re-selected over the whole row
 *   VTS_TUNE_LDS_SLOTS    on-chip candidate slots before spilling to the
 *                         workspace (0 = default; 64..3776)
 *   VTS_TUNE_SPILL_SLOTS  candidate slots per workgroup, on chip and in the
 *                         workspace, before a chunk is re-filtered
 *                         (0 = default; 64..8192)
 *   VTS_TUNE_SAMPLE_SIGMA margin of the safe threshold rung in tenths of a
 *                         standard deviation of the sample count (0 = 50)
 *   VTS_TUNE_LIKELY_SIGMA margin of the likely rung, same unit (0 = 20; a
 *                         value >= the safe margin merges the two rungs)
 *   VTS_TUNE_MIN_CHUNK    valid columns per workgroup below which a row is not
 *                         split further (0 = default: 32768, and 128 KB of
 *                         columns for the length-balanced units of 512-row
 *                         batches; 256..2^20)
 *   VTS_TUNE_NO_BALANCE   1 turns off the length-balanced placement of rows on
 *                         compute units (0 = on where it applies)
 *   VTS_TUNE_HINT_RUNG    1: vts_topk_varlen calls with a pre_idx and top_k
 *                         <= 2048 also bound the safe threshold from below by the
 *                         k-th largest value read at the hinted columns
 *                         (0 = hint not read)
 * The workspace size follows the split count in force when it is queried.
 * Returns VTS_OK or VTS_ERR_INVALID for an unknown key or value. */
enum {
    VTS_TUNE_NSPLIT = 1,
    VTS_TUNE_FORCE_PATH = 2,
    VTS_TUNE_LDS_SLOTS = 3,
    VTS_TUNE_SPILL_SLOTS = 4,
    VTS_TUNE_SAMPLE_SIGMA = 5,
    VTS_TUNE_MIN_CHUNK = 6,
    VTS_TUNE_LIKELY_SIGMA = 7,
    VTS_TUNE_NO_BALANCE = 8,
    VTS_TUNE_HINT_RUNG = 9
};
int vts_set_tuning(int32_t key, int64_t value);

#ifdef __cplusplus
}
#endif

#endif /* VTS_H */
