// vts_decode_api.hip -- C ABI of the decode-step operators (attention over a
// paged cache, accumulated attention weight, eviction, draft verification):
// argument checks on the host before any HIP call, plans that are pure functions
// of the shape, and the launches.
#include "vts_decode_checks.h"

namespace {

using namespace vts;

// Whether rows of `width` elements at i * s + j * t, i < m and j < n, have no
// element in common.
bool rows_apart(int64_t m, int64_t s, int64_t n, int64_t t, int64_t width) {
    if (n <= 1 || (m > 1 && s < t)) {  // the larger stride first
        const int64_t m0 = m, s0 = s;
        m = n, s = t, n = m0, t = s0;
    }
    // m <= 1 here means that at most one stride counts
    if (n > 1 && t < width) return false;
    if (m <= 1) return true;
    if (s < width) return false;
    if (n <= 1) return true;
    // i rows on, the nearest of the others on either side; s >= t, so the loop
    // leaves their reach within n steps
    const __int128 last = (__int128)t * (n - 1);
    for (int64_t i = 1; i < m && (__int128)i * s < last + width; ++i) {
        const __int128 at = (__int128)i * s, below = at / t * t;
        if (at - (below < last ? below : last) < width) return false;
        if (below < last && below + t - at < width) return false;
    }
    return true;
}

// Workgroups per request: as many as the device holds at once (one of 16 waves
// on each compute unit; with two rounds of them 64 requests of 131072 fp32 took
// 49 us for 33), of at least 4096 values each.
int32_t verify_slices(int64_t batch, int64_t vocab) {
    if (batch < 1 || batch > MAX_TICKETS) return 1;
    int64_t s = CUS / batch;
    const int64_t most = (vocab + 4095) / 4096;
    if (s > most) s = most;
    if (s > 64) s = 64;  // 1024 segments, one to a thread of the joining workgroup
    return s < 1 ? 1 : (int32_t)s;
}

struct VerifyLayout {
    size_t sums, states, total;
};

VerifyLayout verify_layout(int64_t batch, int64_t vocab) {
    const size_t n = batch < 1 ? 1 : (size_t)batch;
    VerifyLayout v;
    v.sums = TICKET_BYTES;
    v.states = v.sums + align256(2 * n * verify_slices(batch, vocab) * 16 * sizeof(double));
    v.total = v.states + align256(2 * n * sizeof(VerifyState));
    return v;
}

}  // namespace

extern "C" {

size_t vts_tree_attention_workspace_bytes(int32_t batch, int32_t draft, int32_t heads, int32_t kv_heads,
                                          int32_t head_dim, int32_t top_k) {
    AttendPlan plan;
    if (batch < 0 || draft < 1 || draft > MAX_DRAFT || kv_heads < 1 || heads < kv_heads ||
        heads % kv_heads != 0 || heads > MAX_HEADS || head_dim < 1 || head_dim > 1024)
        return 0;
    if (attend_plan(batch, draft, heads, kv_heads, head_dim, top_k, 16, &plan) != VTS_OK) return 0;
    return plan.total;
}

int vts_tree_attention(const vts_paged_cache* cache, const void* q, const int64_t* q_strides,
                       int32_t draft, int32_t heads, const int64_t* tree_mask,
                       const int32_t* slots, int32_t top_k, float scale, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
    return attend(cache, nullptr, q, q_strides, draft, heads, tree_mask, slots, top_k, scale, out, lse,
                  workspace, workspace_bytes, stream, [&](const AttendParams& p) {
                      return launch_attend(cache->dtype, cache->head_dim, p,
                                           static_cast<hipStream_t>(stream));
                  });
}

int vts_attention_weight_add(const vts_paged_cache* cache, const void* q,
                             const int64_t* q_strides, int32_t draft, int32_t heads,
                             const int64_t* tree_mask, const float* lse, const uint8_t* row_keep,
                             float scale, float* weights, int64_t weights_batch_stride,
                             int64_t weights_head_stride, int64_t width, void* stream) {
    WeighParams p;
    memset(&p, 0, sizeof(p));
    int st = paged(cache, draft, heads, false, &p.c);
    if (st != VTS_OK) return st;
    if (isnan(scale) || width < 0 || weights_batch_stride < 0 || weights_head_stride < 0)
        return VTS_ERR_INVALID;
    if (p.c.batch == 0 || width == 0) return VTS_OK;
    if (!rows_apart(p.c.batch, weights_batch_stride, p.c.kv_heads, weights_head_stride, width))
        return VTS_ERR_INVALID;
    st = check_q(q, q_strides, p.c);
    if (st != VTS_OK) return st;
    if (lse == nullptr || weights == nullptr || !aligned(lse, 4) || !aligned(weights, 4))
        return VTS_ERR_INVALID;
    st = check_device(stream);
    if (st != VTS_OK) return st;
    p.q = q;
    p.q_batch = q_strides[0];
    p.q_row = q_strides[1];
    p.q_head = q_strides[2];
    p.tree_mask = tree_mask;
    p.lse = lse;
    p.row_keep = row_keep;
    p.scale_log2e = (float)((double)scale * 1.4426950408889634);
    p.weights = weights;
    p.w_batch = weights_batch_stride;
    p.w_head = weights_head_stride;
    p.width = (int32_t)(width > INT32_MAX ? INT32_MAX : width);
    p.rows = draft * p.c.group;
    p.heads_on_waves = p.c.kv_heads % 4 == 0 && p.rows <= 64;
    p.workers = 2 * CUS;
    return launch_weigh(cache->dtype, cache->head_dim, p, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? VTS_OK
               : VTS_ERR_HIP;
}

int vts_evict_cache(const vts_paged_cache* cache, const float* weights,
                    int64_t weights_batch_stride, int64_t weights_head_stride, int64_t width,
                    int32_t keep, int32_t sinks, int32_t recent, void* k_out,
                    const int64_t* k_out_strides, void* v_out, const int64_t* v_out_strides,
                    int64_t out_pages, const int32_t* out_page_table,
                    int64_t out_page_table_stride, int64_t out_page_table_width, int32_t* kept,
                    int32_t* out_lens, float* out_weights, void* stream) {
    EvictParams p;
    memset(&p, 0, sizeof(p));
    int st = paged(cache, 1, cache ? cache->kv_heads : 1, true, &p.c);
    if (st != VTS_OK) return st;
    if (keep < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep)
        return VTS_ERR_INVALID;
    if (width < 1 || weights_batch_stride < 0 || weights_head_stride < 0) return VTS_ERR_INVALID;
    if (k_out_strides == nullptr || v_out_strides == nullptr || out_pages < 1)
        return VTS_ERR_INVALID;
    if (out_pages > INT32_MAX || keep > INT32_MAX - 1024) return VTS_ERR_UNSUPPORTED;
    // every kept entry has a page to go to
    if (out_page_table_width < 1 || out_page_table_stride < out_page_table_width ||
        out_page_table_width < ((int64_t)keep + cache->page_size - 1) / cache->page_size)
        return VTS_ERR_INVALID;
    st = cache_view(k_out, k_out_strides, out_pages, cache->page_size, cache->kv_heads,
                    cache->head_dim, &p.k_out);
    if (st != VTS_OK) return st;
    st = cache_view(v_out, v_out_strides, out_pages, cache->page_size, cache->kv_heads,
                    cache->head_dim, &p.v_out);
    if (st != VTS_OK) return st;
    if (p.c.batch == 0) return VTS_OK;
    const int64_t rows = (int64_t)p.c.batch * cache->kv_heads;
    // a grid has below 2^32 threads: 1024 to a row, then 256 to 64 kept rows
    if (rows > (1 << 21) || rows * (((int64_t)keep + 63) / 64) > (1 << 23)) return VTS_ERR_UNSUPPORTED;
    if (weights == nullptr || out_page_table == nullptr || kept == nullptr ||
        out_lens == nullptr || out_weights == nullptr || !aligned(weights, 4) ||
        !aligned(kept, 4) || !aligned(out_weights, 4))
        return VTS_ERR_INVALID;
    const size_t n = (size_t)rows * keep * 4;
    if (overlap(kept, n, out_weights, n)) return VTS_ERR_INVALID;
    st = check_device(stream);
    if (st != VTS_OK) return st;
    p.weights = weights;
    p.w_batch = weights_batch_stride;
    p.w_head = weights_head_stride;
    p.width = (int32_t)(width > INT32_MAX ? INT32_MAX : width);
    p.keep = keep;
    p.sinks = sinks;
    p.recent = recent;
    p.out_table = out_page_table;
    p.out_table_stride = out_page_table_stride;
    p.out_pages = (int32_t)out_pages;
    p.row_vecs = cache->head_dim / 8;
    p.kept = kept;
    p.out_lens = out_lens;
    p.out_weights = out_weights;
    return launch_evict(p, static_cast<hipStream_t>(stream)) == hipSuccess ? VTS_OK : VTS_ERR_HIP;
}

size_t vts_verify_draft_workspace_bytes(int64_t batch, int64_t vocab) {
    return verify_layout(batch, vocab).total;
}

int vts_verify_draft(const void* target_probs, int32_t dtype, int64_t target_batch_stride,
                     int64_t target_row_stride, const void* draft_probs,
                     int64_t draft_batch_stride, int64_t draft_row_stride,
                     const int32_t* draft_tokens, const int32_t* parents, const float* uniforms,
                     int64_t batch, int32_t draft, int64_t vocab, int32_t* path, int32_t* count,
                     int32_t* next_token, void* workspace, size_t workspace_bytes, void* stream) {
    if (dtype != VTS_F32 && dtype != VTS_BF16 && dtype != VTS_F16) return VTS_ERR_INVALID;
    if (batch < 0 || draft < 1 || vocab < 1) return VTS_ERR_INVALID;
    if (target_batch_stride < 0 || target_row_stride < 0 || draft_batch_stride < 0 ||
        draft_row_stride < 0)
        return VTS_ERR_INVALID;
    // (a grid has below 2^32 threads; the scans look past the vocabulary's end)
    if (draft > MAX_DRAFT || vocab > INT32_MAX - 65536 || batch > (1 << 21))
        return VTS_ERR_UNSUPPORTED;
    if (batch == 0) return VTS_OK;
    const size_t e = dtype == VTS_F32 ? 4 : 2;
    if (target_probs == nullptr || !aligned(target_probs, e) ||
        (draft_probs && !aligned(draft_probs, e)))
        return VTS_ERR_INVALID;
    if (draft_tokens == nullptr || uniforms == nullptr || path == nullptr || count == nullptr ||
        next_token == nullptr)
        return VTS_ERR_INVALID;
    if (workspace == nullptr || !aligned(workspace, 16) ||
        workspace_bytes < verify_layout(batch, vocab).total)
        return VTS_ERR_WORKSPACE;
    const int st = check_device(stream);
    if (st != VTS_OK) return st;
    VerifyParams p;
    memset(&p, 0, sizeof(p));
    p.target = target_probs;
    p.target_batch = target_batch_stride;
    p.target_row = target_row_stride;
    p.draft_probs = draft_probs;
    p.draft_batch = draft_batch_stride;
    p.draft_row = draft_row_stride;
    p.tokens = draft_tokens;
    p.parents = parents;
    p.uniforms = uniforms;
    p.batch = (int32_t)batch;
    p.draft = draft;
    p.vocab = (int32_t)vocab;
    p.slices = verify_slices(batch, vocab);
    p.path = path;
    p.count = count;
    p.token = next_token;
    char* w = static_cast<char*>(workspace);
    p.tickets = reinterpret_cast<uint32_t*>(w);
    const VerifyLayout layout = verify_layout(batch, vocab);
    p.sums = reinterpret_cast<double*>(w + layout.sums);
    p.states = reinterpret_cast<VerifyState*>(w + layout.states);
    return launch_verify(dtype, p, static_cast<hipStream_t>(stream)) == hipSuccess ? VTS_OK
                                                                                  : VTS_ERR_HIP;
}

}  // extern "C"
