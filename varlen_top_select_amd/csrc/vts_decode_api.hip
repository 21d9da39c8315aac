// vts_decode_api.hip -- C ABI of the decode-step operators (attention over a
// paged cache, accumulated attention weight, eviction, draft verification):
// argument checks on the host before any HIP call, plans that are pure functions
// of the shape, and the launches.
#include <float.h>
#include <math.h>
#include <string.h>

#include "../../include/vts.h"
#include "vts_decode.h"
#include "vts_internal.h"

namespace {

using namespace vts;

// Compute units the plans are made for; a constant, so that the plan and the
// workspace size do not depend on a device query.
constexpr int32_t CUS = 256;
// Kernels look a few units past the end of a list: places stay below 2^31.
constexpr int32_t MARGIN = 1024;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

// A cache's strides in 16-byte vectors, which must reach its last row in 32 bits
// (0 for a dimension of one, whose stride means nothing).
int cache_view(const void* base, const int64_t* strides, int64_t pages, int32_t page_size,
               int32_t kv_heads, int32_t head_dim, CacheView* out) {
    if (base == nullptr || !aligned(base, 16)) return VTS_ERR_INVALID;
    const int64_t sizes[3] = {pages, page_size, kv_heads};
    uint64_t s[3];
    for (int i = 0; i < 3; ++i) {
        s[i] = 0;
        if (sizes[i] == 1) continue;
        if (strides[i] < 0 || strides[i] % 8 != 0) return VTS_ERR_INVALID;
        if (strides[i] / 8 > UINT32_MAX) return VTS_ERR_UNSUPPORTED;
        s[i] = (uint64_t)strides[i] / 8;
    }
    const uint64_t s0 = s[0], s1 = s[1], s2 = s[2];
    // each factor is below 2^32, so no product wraps; the sums stay below 2^66 / 4
    const uint64_t a = (uint64_t)(pages - 1) * s0, b = (uint64_t)(page_size - 1) * s1,
                   c = (uint64_t)(kv_heads - 1) * s2 + (uint64_t)head_dim / 8;
    const uint64_t lim = UINT32_MAX - 1;
    if (a > lim || b > lim || c > lim || a + b + c > lim) return VTS_ERR_UNSUPPORTED;
    out->base = base;
    out->page_stride = (uint32_t)s0;
    out->pos_stride = (uint32_t)s1;
    out->head_stride = (uint32_t)s2;
    return VTS_OK;
}

int paged(const vts_paged_cache* c, int32_t draft, int32_t heads, bool with_v, PagedParams* out) {
    memset(out, 0, sizeof(*out));
    if (c == nullptr) return VTS_ERR_INVALID;
    if (c->dtype != VTS_BF16 && c->dtype != VTS_F16)
        return c->dtype == VTS_F32 ? VTS_ERR_UNSUPPORTED : VTS_ERR_INVALID;
    if (c->batch < 0 || c->kv_heads < 1 || c->page_size < 1 || c->num_pages < 1 ||
        c->page_table_width < 1 || c->page_table_stride < c->page_table_width)
        return VTS_ERR_INVALID;
    if (c->head_dim < 1) return VTS_ERR_INVALID;
    if (c->head_dim != 64 && c->head_dim != 128) return VTS_ERR_UNSUPPORTED;
    if (c->page_size > (1 << 30) || c->num_pages > INT32_MAX ||
        c->num_pages * (int64_t)c->page_size > INT32_MAX || c->kv_heads > MAX_HEADS)
        return VTS_ERR_UNSUPPORTED;
    if (draft < 1) return VTS_ERR_INVALID;
    if (draft > MAX_DRAFT) return VTS_ERR_UNSUPPORTED;
    if (heads < c->kv_heads || heads % c->kv_heads != 0) return VTS_ERR_INVALID;
    if (heads > MAX_HEADS) return VTS_ERR_UNSUPPORTED;
    int st = cache_view(c->k, c->k_strides, c->num_pages, c->page_size, c->kv_heads, c->head_dim,
                        &out->k);
    if (st != VTS_OK) return st;
    if (with_v) {
        st = cache_view(c->v, c->v_strides, c->num_pages, c->page_size, c->kv_heads, c->head_dim,
                        &out->v);
        if (st != VTS_OK) return st;
    } else {
        out->v = out->k;
    }
    if (c->batch > 0 && (c->page_table == nullptr || c->seq_lens == nullptr))
        return VTS_ERR_INVALID;
    out->table = c->page_table;
    out->table_stride = c->page_table_stride;
    out->num_pages = (int32_t)c->num_pages;
    out->page_size = c->page_size;
    out->page_shift = -1;
    if ((c->page_size & (c->page_size - 1)) == 0) out->page_shift = __builtin_ctz(c->page_size);
    const int64_t cap = c->page_table_width > INT32_MAX / c->page_size
                            ? INT32_MAX - MARGIN
                            : c->page_table_width * c->page_size;
    out->capacity = (int32_t)(cap > INT32_MAX - MARGIN ? INT32_MAX - MARGIN : cap);
    out->seq_lens = c->seq_lens;
    out->batch = c->batch;
    out->draft = draft;
    out->heads = heads;
    out->kv_heads = c->kv_heads;
    out->group = heads / c->kv_heads;
    if ((int64_t)c->batch * draft * heads > INT32_MAX) return VTS_ERR_UNSUPPORTED;
    return VTS_OK;
}

int check_q(const void* q, const int64_t* strides, const PagedParams& c) {
    if (q == nullptr || strides == nullptr || !aligned(q, 16)) return VTS_ERR_INVALID;
    const int32_t sizes[3] = {c.batch, c.draft, c.heads};
    for (int i = 0; i < 3; ++i)  // (a dimension of one has no step, and none is taken)
        if (sizes[i] > 1 && (strides[i] < 0 || strides[i] % 8 != 0)) return VTS_ERR_INVALID;
    return VTS_OK;
}

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

struct AttendPlan {
    int32_t rows, block_rows, row_blocks, workers, heads_on_waves;
    size_t part_o, part_ml, total;
};

// Rows go to blocks of 16, 32, 64 or 128, the smallest that holds them (128 from
// 65 on).  One workgroup per compute unit, shared among the blocks of rows: with
// 16 KB on its way per wave it keeps the memory busy, and two of them per unit
// read more places of the cache at once and are slower (64 requests up to
// 16384, 64 heads: 504 us with two, 467 with one, 546 with three).  Slots lie
// apart in any case, and two are faster there (99 us for 104).
int attend_plan(int64_t batch, int32_t draft, int32_t heads, int32_t kv_heads, int32_t head_dim,
                int32_t top_k, AttendPlan* out) {
    const int32_t group = heads / kv_heads;
    out->rows = top_k > 0 ? group : draft * group;
    int32_t block = 16;
    while (block < out->rows && block < 128) block *= 2;
    out->block_rows = block;
    out->row_blocks = (out->rows + block - 1) / block;
    if (out->row_blocks > MAX_TICKETS) return VTS_ERR_UNSUPPORTED;
    out->workers = CUS * (top_k > 0 && block == 16 ? 2 : 1) / out->row_blocks;
    if (out->workers < 8) out->workers = 8;
    if (out->workers > MAX_TICKETS / out->row_blocks) out->workers = MAX_TICKETS / out->row_blocks;
    // A workgroup that reads whole rows of the cache, four heads of them, reads
    // faster than one that reads every kv_heads-th 256 bytes (see vts_attend.hip);
    // more rows a head do not fit, and slots lie apart in either case.
    // The workgroups that share a list leave four times the parts, so not where
    // many share one.  (64 requests, 16 rows to each of 8 heads: 349 us for 369 at
    // lengths of 8192, 187 for 192 at 4096; the rule knows no lengths, and below it
    // costs, 107 us for 104 at 2048 and 68 for 52 at 1024.)
    out->heads_on_waves =
        top_k == 0 && block <= 32 && kv_heads % 4 == 0 && batch * kv_heads >= 128;
    const size_t parts =
        2 * (size_t)out->workers * out->row_blocks * block * (out->heads_on_waves ? 4 : 1);
    out->part_o = TICKET_BYTES;
    out->part_ml = out->part_o + align256(parts * head_dim * 4);
    out->total = out->part_ml + align256(parts * 2 * 4);
    return VTS_OK;
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
    if (attend_plan(batch, draft, heads, kv_heads, head_dim, top_k, &plan) != VTS_OK) return 0;
    return plan.total;
}

int vts_tree_attention(const vts_paged_cache* cache, const void* q, const int64_t* q_strides,
                       int32_t draft, int32_t heads, const int64_t* tree_mask,
                       const int32_t* slots, int32_t top_k, float scale, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
    AttendParams p;
    memset(&p, 0, sizeof(p));
    int st = paged(cache, draft, heads, true, &p.c);
    if (st != VTS_OK) return st;
    // (an empty batch's slots may have no address)
    if (slots != nullptr ? top_k < 1 : top_k < 0 || (top_k > 0 && p.c.batch > 0))
        return VTS_ERR_INVALID;
    if (top_k > INT32_MAX - MARGIN) return VTS_ERR_UNSUPPORTED;
    if (isnan(scale)) return VTS_ERR_INVALID;
    if (p.c.batch == 0) return VTS_OK;
    st = check_q(q, q_strides, p.c);
    if (st != VTS_OK) return st;
    const size_t rows = (size_t)p.c.batch * draft * heads;
    const size_t out_bytes = rows * cache->head_dim * 2;
    if (out == nullptr || !aligned(out, 16)) return VTS_ERR_INVALID;
    if (lse && (!aligned(lse, 4) || overlap(out, out_bytes, lse, rows * 4))) return VTS_ERR_INVALID;
    AttendPlan plan;
    st = attend_plan(cache->batch, draft, heads, cache->kv_heads, cache->head_dim, top_k, &plan);
    if (st != VTS_OK) return st;
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < plan.total)
        return VTS_ERR_WORKSPACE;
    st = check_device(stream);
    if (st != VTS_OK) return st;
    p.q = q;
    p.q_batch = q_strides[0];
    p.q_row = q_strides[1];
    p.q_head = q_strides[2];
    p.tree_mask = tree_mask;
    p.slots = slots;
    p.top_k = top_k;
    p.scale_log2e = (float)(fabs((double)scale) * 1.4426950408889634);
    if (p.scale_log2e < FLT_MIN) p.scale_log2e = FLT_MIN;  // (0 * -inf is no -inf)
    p.q_sign = scale < 0 ? 0x80008000u : 0;
    p.out = out;
    p.lse = lse;
    p.rows = plan.rows;
    p.block_rows = plan.block_rows;
    p.row_blocks = plan.row_blocks;
    p.workers = plan.workers;
    p.heads_on_waves = plan.heads_on_waves;
    char* w = static_cast<char*>(workspace);
    p.tickets = reinterpret_cast<uint32_t*>(w);
    p.part_o = reinterpret_cast<float*>(w + plan.part_o);
    p.part_ml = reinterpret_cast<float*>(w + plan.part_ml);
    return launch_attend(cache->dtype, cache->head_dim, p,
                         static_cast<hipStream_t>(stream)) == hipSuccess
               ? VTS_OK
               : VTS_ERR_HIP;
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
