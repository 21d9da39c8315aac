// vts_decode_checks.h -- host side of the decode-step operators that more than one
// C ABI file needs: checks of caches and queries, and the attention's plan and call.
#pragma once

#include <float.h>
#include <math.h>
#include <string.h>

#include "../../include/vts.h"
#include "vts_decode.h"
#include "vts_internal.h"

namespace vts {

// Compute units the plans are made for; a constant, so that the plan and the
// workspace size do not depend on a device query.
constexpr int32_t CUS = 256;
// Kernels look a few units past the end of a list: places stay below 2^31.
constexpr int32_t MARGIN = 1024;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

// The strides of pages, positions and heads in units of `unit`, which must reach the
// end of the last row, `row` units long, in 32 bits (0 for a dimension of one, whose
// stride means nothing).
inline int unit_strides(const int64_t* strides, int64_t pages, int32_t page_size, int32_t kv_heads,
                        int32_t unit, int32_t row, uint32_t* out) {
    const int64_t sizes[3] = {pages, page_size, kv_heads};
    uint64_t s[3];
    for (int i = 0; i < 3; ++i) {
        s[i] = 0;
        if (sizes[i] == 1) continue;
        if (strides[i] < 0 || strides[i] % unit != 0) return VTS_ERR_INVALID;
        if (strides[i] / unit > UINT32_MAX) return VTS_ERR_UNSUPPORTED;
        s[i] = (uint64_t)strides[i] / unit;
    }
    // each factor is below 2^32, so no product wraps; the sums stay below 2^66 / 4
    const uint64_t a = (uint64_t)(pages - 1) * s[0], b = (uint64_t)(page_size - 1) * s[1],
                   c = (uint64_t)(kv_heads - 1) * s[2] + (uint64_t)row;
    const uint64_t lim = UINT32_MAX - 1;
    if (a > lim || b > lim || c > lim || a + b + c > lim) return VTS_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i) out[i] = (uint32_t)s[i];
    return VTS_OK;
}

// A cache of `bits` to an element: strides in elements of a 16-bit cache, in bytes of
// a microscaled one.
inline int cache_view(const void* base, const int64_t* strides, int64_t pages, int32_t page_size,
                      int32_t kv_heads, int32_t head_dim, CacheView* out, int32_t bits = 16) {
    if (base == nullptr || !aligned(base, 16)) return VTS_ERR_INVALID;
    uint32_t s[3];
    const int st = unit_strides(strides, pages, page_size, kv_heads, bits == 16 ? 8 : 16,
                                head_dim * bits / 128, s);
    if (st != VTS_OK) return st;
    *out = {base, s[0], s[1], s[2]};
    return VTS_OK;
}

inline int scale_view(const uint8_t* base, const int64_t* strides, int64_t pages, int32_t page_size,
                      int32_t kv_heads, int32_t head_dim, ScaleView* out) {
    const int32_t row = head_dim / 32;
    if (base == nullptr || !aligned(base, row)) return VTS_ERR_INVALID;
    uint32_t s[3];
    const int st = unit_strides(strides, pages, page_size, kv_heads, row, 1, s);
    if (st != VTS_OK) return st;
    *out = {base, s[0], s[1], s[2]};
    return VTS_OK;
}

inline int check_bits(const vts_microscales* m) {
    return m == nullptr || (m->bits != 4 && m->bits != 8) ? VTS_ERR_INVALID : VTS_OK;
}

// The caches of `c` (microscaled if `m` is given), without their page table.
inline int cache_rows(const vts_paged_cache* c, const vts_microscales* m, bool with_v, CacheView* k,
                      CacheView* v, ScaleView* ks, ScaleView* vs) {
    if (c == nullptr) return VTS_ERR_INVALID;
    if (c->dtype != VTS_BF16 && c->dtype != VTS_F16)
        return c->dtype == VTS_F32 ? VTS_ERR_UNSUPPORTED : VTS_ERR_INVALID;
    if (c->kv_heads < 1 || c->page_size < 1 || c->num_pages < 1 || c->head_dim < 1)
        return VTS_ERR_INVALID;
    if (c->head_dim != 64 && c->head_dim != 128) return VTS_ERR_UNSUPPORTED;
    if (c->page_size > (1 << 30) || c->num_pages > INT32_MAX ||
        c->num_pages * (int64_t)c->page_size > INT32_MAX || c->kv_heads > MAX_HEADS)
        return VTS_ERR_UNSUPPORTED;
    if (m != nullptr && check_bits(m) != VTS_OK) return VTS_ERR_INVALID;
    const int32_t bits = m ? m->bits : 16;
    int st = cache_view(c->k, c->k_strides, c->num_pages, c->page_size, c->kv_heads, c->head_dim, k, bits);
    if (st != VTS_OK) return st;
    if (!with_v) {
        *v = *k;
    } else {
        st = cache_view(c->v, c->v_strides, c->num_pages, c->page_size, c->kv_heads, c->head_dim, v, bits);
        if (st != VTS_OK) return st;
    }
    if (m == nullptr) return VTS_OK;
    st = scale_view(m->k, m->k_strides, c->num_pages, c->page_size, c->kv_heads, c->head_dim, ks);
    if (st != VTS_OK) return st;
    return scale_view(m->v, m->v_strides, c->num_pages, c->page_size, c->kv_heads, c->head_dim, vs);
}

inline int32_t log2_of(int32_t n) { return (n & (n - 1)) == 0 ? __builtin_ctz(n) : -1; }

inline int paged(const vts_paged_cache* c, int32_t draft, int32_t heads, bool with_v, PagedParams* out,
                 const vts_microscales* m = nullptr, ScaleView* ks = nullptr, ScaleView* vs = nullptr) {
    memset(out, 0, sizeof(*out));
    if (c == nullptr) return VTS_ERR_INVALID;
    if (c->batch < 0 || c->page_table_width < 1 || c->page_table_stride < c->page_table_width)
        return VTS_ERR_INVALID;
    if (draft < 1) return VTS_ERR_INVALID;
    int st = cache_rows(c, m, with_v, &out->k, &out->v, ks, vs);
    if (st != VTS_OK) return st;
    if (draft > MAX_DRAFT) return VTS_ERR_UNSUPPORTED;
    if (heads < c->kv_heads || heads % c->kv_heads != 0) return VTS_ERR_INVALID;
    if (heads > MAX_HEADS) return VTS_ERR_UNSUPPORTED;
    if (c->batch > 0 && (c->page_table == nullptr || c->seq_lens == nullptr))
        return VTS_ERR_INVALID;
    out->table = c->page_table;
    out->table_stride = c->page_table_stride;
    out->num_pages = (int32_t)c->num_pages;
    out->page_size = c->page_size;
    out->page_shift = log2_of(c->page_size);
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

inline int check_q(const void* q, const int64_t* strides, const PagedParams& c) {
    if (q == nullptr || strides == nullptr || !aligned(q, 16)) return VTS_ERR_INVALID;
    const int32_t sizes[3] = {c.batch, c.draft, c.heads};
    for (int i = 0; i < 3; ++i)  // (a dimension of one has no step, and none is taken)
        if (sizes[i] > 1 && (strides[i] < 0 || strides[i] % 8 != 0)) return VTS_ERR_INVALID;
    return VTS_OK;
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
// apart in any case, and two are faster there (99 us for 104).  Of a microscaled cache
// two keep as much on its way as one of a 16-bit cache (64 requests up to 16384, 64
// heads, 4 bits: 194 us with two, 219 with one; 8 bits 259 and 252).
inline int attend_plan(int64_t batch, int32_t draft, int32_t heads, int32_t kv_heads, int32_t head_dim,
                int32_t top_k, int32_t bits, AttendPlan* out) {
    const int32_t group = heads / kv_heads;
    out->rows = top_k > 0 ? group : draft * group;
    int32_t block = 16;
    while (block < out->rows && block < 128) block *= 2;
    out->block_rows = block;
    out->row_blocks = (out->rows + block - 1) / block;
    if (out->row_blocks > MAX_TICKETS) return VTS_ERR_UNSUPPORTED;
    const bool two = bits != 16 || (top_k > 0 && block == 16);
    out->workers = CUS * (two ? 2 : 1) / out->row_blocks;
    if (out->workers < 8) out->workers = 8;
    if (out->workers > MAX_TICKETS / out->row_blocks) out->workers = MAX_TICKETS / out->row_blocks;
    // A workgroup that reads whole rows of the cache, four heads of them, reads
    // faster than one that reads every kv_heads-th 256 bytes (see vts_attend.hip);
    // more rows a head do not fit, and slots of a 16-bit cache lie apart in either case.
    // (Those of four heads' microscaled rows, 128 lists of 2048: 52 us for 87 with 4 bits,
    // 78 for 87 with 8.)
    // The workgroups that share a list leave four times the parts, so not where
    // many share one.  (64 requests, 16 rows to each of 8 heads: 349 us for 369 at
    // lengths of 8192, 187 for 192 at 4096; the rule knows no lengths, and below it
    // costs, 107 us for 104 at 2048 and 68 for 52 at 1024.)
    out->heads_on_waves =
        (top_k == 0 || bits != 16) && block <= 32 && kv_heads % 4 == 0 &&
        batch * kv_heads * (top_k > 0 ? draft : 1) >= 128;
    const size_t parts =
        2 * (size_t)out->workers * out->row_blocks * block * (out->heads_on_waves ? 4 : 1);
    out->part_o = TICKET_BYTES;
    out->part_ml = out->part_o + align256(parts * head_dim * 4);
    out->total = out->part_ml + align256(parts * 2 * 4);
    return VTS_OK;
}

// The attention of vts_tree_attention, and over a microscaled cache.  `launch` starts the
// kernels with the parameters it is given.
template <class Launch>
inline int attend(const vts_paged_cache* cache, const vts_microscales* scales, const void* q, const int64_t* q_strides,
                  int32_t draft, int32_t heads, const int64_t* tree_mask, const int32_t* slots, int32_t top_k,
                  float scale, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream,
                  Launch launch) {
    AttendParams p;
    memset(&p, 0, sizeof(p));
    int st = paged(cache, draft, heads, true, &p.c, scales, &p.k_scale, &p.v_scale);
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
    st = attend_plan(cache->batch, draft, heads, cache->kv_heads, cache->head_dim, top_k,
                     scales ? scales->bits : 16, &plan);
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
    return launch(p) == hipSuccess ? VTS_OK : VTS_ERR_HIP;
}

}  // namespace vts
