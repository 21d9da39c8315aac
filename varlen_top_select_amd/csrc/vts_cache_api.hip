// vts_cache_api.hip -- C ABI of the calls that fill and read a paged cache and attend a
// prompt (write_cache, read_cache, prompt_attention), and of the decode step's
// attention over a microscaled cache: argument checks on the host before any HIP call,
// plans that are pure functions of the shape, and the launches.
#include "vts_cache.h"
#include "vts_decode_checks.h"

namespace {

using namespace vts;

// Waves that fill the device once over (three or four to each of 1024 SIMDs): fewer
// tokens are shared among several waves each.
constexpr int64_t FULL = 4096;

int slot_cache(const vts_paged_cache* c, const vts_microscales* m, SlotCache* out) {
    const int st = cache_rows(c, m, true, &out->k, &out->v, &out->k_scale, &out->v_scale);
    if (st != VTS_OK) return st;
    out->num_slots = (int32_t)(c->num_pages * c->page_size);
    out->page_size = c->page_size;
    out->page_shift = log2_of(c->page_size);
    out->kv_heads = c->kv_heads;
    return VTS_OK;
}

// Rows [n, heads] of 16-bit elements at the strides given.
int check_rows(const void* p, const int64_t* strides, int64_t n, int64_t heads) {
    if (p == nullptr || !aligned(p, 16)) return VTS_ERR_INVALID;
    const int64_t sizes[2] = {n, heads};
    for (int i = 0; i < 2; ++i)  // (a dimension of one has no step, and none is taken)
        if (sizes[i] > 1 && (strides[i] < 0 || strides[i] % 8 != 0)) return VTS_ERR_INVALID;
    return VTS_OK;
}

struct PromptPlan {
    int64_t tiles;
    int32_t splits;
    size_t part_ml, total;
};

// Two workgroups to a compute unit fill the device: where there are half as many tiles or fewer,
// and on average 1024 keys or more to a sequence, a tile's keys are shared, 512 or more to each
// (one request's 16 queries of 32 heads behind 16400 keys: 60 us for 292; four of them behind
// 2060 to 4100: 32 for 78; two of 128 behind 4100 and 8200: 53 for 152).
PromptPlan prompt_plan(int64_t batch, int64_t total_q, int64_t total_k, int32_t heads, int32_t kv_heads,
                       int32_t head_dim) {
    PromptPlan plan;
    plan.tiles = total_q * (heads / kv_heads) / PROMPT_ROWS + (batch < total_q ? batch : total_q);
    const int64_t keys = batch > 0 ? total_k / batch : 0, work = plan.tiles * kv_heads;
    int64_t n = work > 0 && keys >= 1024 ? 512 / work : 1;
    if (n > keys / 512) n = keys / 512;
    if (n > 32) n = 32;
    plan.splits = n < 2 ? 1 : (int32_t)n;
    const size_t rows = plan.splits > 1 ? (size_t)work * plan.splits * PROMPT_ROWS : 0;
    plan.part_ml = align256(rows * head_dim * 4);
    plan.total = plan.part_ml + align256(rows * 2 * 4);
    return plan;
}

int status(hipError_t e) { return e == hipSuccess ? VTS_OK : VTS_ERR_HIP; }

}  // namespace

extern "C" {

size_t vts_tree_attention_microscaled_workspace_bytes(int32_t batch, int32_t draft, int32_t heads,
                                                      int32_t kv_heads, int32_t head_dim, int32_t top_k) {
    AttendPlan plan;
    if (batch < 0 || draft < 1 || draft > MAX_DRAFT || kv_heads < 1 || heads < kv_heads ||
        heads % kv_heads != 0 || heads > MAX_HEADS || head_dim < 1 || head_dim > 1024)
        return 0;
    if (attend_plan(batch, draft, heads, kv_heads, head_dim, top_k, 4, &plan) != VTS_OK) return 0;
    return plan.total;
}

int vts_tree_attention_microscaled(const vts_paged_cache* cache, const vts_microscales* scales, const void* q,
                                   const int64_t* q_strides, int32_t draft, int32_t heads,
                                   const int64_t* tree_mask, const int32_t* slots, int32_t top_k, float scale,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    if (scales == nullptr) return VTS_ERR_INVALID;
    return attend(cache, scales, q, q_strides, draft, heads, tree_mask, slots, top_k, scale, out, lse,
                  workspace, workspace_bytes, stream, [&](const AttendParams& p) {
                      const hipStream_t s = static_cast<hipStream_t>(stream);
                      return cache->dtype == VTS_BF16
                                 ? launch_attend_micro_bf16(cache->head_dim, scales->bits, p, s)
                                 : launch_attend_micro_f16(cache->head_dim, scales->bits, p, s);
                  });
}

int vts_write_cache(const vts_paged_cache* cache, const vts_microscales* scales, const vts_new_tokens* t,
                    void* stream) {
    WriteParams p;
    memset(&p, 0, sizeof(p));
    int st = slot_cache(cache, scales, &p.c);
    if (st != VTS_OK) return st;
    if (t == nullptr || t->tokens < 0 || t->heads < 1) return VTS_ERR_INVALID;
    if (!(t->eps >= 0) || isinf(t->eps)) return VTS_ERR_INVALID;
    if (t->heads > MAX_HEADS || t->tokens > (1 << 25)) return VTS_ERR_UNSUPPORTED;
    if (t->rotary != nullptr) {
        if (t->rot < 16 || t->rot % 16 != 0 || t->rot > cache->head_dim || t->max_position < 1 ||
            !aligned(t->rotary, 16))
            return VTS_ERR_INVALID;
        if (t->max_position > INT32_MAX) return VTS_ERR_UNSUPPORTED;
    } else if (t->rot != 0) {
        return VTS_ERR_INVALID;
    }
    if ((t->q_norm || t->k_norm) && t->norm_dtype != VTS_F32 && t->norm_dtype != cache->dtype)
        return VTS_ERR_INVALID;
    if ((t->q_norm && !aligned(t->q_norm, 16)) || (t->k_norm && !aligned(t->k_norm, 16)))
        return VTS_ERR_INVALID;
    if (t->tokens == 0) return VTS_OK;
    st = check_rows(t->q, t->q_strides, t->tokens, t->heads);
    if (st == VTS_OK) st = check_rows(t->k, t->k_strides, t->tokens, cache->kv_heads);
    if (st == VTS_OK) st = check_rows(t->v, t->v_strides, t->tokens, cache->kv_heads);
    if (st != VTS_OK) return st;
    if (t->slots == nullptr || (t->rotary && t->positions == nullptr)) return VTS_ERR_INVALID;
    if (t->q_out == nullptr || !aligned(t->q_out, 16) || !aligned(t->k_out, 16)) return VTS_ERR_INVALID;
    const size_t row = (size_t)cache->head_dim * 2;
    if (t->k_out && overlap(t->q_out, row * t->tokens * t->heads, t->k_out, row * t->tokens * cache->kv_heads))
        return VTS_ERR_INVALID;
    st = check_device(stream);
    if (st != VTS_OK) return st;
    p.q = t->q;
    p.k = t->k;
    p.v = t->v;
    p.q_token = t->q_strides[0];
    p.q_head = t->q_strides[1];
    p.k_token = t->k_strides[0];
    p.k_head = t->k_strides[1];
    p.v_token = t->v_strides[0];
    p.v_head = t->v_strides[1];
    p.q_norm = t->q_norm;
    p.k_norm = t->k_norm;
    p.norm_f32 = t->norm_dtype == VTS_F32;
    p.eps = t->eps;
    p.rotary = t->rotary;
    p.max_position = (int32_t)t->max_position;
    p.rot = t->rot;
    p.interleaved = t->interleaved != 0;
    p.positions = t->positions;
    p.slots = t->slots;
    p.tokens = (int32_t)t->tokens;
    p.heads = t->heads;
    p.q_out = t->q_out;
    p.k_out = t->k_out;
    const int32_t per = 512 / cache->head_dim;  // rows of a wave at a time
    const int32_t steps = (t->heads + per - 1) / per + 2 * ((cache->kv_heads + per - 1) / per);
    int64_t parts = FULL / t->tokens;
    if (parts > steps) parts = steps;
    p.parts = parts < 1 ? 1 : (int32_t)parts;
    return status(launch_write(cache->dtype, cache->head_dim, scales ? scales->bits : 16, p,
                               static_cast<hipStream_t>(stream)));
}

int vts_read_cache(const vts_paged_cache* cache, const vts_microscales* scales, const int32_t* slots,
                   int64_t count, void* k_out, void* v_out, void* stream) {
    ReadParams p;
    memset(&p, 0, sizeof(p));
    int st = slot_cache(cache, scales, &p.c);
    if (st != VTS_OK) return st;
    if (count < 0) return VTS_ERR_INVALID;
    p.per_slot = cache->kv_heads * (cache->head_dim / 8);
    // a grid has below 2^32 threads, of four chunks each
    if (count > (1ll << 33) / p.per_slot) return VTS_ERR_UNSUPPORTED;
    if (count == 0) return VTS_OK;
    const size_t bytes = (size_t)count * p.per_slot * 16;
    if (slots == nullptr || k_out == nullptr || v_out == nullptr || !aligned(k_out, 16) ||
        !aligned(v_out, 16) || overlap(k_out, bytes, v_out, bytes))
        return VTS_ERR_INVALID;
    st = check_device(stream);
    if (st != VTS_OK) return st;
    p.slots = slots;
    p.chunks = count * p.per_slot;
    p.k_out = k_out;
    p.v_out = v_out;
    return status(launch_read(cache->dtype, cache->head_dim, scales ? scales->bits : 16, p,
                              static_cast<hipStream_t>(stream)));
}

size_t vts_prompt_attention_workspace_bytes(int64_t batch, int64_t total_q, int64_t total_k, int32_t heads,
                                            int32_t kv_heads, int32_t head_dim) {
    if (batch < 0 || total_q < 0 || total_k < 0 || kv_heads < 1 || heads < kv_heads || heads > MAX_HEADS ||
        heads % kv_heads != 0 || head_dim < 1 || head_dim > 1024 || batch > INT32_MAX || total_k > INT32_MAX ||
        total_q > INT32_MAX / heads)
        return 0;
    return prompt_plan(batch, total_q, total_k, heads, kv_heads, head_dim).total;
}

int vts_prompt_attention(const vts_prompts* a, int32_t causal, float scale, void* out, float* lse,
                         int32_t clear, void* workspace, size_t workspace_bytes, void* stream) {
    PromptParams p;
    memset(&p, 0, sizeof(p));
    if (a == nullptr || isnan(scale)) return VTS_ERR_INVALID;
    if (a->dtype != VTS_BF16 && a->dtype != VTS_F16)
        return a->dtype == VTS_F32 ? VTS_ERR_UNSUPPORTED : VTS_ERR_INVALID;
    if (a->head_dim < 1 || a->batch < 0 || a->total_q < 0 || a->total_k < 0) return VTS_ERR_INVALID;
    if (a->head_dim != 64 && a->head_dim != 128) return VTS_ERR_UNSUPPORTED;
    if (a->kv_heads < 1 || a->heads < a->kv_heads || a->heads % a->kv_heads != 0) return VTS_ERR_INVALID;
    if (a->heads > MAX_HEADS) return VTS_ERR_UNSUPPORTED;
    // (positions are 32-bit numbers, with a tile to spare)
    if (a->total_q > (INT32_MAX - MARGIN) / a->heads || a->total_k > INT32_MAX - MARGIN ||
        a->batch > INT32_MAX - MARGIN)
        return VTS_ERR_UNSUPPORTED;
    if (a->total_q == 0) return VTS_OK;
    int st = check_rows(a->q, a->q_strides, a->total_q, a->heads);
    if (st == VTS_OK && a->total_k > 0) st = check_rows(a->k, a->k_strides, a->total_k, a->kv_heads);
    if (st == VTS_OK && a->total_k > 0) st = check_rows(a->v, a->v_strides, a->total_k, a->kv_heads);
    if (st != VTS_OK) return st;
    if (a->batch > 0 && (a->cu_q == nullptr || a->cu_k == nullptr)) return VTS_ERR_INVALID;
    const size_t rows = (size_t)a->total_q * a->heads;
    if (out == nullptr || !aligned(out, 16)) return VTS_ERR_INVALID;
    if (lse && (!aligned(lse, 4) || overlap(out, rows * a->head_dim * 2, lse, rows * 4))) return VTS_ERR_INVALID;
    p.group = a->heads / a->kv_heads;
    const PromptPlan plan = prompt_plan(a->batch, a->total_q, a->total_k, a->heads, a->kv_heads, a->head_dim);
    // (a grid has below 2^32 threads, and with `clear` 64 workgroups more)
    if (plan.tiles * a->kv_heads >= (1 << 24) - 64) return VTS_ERR_UNSUPPORTED;
    if (plan.total > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < plan.total))
        return VTS_ERR_WORKSPACE;
    if (a->batch == 0 && !clear) return VTS_OK;  // (a grid may not be empty)
    st = check_device(stream);
    if (st != VTS_OK) return st;
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.q_token = a->q_strides[0];
    p.q_head = a->q_strides[1];
    p.k_token = a->k_strides[0];
    p.k_head = a->k_strides[1];
    p.v_token = a->v_strides[0];
    p.v_head = a->v_strides[1];
    p.cu_q = a->cu_q;
    p.cu_k = a->cu_k;
    p.batch = (int32_t)a->batch;
    p.total_q = (int32_t)a->total_q;
    p.total_k = (int32_t)a->total_k;
    p.heads = a->heads;
    p.kv_heads = a->kv_heads;
    p.causal = causal != 0;
    p.scale_log2e = (float)(fabs((double)scale) * 1.4426950408889634);
    if (p.scale_log2e < FLT_MIN) p.scale_log2e = FLT_MIN;  // (0 * -inf is no -inf)
    p.q_sign = scale < 0 ? 0x80008000u : 0;
    p.out = out;
    p.lse = lse;
    p.clear = clear != 0;
    p.tiles = (int32_t)plan.tiles;
    p.splits = plan.splits;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + (plan.total > 0 ? plan.part_ml : 0));
    // The last workgroups to start are then those of the shortest sequences (8 times 512
    // queries of 64 heads behind up to 16384 keys: 1624 us for 1661; 16 times up to 256 of 32
    // heads 641 for 681; 32 times 128, head size 64, 543 for 576); finding the order takes a
    // workgroup half a microsecond, and is left where its work is a few.
    p.longest_first = a->batch > 1 && a->batch <= 64 && a->total_k / a->batch >= 4096;
    p.direct = a->k_strides[0] < (1 << 24) && a->v_strides[0] < (1 << 24);
    return status(launch_prompt(a->dtype, a->head_dim, p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
