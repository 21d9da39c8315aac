// vts_cache.h -- parameter blocks and launch entry points shared by the kernels that
// fill and read back a paged cache (vts_cache.hip), a prompt's attention
// (vts_prompt.hip), and their C ABI (vts_cache_api.hip).
#pragma once

#include "vts_decode.h"

namespace vts {

// Both caches, by slot (page * page_size + position in the page).
struct SlotCache {
    CacheView k, v;
    ScaleView k_scale, v_scale;
    int32_t num_slots, page_size, page_shift, kv_heads;
};

struct WriteParams {
    SlotCache c;
    const void *q, *k, *v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;  // strides, elements
    const void *q_norm, *k_norm;  // [head_dim] or null
    int32_t norm_f32;             // whether they are 32-bit
    double eps;
    const float* rotary;  // [max_position, rot]: cosines, then sines; or null
    int32_t max_position, rot, interleaved;
    const int32_t* positions;  // [tokens]
    const int32_t* slots;      // [tokens]
    int32_t tokens, heads;
    void* q_out;  // [tokens, heads, head_dim]
    void* k_out;  // [tokens, kv_heads, head_dim] or null
    int32_t parts;  // waves per token
};

struct ReadParams {
    SlotCache c;
    const int32_t* slots;
    int64_t chunks;    // of eight elements, in each of the outputs
    int32_t per_slot;  // such chunks of one slot
    void *k_out, *v_out;
};

constexpr int PROMPT_ROWS = 128;  // rows of a workgroup: tokens times heads of a KV head

struct PromptParams {
    const void *q, *k, *v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;  // strides, elements
    const int32_t *cu_q, *cu_k;  // [batch + 1]
    int32_t batch, total_q, total_k, heads, kv_heads, group;
    int32_t causal;
    float scale_log2e;  // as in AttendParams
    uint32_t q_sign;
    void* out;
    float* lse;  // or null
    int32_t clear;  // 1: rows of no sequence get zeros and -inf
    int32_t tiles;   // of 128 rows, per KV head, at most
    int32_t splits;  // workgroups that share a tile's keys
    // their parts: [tiles][kv_heads][splits][128] rows of head_dim outputs, and of maximum and sum
    float *part_o, *part_ml;
    int32_t longest_first;  // 1: at most 64 sequences, the longest first
    int32_t direct;  // 1: 32 rows of K and of V span less than 2^31 bytes
};

hipError_t launch_write(int dtype, int head_dim, int bits, const WriteParams& p, hipStream_t stream);
hipError_t launch_read(int dtype, int head_dim, int bits, const ReadParams& p, hipStream_t stream);
hipError_t launch_prompt(int dtype, int head_dim, const PromptParams& p, hipStream_t stream);

}  // namespace vts
