// vts_decode.h -- parameter blocks and launch entry points shared by the
// decode-step kernels (vts_attend.hip, vts_weigh.hip, vts_evict.hip,
// vts_verify.hip) and their C ABI (vts_decode_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace vts {

// Drafted tokens of a request, at most: the bits of one tree_mask word.
constexpr int MAX_DRAFT = 64;
constexpr int MAX_HEADS = 8192;
// Workgroups that may hold a ticket: two words each are the fixed first part of
// every decode workspace, so that calls of different shapes can share one.
constexpr int MAX_TICKETS = 8192;
constexpr size_t TICKET_BYTES = (size_t)MAX_TICKETS * 2 * 4;

// One of the two caches: rows of head_dim elements, found by page, position in
// the page and KV head.  Strides are in 16-byte vectors.
struct CacheView {
    const void* base;
    uint32_t page_stride, pos_stride, head_stride;
};

struct PagedParams {
    CacheView k, v;
    const int32_t* table;
    int64_t table_stride;
    int32_t num_pages, page_size;
    int32_t page_shift;  // log2(page_size), or -1
    int32_t capacity;    // positions that a page-table row can name
    const int32_t* seq_lens;
    int32_t batch, draft, heads, kv_heads, group;  // group: query heads per KV head
};

struct AttendParams {
    PagedParams c;
    const void* q;
    int64_t q_batch, q_row, q_head;  // strides, elements
    const int64_t* tree_mask;        // [batch, draft] or null (chain)
    const int32_t* slots;            // [batch * draft, top_k] or null
    int32_t top_k;
    float scale_log2e;  // > 0: a negative scale's sign goes to q, and 0 is the least normal
    uint32_t q_sign;    // 0x80008000 for a negative scale
    void* out;
    float* lse;  // or null
    // plan
    int32_t rows;      // query rows that share one list of positions: draft * group, or group
    int32_t block_rows;  // 16, 32, 64 or 128 rows to a workgroup (times four heads)
    int32_t row_blocks;
    int32_t workers;   // workgroups per row block
    // 1: a workgroup's waves take a KV head each and walk the same places, so that
    // it reads whole rows of the cache; 0: they take 32 places each of one head
    int32_t heads_on_waves;
    uint32_t* tickets;
    // two parts per workgroup, of block_rows rows (times four heads): outputs
    // [..][D], maximum and sum [..][2]
    float* part_o;
    float* part_ml;
};

struct WeighParams {
    PagedParams c;
    const void* q;
    int64_t q_batch, q_row, q_head;
    const int64_t* tree_mask;
    const float* lse;         // [batch, draft, heads]
    const uint8_t* row_keep;  // [batch, draft] or null
    float scale_log2e;
    float* weights;  // [batch, kv_heads, width]
    int64_t w_batch, w_head;
    int32_t width;
    int32_t rows;
    int32_t workers;
    int32_t heads_on_waves;  // as in AttendParams
};

struct EvictParams {
    PagedParams c;
    const float* weights;
    int64_t w_batch, w_head;
    int32_t width;
    int32_t keep, sinks, recent;
    CacheView k_out, v_out;
    const int32_t* out_table;
    int64_t out_table_stride;
    int32_t out_pages;
    int32_t row_vecs;  // 16-byte vectors per cache row
    int32_t* kept;
    int32_t* out_lens;
    float* out_weights;
};

// A request's walk between two launches.
struct VerifyState {
    int32_t cur, next, steps;
    int32_t more;  // 0: ended
    int32_t sums;  // which half of VerifyParams::sums holds the residual's
    int32_t pad;
    double a, mass;
    int32_t path[MAX_DRAFT];
};

struct VerifyParams {
    const void* target;
    int64_t target_batch, target_row;
    const void* draft_probs;  // or null: the drafted tokens were chosen
    int64_t draft_batch, draft_row;
    const int32_t* tokens;    // [batch, draft]
    const int32_t* parents;   // [batch, draft] or null (chain)
    const float* uniforms;    // [batch, draft + 1]
    int32_t batch, draft, vocab;
    int32_t slices;  // workgroups per request
    int32_t* path;   // [batch, draft]
    int32_t* count;  // [batch]
    int32_t* token;  // [batch]
    uint32_t* tickets;
    double* sums;    // [2][batch][16 * slices]
    VerifyState* states;  // [batch][2]
};

hipError_t launch_attend(int dtype, int head_dim, const AttendParams& p, hipStream_t stream);
hipError_t launch_weigh(int dtype, int head_dim, const WeighParams& p, hipStream_t stream);
hipError_t launch_evict(const EvictParams& p, hipStream_t stream);
hipError_t launch_verify(int dtype, const VerifyParams& p, hipStream_t stream);

}  // namespace vts
