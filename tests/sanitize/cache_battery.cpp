// Exercise of the host side of vts_write_cache, vts_read_cache, vts_prompt_attention and
// vts_tree_attention_microscaled (argument checks, plans) under AddressSanitizer and
// UndefinedBehaviorSanitizer.  Every call uses fake device pointers; the launches below
// stand in for the kernels and check that the plans they get hold together.  Exits
// non-zero on an unexpected status.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/vts.h"
#include "../../varlen_top_select_amd/csrc/vts_cache.h"

static int bad = 0, launched = 0;
static void expect(const char* what, long long got, long long want) {
    if (got != want) {
        fprintf(stderr, "%s: %lld, expected %lld\n", what, got, want);
        ++bad;
    }
}

namespace vts {
int check_device(void*, int*, int*) { return VTS_OK; }
static hipError_t attend_seen(int bits, const AttendParams& p) {
    ++launched;
    expect("bits", bits == 4 || bits == 8, 1);
    expect("rows fit their blocks", (int64_t)p.block_rows * p.row_blocks >= p.rows, 1);
    expect("tickets", (int64_t)p.workers * p.row_blocks <= MAX_TICKETS && p.workers > 0, 1);
    expect("scales", p.k_scale.base != nullptr && p.v_scale.base != nullptr, 1);
    return hipSuccess;
}
hipError_t launch_attend_micro_bf16(int, int bits, const AttendParams& p, hipStream_t) { return attend_seen(bits, p); }
hipError_t launch_attend_micro_f16(int, int bits, const AttendParams& p, hipStream_t) { return attend_seen(bits, p); }
hipError_t launch_write(int, int head_dim, int, const WriteParams& p, hipStream_t) {
    ++launched;
    const int per = 512 / head_dim;
    const int64_t steps = (p.heads + per - 1) / per + 2 * ((p.c.kv_heads + per - 1) / per);
    expect("parts", p.parts >= 1 && p.parts <= steps, 1);
    expect("a grid", (int64_t)p.tokens * p.parts <= 1 << 26, 1);
    expect("slots", p.c.num_slots > 0, 1);
    return hipSuccess;
}
hipError_t launch_read(int, int head_dim, int, const ReadParams& p, hipStream_t) {
    ++launched;
    expect("chunks", p.chunks % p.per_slot == 0 && p.chunks > 0 && p.chunks <= (1ll << 33), 1);
    expect("chunks of a slot", p.per_slot, p.c.kv_heads * head_dim / 8);
    return hipSuccess;
}
hipError_t launch_prompt(int, int, const PromptParams& p, hipStream_t) {
    ++launched;
    expect("tiles hold the rows", (int64_t)p.tiles * PROMPT_ROWS + PROMPT_ROWS > (int64_t)p.total_q * p.group, 1);
    expect("a grid", (int64_t)p.tiles * p.kv_heads * p.splits + 64 <= 1 << 24, 1);
    expect("splits", p.splits == 1 || (p.splits <= 32 && (int64_t)p.tiles * p.kv_heads * p.splits <= 512), 1);
    expect("scale", p.scale_log2e > 0, 1);
    return hipSuccess;
}
}  // namespace vts

int main() {
    char* A = reinterpret_cast<char*>(0x10000000);  // never dereferenced on the host
    char* B = A + (1ll << 50);
    int32_t* I = reinterpret_cast<int32_t*>(A);
    float* F = reinterpret_cast<float*>(A);
    uint8_t* U = reinterpret_cast<uint8_t*>(A);
    const int kvs[] = {1, 2, 3, 8, 128}, groups[] = {1, 5, 8, 64}, dims[] = {64, 128}, all_bits[] = {4, 8, 16};
    const int sizes[] = {1, 7, 64, 1 << 20};
    const int64_t counts[] = {0, 1, 63, 4096, 1 << 20, 1 << 25, 1ll << 40, INT64_MAX};
    for (int kv : kvs)
        for (int group : groups)
            for (int dim : dims)
                for (int bits : all_bits)
                    for (int size : sizes) {
                        const int heads = kv * group;
                        vts_paged_cache c;
                        memset(&c, 0, sizeof(c));
                        c.k = c.v = A;
                        const int64_t row = bits == 16 ? dim : dim * bits / 8, page = size < 100 ? size : 64;
                        const int64_t s[3] = {row * kv * page, row * kv, row};
                        memcpy(c.k_strides, s, sizeof(s));
                        memcpy(c.v_strides, s, sizeof(s));
                        c.num_pages = 100;
                        c.page_size = (int32_t)page;
                        c.kv_heads = kv;
                        c.head_dim = dim;
                        c.dtype = VTS_F16;
                        vts_microscales m;
                        memset(&m, 0, sizeof(m));
                        m.k = m.v = U;
                        const int64_t r = dim / 32, t[3] = {r * kv * page, r * kv, r};
                        memcpy(m.k_strides, t, sizeof(t));
                        memcpy(m.v_strides, t, sizeof(t));
                        m.bits = bits;
                        const vts_microscales* given = bits == 16 ? nullptr : &m;
                        for (int64_t n : counts) {
                            vts_new_tokens x;
                            memset(&x, 0, sizeof(x));
                            x.q = x.k = x.v = A;
                            x.q_strides[0] = x.k_strides[0] = x.v_strides[0] = INT64_MAX / 8 * 8;
                            x.q_strides[1] = x.k_strides[1] = x.v_strides[1] = dim;
                            x.rotary = F;
                            x.rot = dim;
                            x.max_position = INT32_MAX;
                            x.positions = x.slots = I;
                            x.tokens = n;
                            x.q_out = B;
                            x.heads = heads;
                            expect("write", vts_write_cache(&c, given, &x, 0),
                                   n > (1 << 25) ? VTS_ERR_UNSUPPORTED : VTS_OK);
                            const bool fits = n <= (1ll << 33) / (kv * dim / 8);
                            expect("read", vts_read_cache(&c, given, I, n, A, B, 0),
                                   fits ? VTS_OK : VTS_ERR_UNSUPPORTED);
                            for (int64_t batch : {(int64_t)0, (int64_t)1, (int64_t)1000, n}) {
                                vts_prompts a;
                                memset(&a, 0, sizeof(a));
                                a.q = a.k = a.v = A;
                                a.q_strides[0] = (int64_t)heads * dim;
                                a.q_strides[1] = a.k_strides[1] = a.v_strides[1] = dim;
                                a.k_strides[0] = a.v_strides[0] = (int64_t)kv * dim;
                                a.cu_q = a.cu_k = I;
                                a.batch = batch;
                                a.total_q = a.total_k = n;
                                a.heads = heads;
                                a.kv_heads = kv;
                                a.head_dim = dim;
                                a.dtype = VTS_BF16;
                                const size_t need =
                                    vts_prompt_attention_workspace_bytes(batch, n, n, heads, kv, dim);
                                const int st = vts_prompt_attention(&a, 1, -0.1f, B, 0, 1, A, need, 0);
                                expect("prompt", st == VTS_OK || (st == VTS_ERR_UNSUPPORTED && n >= (1 << 20)), 1);
                            }
                        }
                        if (bits == 16) continue;
                        for (int batch : {0, 1, 63, 4096})
                            for (int draft : {1, 7, 64})
                                for (int k = 0; k < 2; ++k) {
                                    if ((int64_t)batch * draft * heads > INT32_MAX) continue;
                                    const int64_t q[3] = {8192, 4096, 128};
                                    c.batch = batch;
                                    c.page_table = c.seq_lens = I;
                                    c.page_table_stride = c.page_table_width = size > 100 ? 9000 : INT32_MAX;
                                    const size_t need = vts_tree_attention_microscaled_workspace_bytes(
                                        batch, draft, heads, kv, dim, k * 2048);
                                    expect("size", need > 65536, 1);
                                    expect("attend",
                                           vts_tree_attention_microscaled(&c, &m, A, q, draft, heads, 0, k ? I : 0,
                                                                          k * 2048, 0.1f, A, 0, A, need, 0), VTS_OK);
                                    if (batch)
                                        expect("attend ws",
                                               vts_tree_attention_microscaled(&c, &m, A, q, draft, heads, 0,
                                                                              k ? I : 0, k * 2048, 0.1f, A, 0, A,
                                                                              need - 1, 0),
                                               VTS_ERR_WORKSPACE);
                                }
                    }
    if (bad || !launched) return 1;
    printf("cache battery clean: %d launches\n", launched);
    return 0;
}
