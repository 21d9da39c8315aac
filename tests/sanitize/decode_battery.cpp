// Exercise of the decode-step operators' host side (argument checks, plans, workspace
// sizes) under AddressSanitizer and UndefinedBehaviorSanitizer.  Every call uses
// fake device pointers; the launches below stand in for the kernels and check that
// the plans they get hold together.  Exits non-zero on an unexpected status.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "../../include/vts.h"
#include "../../varlen_top_select_amd/csrc/vts_decode.h"

static int bad = 0, launched = 0;
static void expect(const char* what, long long got, long long want) {
    if (got != want) {
        fprintf(stderr, "%s: %lld, expected %lld\n", what, got, want);
        ++bad;
    }
}

namespace vts {
int check_device(void*, int*, int*) { return VTS_OK; }
hipError_t launch_attend(int, int, const AttendParams& p, hipStream_t) {
    ++launched;
    expect("rows fit their blocks", (int64_t)p.block_rows * p.row_blocks >= p.rows, 1);
    expect("tickets", (int64_t)p.workers * p.row_blocks <= MAX_TICKETS && p.workers > 0, 1);
    expect("scale", p.scale_log2e > 0, 1);
    return hipSuccess;
}
hipError_t launch_weigh(int, int, const WeighParams&, hipStream_t) { return ++launched, hipSuccess; }
hipError_t launch_evict(const EvictParams&, hipStream_t) { return ++launched, hipSuccess; }
hipError_t launch_verify(int, const VerifyParams& p, hipStream_t) {
    ++launched;
    expect("slices", p.slices >= 1 && p.slices <= 64, 1);
    return hipSuccess;
}
}  // namespace vts

int main() {
    char* A = reinterpret_cast<char*>(0x10000000);  // never dereferenced on the host
    int32_t* I = reinterpret_cast<int32_t*>(A);
    float* F = reinterpret_cast<float*>(A);
    const size_t big = (size_t)1 << 50;
    const int64_t q[3] = {8192, 4096, 128};
    const int drafts[] = {1, 2, 7, 33, 64}, kvs[] = {1, 2, 3, 8, 128}, groups[] = {1, 5, 8, 64};
    const int sizes[] = {1, 7, 64, 1 << 20}, batches[] = {0, 1, 63, 4096};
    for (int draft : drafts)
        for (int kv : kvs)
            for (int group : groups)
                for (int size : sizes)
                    for (int batch : batches) {
                        if ((int64_t)batch * draft * kv * group > INT32_MAX) continue;
                        vts_paged_cache c;
                        memset(&c, 0, sizeof(c));
                        c.k = c.v = A;
                        const int64_t s[3] = {(int64_t)128 * kv * (size < 100 ? size : 64), 128 * kv, 128};
                        memcpy(c.k_strides, s, sizeof(s));
                        memcpy(c.v_strides, s, sizeof(s));
                        c.page_table = c.seq_lens = I;
                        c.page_table_stride = c.page_table_width = size > 100 ? 9000 : INT32_MAX;
                        c.num_pages = 100;
                        c.page_size = size < 100 ? size : 64;
                        c.kv_heads = kv;
                        c.head_dim = 128;
                        c.batch = batch;
                        c.dtype = VTS_BF16;
                        const int heads = kv * group;
                        for (int k = 0; k < 2; ++k) {
                            const size_t need =
                                vts_tree_attention_workspace_bytes(batch, draft, heads, kv, 128, k * 2048);
                            expect("size", need > 65536, 1);
                            expect("attend", vts_tree_attention(&c, A, q, draft, heads, 0, k ? I : 0, k * 2048,
                                                                k ? -0.1f : 0.0f, A, 0, A, need, 0), VTS_OK);
                            if (batch)
                                expect("attend ws", vts_tree_attention(&c, A, q, draft, heads, 0, k ? I : 0,
                                                                       k * 2048, 1.0f, A, 0, A, need - 1, 0),
                                       VTS_ERR_WORKSPACE);
                        }
                        expect("weigh", vts_attention_weight_add(&c, A, q, draft, heads, 0, F, 0, 1.0f, F,
                                                                 1 << 20, 1 << 10, 1 << 10, 0), VTS_OK);
                        expect("evict", vts_evict_cache(&c, F, 1 << 20, 1 << 10, 1 << 10, 64, 4, 8, A, s, A, s,
                                                        64, I, 64, 64, I, I, F + (1 << 28), 0), VTS_OK);
                    }
    const int64_t vocabs[] = {1, 4095, 131072, INT32_MAX - 65536}, counts[] = {1, 16, 8192, 8193, 1 << 21};
    for (int64_t vocab : vocabs)
        for (int64_t n : counts) {
            const size_t need = vts_verify_draft_workspace_bytes(n, vocab);
            expect("verify", vts_verify_draft(A, VTS_F16, vocab * 4, vocab, A, vocab * 3, vocab, I, I, F, n, 3,
                                              vocab, I, I, I, A, need, 0), VTS_OK);
            expect("verify ws", vts_verify_draft(A, VTS_F16, vocab * 4, vocab, A, vocab * 3, vocab, I, I, F, n,
                                                 3, vocab, I, I, I, A, need - 1, 0), VTS_ERR_WORKSPACE);
        }
    expect("null cache", vts_tree_attention(0, A, q, 1, 8, 0, 0, 0, 1.0f, A, 0, A, big, 0), VTS_ERR_INVALID);
    expect("null cache", vts_attention_weight_add(0, A, q, 1, 8, 0, F, 0, 1.0f, F, 1, 1, 1, 0), VTS_ERR_INVALID);
    expect("null cache", vts_evict_cache(0, F, 1, 1, 1, 1, 0, 0, A, q, A, q, 1, I, 1, 1, I, I, F, 0),
           VTS_ERR_INVALID);
    if (bad || !launched) return 1;
    printf("decode battery clean: %d launches\n", launched);
    return 0;
}
