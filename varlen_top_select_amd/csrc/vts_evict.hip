// vts_evict.hip -- eviction from a paged KV cache by accumulated weight.
//
// Two launches.  evict_select: one workgroup per request and KV head finds the
// weight of the last entry to stay by a radix select over order-preserving
// keys (8 bits a pass), then writes the kept positions in order; of equal
// weights the lowest positions stay.  evict_move: the kept K and V rows go to
// the new pages, 16 bytes a lane; that is nearly all of the traffic and runs at
// the rate of a large copy (32 requests of up to 8192 to 4096, 8 heads of 128:
// 208 us of 233, 5.0 TB/s).
//
// The select reads the weights again in each pass, from the cache.  With the
// keys of 16384 entries in registers, its loops unrolled, the same batch took 228
// us, but one row of 1088 18 us for 13: code that runs once waits for its own
// instructions.
#include "vts_paged.hpp"

namespace vts {

constexpr int ET = 1024;  // threads of evict_select
constexpr int EW = ET / 64;

struct EvictShared {
    uint32_t hist[256];
    uint32_t scan[2][EW];
    uint32_t digit, above;
};

__global__ __launch_bounds__(ET) void evict_select(EvictParams p) {
    __shared__ EvictShared sm;
    const PagedParams& c = p.c;
    const int32_t b = (int32_t)(blockIdx.x / c.kv_heads), h = (int32_t)(blockIdx.x % c.kv_heads);
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
    int32_t n = clamped_len(c, b);
    if (n > p.width) n = p.width;
    const int32_t count = n < p.keep ? n : p.keep;
    const float* w = p.weights + b * p.w_batch + h * p.w_head;
    const int64_t row = (int64_t)blockIdx.x * p.keep;
    if (tid == 0 && h == 0) gstore(p.out_lens + b, count);
    for (int32_t i = count + tid; i < p.keep; i += ET) {
        gstore(p.kept + row + i, -1);
        gstore(p.out_weights + row + i, 0.0f);
    }
    if (n <= p.keep) {
        for (int32_t i = tid; i < n; i += ET) {
            gstore(p.kept + row + i, i);
            gstore(p.out_weights + row + i, gload(w + i));
        }
        return;
    }
    // positions [s0, s1) compete for `need` places
    const int32_t s0 = p.sinks, s1 = n - p.recent;
    const uint32_t need = (uint32_t)(p.keep - p.sinks - p.recent);
    uint32_t key = 0, left = need;  // the key's digits so far, places left among them
    for (int shift = 24; need && shift >= 0; shift -= 8) {
        if (tid < 256) sm.hist[tid] = 0;
        __syncthreads();
        for (int32_t i = s0 + tid; i < s1; i += ET) {
            const uint32_t k = canon_key<F32>(to_key<F32>(__builtin_bit_cast(uint32_t, gload(w + i))));
            if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8)))
                atomicAdd(&sm.hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (wave == 0) {
            // lane l: bins 4 * (63 - l) .. + 3, so lanes run from the largest digit
            const int base = 4 * (63 - lane);
            const uint32_t h3 = sm.hist[base + 3], h2 = sm.hist[base + 2], h1 = sm.hist[base + 1],
                           h0 = sm.hist[base];
            uint32_t inc = h0 + h1 + h2 + h3;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_up(inc, d);
                if (lane >= d) inc += o;
            }
            uint32_t above = inc - (h0 + h1 + h2 + h3);
            if (above < left && inc >= left) {
                uint32_t digit = base + 3;
                if (above + h3 < left) {
                    above += h3, digit = base + 2;
                    if (above + h2 < left) {
                        above += h2, digit = base + 1;
                        if (above + h1 < left) above += h1, digit = base;
                    }
                }
                sm.digit = digit;
                sm.above = above;
            }
        }
        __syncthreads();
        key |= sm.digit << shift;
        left -= sm.above;
        __syncthreads();
    }
    // everything above `key` stays, and the first `left` of the entries equal to it
    uint32_t kept = 0, ties = 0;
    for (int32_t i0 = 0; i0 < n; i0 += ET) {
        const int32_t i = i0 + tid;
        bool take = false, tie = false;
        if (i < n) {
            if (i < s0 || i >= s1) {
                take = true;
            } else if (need) {
                const uint32_t k =
                    canon_key<F32>(to_key<F32>(__builtin_bit_cast(uint32_t, gload(w + i))));
                take = k > key;
                tie = k == key;
            }
        }
        const uint64_t mt = ballot(tie);
        if (lane == 0) sm.scan[0][wave] = (uint32_t)__popcll(mt);
        __syncthreads();
        uint32_t before = ties, all = 0;
        for (int v = 0; v < EW; ++v) {
            if (v < wave) before += sm.scan[0][v];
            all += sm.scan[0][v];
        }
        ties += all;
        take = take || (tie && before + mbcnt(mt) < left);
        const uint64_t mk = ballot(take);
        if (lane == 0) sm.scan[1][wave] = (uint32_t)__popcll(mk);
        __syncthreads();
        uint32_t at = kept;
        all = 0;
        for (int v = 0; v < EW; ++v) {
            if (v < wave) at += sm.scan[1][v];
            all += sm.scan[1][v];
        }
        kept += all;
        at += mbcnt(mk);
        if (take && at < (uint32_t)p.keep) {
            gstore(p.kept + row + at, i);
            gstore(p.out_weights + row + at, gload(w + i));
        }
    }
}

constexpr int MOVE_ROWS = 64;  // rows per workgroup of evict_move

__global__ __launch_bounds__(NT) void evict_move(EvictParams p) {
    const PagedParams& c = p.c;
    const int32_t tiles = (p.keep + MOVE_ROWS - 1) / MOVE_ROWS;
    const int32_t bh = (int32_t)(blockIdx.x / tiles), tile = (int32_t)(blockIdx.x % tiles);
    const int32_t b = bh / c.kv_heads, h = bh % c.kv_heads;
    const int32_t vecs = p.row_vecs;
    for (int32_t x = threadIdx.x; x < MOVE_ROWS * vecs; x += NT) {
        const int32_t i = tile * MOVE_ROWS + x / vecs, part = x % vecs;
        if (i >= p.keep) continue;
        const int32_t j = gload(p.kept + (int64_t)bh * p.keep + i);
        if (j < 0) continue;
        const int32_t to = gload(p.out_table + b * p.out_table_stride + i / c.page_size);
        if (to < 0 || to >= p.out_pages) continue;
        const int32_t from = gload(c.table + b * c.table_stride + j / c.page_size);
        u32x4 k = {0, 0, 0, 0}, v = {0, 0, 0, 0};
        if (from >= 0 && from < c.num_pages) {
            const uint32_t js = (uint32_t)(j % c.page_size);
            k = row_load<u32x4>(c.k.base, (uint32_t)from * c.k.page_stride + js * c.k.pos_stride +
                                              h * c.k.head_stride + part, 0);
            v = row_load<u32x4>(c.v.base, (uint32_t)from * c.v.page_stride + js * c.v.pos_stride +
                                              h * c.v.head_stride + part, 0);
        }
        const uint32_t is = (uint32_t)(i % c.page_size);
        const uint32_t ko = (uint32_t)to * p.k_out.page_stride + is * p.k_out.pos_stride +
                            h * p.k_out.head_stride + part;
        const uint32_t vo = (uint32_t)to * p.v_out.page_stride + is * p.v_out.pos_stride +
                            h * p.v_out.head_stride + part;
        gstore((u32x4*)((char*)p.k_out.base + ((uint64_t)ko << 4)), k);
        gstore((u32x4*)((char*)p.v_out.base + ((uint64_t)vo << 4)), v);
    }
}

hipError_t launch_evict(const EvictParams& p, hipStream_t stream) {
    const uint32_t rows = (uint32_t)(p.c.batch * p.c.kv_heads);
    hipLaunchKernelGGL(evict_select, dim3(rows), dim3(ET), 0, stream, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(evict_move, dim3(rows * ((p.keep + MOVE_ROWS - 1) / MOVE_ROWS)), dim3(NT),
                       0, stream, p);
    return hipGetLastError();
}

}  // namespace vts
