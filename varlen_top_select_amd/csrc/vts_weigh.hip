// vts_weigh.hip -- attention weight accumulated per cached entry.
//
//   w[b, hk, j] += sum over the counted rows t and the heads of the group of
//                  exp(scale * q . k_j - lse)
//
// The probabilities are formed again from K and the rows' log-sum-exp, so K is
// read once more and V not at all; places are independent, so nothing has to be
// joined: every place belongs to one wave, which adds the rows in a fixed order.
#include "vts_paged.hpp"

namespace vts {

struct WeighShared {
    int64_t scan[WAVES + 1];
    int32_t found;
};

template <int DT, int D, bool HEADS>
__global__ __launch_bounds__(NT, 2) void weigh_kernel(WeighParams p) {
    constexpr int KS = D / 32;
    __shared__ WeighShared sm;
    const PagedParams& c = p.c;
    const Share sh = dense_share<HEADS>(c, p.workers, (int32_t)blockIdx.x, sm.scan, &sm.found);
    if ((int32_t)blockIdx.x >= sh.workers) return;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, grp = lane >> 4;
    int64_t x = sh.begin;
    int32_t b = sh.b;
    int64_t b_unit = sh.b_unit;
    while (x < sh.end) {
        const int32_t n = clamped_len(c, b);
        const int32_t units = units_of<HEADS>(n);
        const int32_t hu = (int32_t)((x - b_unit) / units);
        const int32_t h = HEADS ? hu * WAVES + wave : hu;
        const int64_t g0 = b_unit + (int64_t)hu * units, g1 = g0 + units;
        const int64_t x1 = g1 < sh.end ? g1 : sh.end;
        Places pl;
        pl.count = n;
        pl.first = n - c.draft;
        pl.draft_pos = pl.first;
        pl.slots = nullptr;
        pl.top_k = 0;
        pl.table = c.table + (int64_t)b * c.table_stride;
        const char* kbase = (const char*)c.k.base + (((uint64_t)h * c.k.head_stride) << 4);
        float* wrow = p.weights + b * p.w_batch + h * p.w_head;
        for (int32_t u = (int32_t)(x - g0); u < (int32_t)(x1 - g0); ++u) {
            const int32_t j0 = HEADS ? u * 32 : u * UNIT + wave * 32;
            const Entry e = issue_entry<false>(c, pl, j0 + (lane & 31));
            const uint32_t off =
                resolve_entry<false>(c, c.k.page_stride, c.k.pos_stride, e);
            const uint32_t have = (uint32_t)ballot(off != NO_PLACE);
            if (have == 0) continue;
            const uint32_t safe = off == NO_PLACE ? 0 : off;
            u32x4 k[2][KS];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const uint32_t r = from_lane(safe, hh * 16 + col);
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    k[hh][s] = row_load<u32x4, HEADS>(kbase, r, s * 64 + grp * 16);
            }
            float acc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0;
            for (int32_t m0 = 0; m0 < p.rows; m0 += 16) {
                const int32_t row = m0 + col;
                const bool ok = row < p.rows;
                const int32_t t = ok ? row / c.group : 0;
                const int32_t head = h * c.group + (ok ? row - t * c.group : 0);
                const char* at = (const char*)p.q + 2 * (b * p.q_batch + t * p.q_row + head * p.q_head);
                u32x4 q[KS];
#pragma unroll
                for (int s = 0; s < KS; ++s) q[s] = gload((const u32x4*)(at + s * 64 + grp * 16));
                const int64_t bt = (int64_t)b * c.draft + t;
                uint64_t bits;
                if (p.tree_mask)
                    bits = (uint64_t)gload(p.tree_mask + bt);
                else
                    bits = t >= 63 ? ~0ull : (2ull << t) - 1;
                const float lse = gload(p.lse + bt * c.heads + head);
                const bool counts = ok && lse != NEG_INF && (!p.row_keep || gload(p.row_keep + bt));
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    f32x4 s = {0, 0, 0, 0};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) s = mfma<DT>(k[hh][ks], q[ks], s);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t d = j0 + hh * 16 + grp * 4 + i - pl.first;
                        const bool see =
                            counts && (d < 0 || (d < MAX_DRAFT && ((bits >> (d & 63)) & 1)));
                        const float y = __builtin_amdgcn_exp2f(s[i] * p.scale_log2e -
                                                               lse * 1.4426950408889634f);
                        acc[hh * 4 + i] += see ? y : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) acc[i] += __shfl_xor(acc[i], d);
            if (col < 8) {
                const int place = (col >> 2) * 16 + grp * 4 + (col & 3);
                float y = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) y = col == i ? acc[i] : y;
                const int32_t j = j0 + place;
                if (((have >> place) & 1u) && j < p.width)
                    gstore(wrow + j, gload(wrow + j) + y);
            }
        }
        x = x1;
        if (hu + 1 == head_units<HEADS>(c) && x1 == g1) {
            b_unit = g1;
            ++b;
        }
    }
}

template <int DT, int D>
static hipError_t launch_dt(const WeighParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)p.workers), block(NT);
    if (p.heads_on_waves)
        hipLaunchKernelGGL((weigh_kernel<DT, D, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((weigh_kernel<DT, D, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_weigh(int dtype, int head_dim, const WeighParams& p, hipStream_t stream) {
    if (dtype == BF16)
        return head_dim == 64 ? launch_dt<BF16, 64>(p, stream) : launch_dt<BF16, 128>(p, stream);
    return head_dim == 64 ? launch_dt<F16, 64>(p, stream) : launch_dt<F16, 128>(p, stream);
}

}  // namespace vts
