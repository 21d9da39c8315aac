// vts_weigh.hip -- attention weight accumulated per cached entry.
//
//   w[b, hk, j] += sum over the counted rows t and the heads of the group of
//                  exp(scale * q . k_j - lse)
//
// The probabilities are formed again from K and the rows' log-sum-exp, so K is
// read once more and V not at all; places are independent, so nothing has to be
// joined: every place belongs to one wave, which adds the rows in a fixed order.
//
// The memory bounds it: K once, and a read and a write of w.  K rows come whole,
// 16 bytes a lane, one tile ahead, and turn into operands in LDS; with four KV
// heads or a multiple the waves take a head each and read whole rows of the
// cache (as in vts_attend.hip).  Up to 16 rows their q stays in registers,
// beyond that it lies in LDS (up to 256 rows) or comes from the caches.
#include "vts_paged.hpp"

namespace vts {

enum { ROWS_REG = 0, ROWS_LDS = 1, ROWS_FAR = 2 };

template <int D, int ROWS>
struct WeighShared {
    u32x4 k[WAVES][32 * (D / 8)];
    u32x4 q[ROWS == ROWS_LDS ? 16 * (D / 32) : 1][64];  // 256 rows, or 64 of each wave's
};

// What a lane holds of row `row`: its operands, and when it counts its log-sum-exp.
template <int DT, int D>
struct WeighRow {
    static constexpr int KS = D / 32;
    u32x4 q[KS];
    uint64_t bits;
    float lse2;
    bool counts;

    __device__ __forceinline__ void load(const WeighParams& p, int32_t b, int32_t h, int32_t row,
                                         int grp, bool with_q) {
        const PagedParams& c = p.c;
        const bool ok = row < p.rows;
        const int32_t t = ok ? row / c.group : 0;
        const int32_t head = h * c.group + (ok ? row - t * c.group : 0);
        if (with_q) {
            const char* at =
                (const char*)p.q + 2 * (b * p.q_batch + t * p.q_row + head * p.q_head);
#pragma unroll
            for (int s = 0; s < KS; ++s) q[s] = gload((const u32x4*)(at + s * 64 + grp * 16));
        }
        const int64_t bt = (int64_t)b * c.draft + t;
        if (p.tree_mask)
            bits = (uint64_t)gload(p.tree_mask + bt);
        else
            bits = t >= 63 ? ~0ull : (2ull << t) - 1;
        const float lse = gload(p.lse + bt * c.heads + head);
        counts = ok && lse != NEG_INF && (!p.row_keep || gload(p.row_keep + bt));
        lse2 = lse * 1.4426950408889634f;
    }
};

template <int DT, int D, bool HEADS, int ROWS>
__global__ __launch_bounds__(NT, ROWS == ROWS_LDS && D == 128 ? 1 : 2) void weigh_kernel(WeighParams p) {
    constexpr int KS = D / 32, CH = D / 8, RPL = 64 / CH, PLACES = HEADS ? 32 : 32 * WAVES;
    __shared__ WeighShared<D, ROWS> sm;
    const PagedParams& c = p.c;
    const Share sh = dense_share<PLACES, HEADS>(c, p.workers, (int32_t)blockIdx.x);
    if ((int32_t)blockIdx.x >= sh.workers) return;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, grp = lane >> 4;
    // the row tiles of this wave's head in sm.q
    const int q0 = ROWS == ROWS_LDS && HEADS ? wave * 4 : 0;
    int64_t x = sh.begin;
    int32_t b = sh.b;
    int64_t b_unit = sh.b_unit;
    while (x < sh.end) {
        const int32_t n = uniform_len(c, b);
        const int32_t units = units_of<PLACES>(n);
        const int32_t hu = (int32_t)((x - b_unit) / units);
        const int32_t h = HEADS ? hu * WAVES + wave : hu;
        const int64_t g0 = b_unit + (int64_t)hu * units, g1 = g0 + units;
        const int64_t x1 = g1 < sh.end ? g1 : sh.end;
        const int32_t u0 = (int32_t)(x - g0), u1 = (int32_t)(x1 - g0);
        Places pl;
        pl.count = n;
        pl.first = n - c.draft;
        pl.draft_pos = pl.first;
        pl.slots = nullptr;
        pl.top_k = 0;
        pl.table = c.table + (int64_t)b * c.table_stride;
        const char* kbase = (const char*)c.k.base + (((uint64_t)h * c.k.head_stride) << 4);
        float* wrow = p.weights + b * p.w_batch + h * p.w_head;
        const auto first_place = [&](int32_t u) { return HEADS ? u * 32 : u * PLACES + wave * 32; };
        const auto issue = [&](int32_t u) {
            return issue_entry<false>(c, pl, first_place(u) + (lane & 31));
        };
        const auto resolve = [&](const Entry& e) {
            return resolve_entry<false>(c, c.k.page_stride, c.k.pos_stride, e);
        };
        u32x4 k[2 * KS];
        const auto load_k = [&](uint32_t off) {
            const uint32_t safe = off == NO_PLACE ? 0 : off;
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i)
                k[i] = row_load<u32x4, true>(kbase, from_lane(safe, i * RPL + lane / CH),
                                             (lane % CH) * 16);
        };
        uint32_t off = resolve(issue(u0));
        Entry next = issue(u0 + 1);
        load_k(off);
        WeighRow<DT, D> row;
        if constexpr (ROWS == ROWS_REG) row.load(p, b, h, col, grp, true);
        if constexpr (ROWS == ROWS_LDS) {
            if (!HEADS) __syncthreads();  // the rows of the last list are done with
            const int tiles = (p.rows + 15) / 16;
            for (int mt = HEADS ? 0 : wave; mt < tiles; mt += HEADS ? 1 : WAVES) {
                row.load(p, b, h, mt * 16 + col, grp, true);
#pragma unroll
                for (int s = 0; s < KS; ++s) sm.q[(q0 + mt) * KS + s][lane] = row.q[s];
            }
            if (!HEADS) __syncthreads();
        }
        for (int32_t u = u0; u < u1; ++u) {
            const int32_t j0 = first_place(u);
            const uint32_t have = (uint32_t)ballot(off != NO_PLACE);
            const bool drafted = j0 + 31 >= pl.first;
            // the value this lane writes at the end, and where: of the lane's eight
            // places (4 * grp + .. of each half) the one its column names
            const int e = col >> 1;
            const int place = (e >> 2) * 16 + grp * 4 + (e & 3);
            const bool mine = !(col & 1) && ((have >> place) & 1u) && j0 + place < p.width;
            float old = 0;
            if (mine) old = gload(wrow + j0 + place);
            const uint32_t off_next = resolve(next);
            next = issue(u + 2);
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) {
                const int r = i * RPL + lane / CH;
                sm.k[wave][r * CH + ((lane % CH) ^ swizzled<D>(r))] = k[i];
            }
            // the wave's own stores come before its loads; the compiler has to know
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (u + 1 < u1) load_k(off_next);
            u32x4 a[2][KS];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int r = hh * 16 + col;
                    a[hh][s] = sm.k[wave][r * CH + ((s * 4 + grp) ^ swizzled<D>(r))];
                }
            __builtin_amdgcn_wave_barrier();
            float acc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0;
            const auto add = [&](const WeighRow<DT, D>& r, const u32x4 (&q)[KS]) {
                f32x4 s[2];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    s[hh] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) s[hh] = mfma<DT>(a[hh][ks], q[ks], s[hh]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    bool see = r.counts;
                    if (drafted) {
                        const int32_t d = j0 + (i >> 2) * 16 + grp * 4 + (i & 3) - pl.first;
                        see = see && (d < 0 || ((r.bits >> (d & 63)) & 1));
                    }
                    const float y = __builtin_amdgcn_exp2f(
                        fmaf(s[i >> 2][i & 3], p.scale_log2e, -r.lse2));
                    acc[i] += see ? y : 0.0f;
                }
            };
            if constexpr (ROWS == ROWS_REG) {
                add(row, row.q);
            } else {
#pragma unroll 1
                for (int32_t m0 = 0; m0 < p.rows; m0 += 16) {
                    row.load(p, b, h, m0 + col, grp, ROWS == ROWS_FAR);
                    if constexpr (ROWS == ROWS_LDS)
#pragma unroll
                        for (int s = 0; s < KS; ++s) row.q[s] = sm.q[(q0 + m0 / 16) * KS + s][lane];
                    add(row, row.q);
                }
            }
            // Sums over the 16 columns: at each step a lane sends half of its values
            // and keeps the other half, so 8 + 4 + 2 + 1 exchanges become 4 + 2 + 1 + 1.
            float four[4], two[2], one;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float send = (col & 8) ? acc[i] : acc[4 + i];
                const float keep = (col & 8) ? acc[4 + i] : acc[i];
                four[i] = keep + __shfl_xor(send, 8);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float send = (col & 4) ? four[i] : four[2 + i];
                const float keep = (col & 4) ? four[2 + i] : four[i];
                two[i] = keep + __shfl_xor(send, 4);
            }
            {
                const float send = (col & 2) ? two[0] : two[1];
                const float keep = (col & 2) ? two[1] : two[0];
                one = keep + __shfl_xor(send, 2);
            }
            one += __shfl_xor(one, 1);
            if (mine) gstore(wrow + j0 + place, old + one);
            off = off_next;
        }
        x = x1;
        if (hu + 1 == head_units<HEADS>(c) && x1 == g1) {
            b_unit = g1;
            ++b;
        }
    }
}

template <int DT, int D, bool HEADS>
static hipError_t launch_rows(const WeighParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)p.workers), block(NT);
    // (with a head to each wave there are at most 64 rows)
    if (p.rows <= 16)
        hipLaunchKernelGGL((weigh_kernel<DT, D, HEADS, ROWS_REG>), grid, block, 0, stream, p);
    else if (HEADS || p.rows <= 256)
        hipLaunchKernelGGL((weigh_kernel<DT, D, HEADS, ROWS_LDS>), grid, block, 0, stream, p);
    else if constexpr (!HEADS)
        hipLaunchKernelGGL((weigh_kernel<DT, D, HEADS, ROWS_FAR>), grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int DT, int D>
static hipError_t launch_dt(const WeighParams& p, hipStream_t stream) {
    return p.heads_on_waves ? launch_rows<DT, D, true>(p, stream)
                            : launch_rows<DT, D, false>(p, stream);
}

hipError_t launch_weigh(int dtype, int head_dim, const WeighParams& p, hipStream_t stream) {
    if (dtype == BF16)
        return head_dim == 64 ? launch_dt<BF16, 64>(p, stream) : launch_dt<BF16, 128>(p, stream);
    return head_dim == 64 ? launch_dt<F16, 64>(p, stream) : launch_dt<F16, 128>(p, stream);
}

}  // namespace vts
