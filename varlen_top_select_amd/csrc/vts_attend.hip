// vts_attend.hip -- attention of drafted tokens over a paged KV cache.
//
//   o = sum_j p_j v_j,  p = softmax_j(scale * q . k_j)
//
// over the places a query row sees: the cached prefix (or a list of slots per
// row) and the drafted tokens its mask names.  All query rows that share a KV
// head and a list of places are taken together (drafted tokens x grouped
// heads), up to 128 of them for each time that K and V are read.
//
// One pass: each wave walks its 32-place tiles with a running maximum m, sum l
// and output O per query row (32-bit), and the waves, then the workgroups that
// share a list, join theirs: O = sum_w 2^(m_w - m) O_w and the same for l.  m is
// only raised when a score passes it by a margin, so that most tiles need no
// exchange between lanes.  p is rounded to the cache's type for the second product
// (at most half a step, 2^-8 of a bf16 p and 2^-11 of an fp16 one, which average
// out over the places); l sums the unrounded p.  In bf16 m is the maximum and the
// margin 2^8: p has its full precision down to 2^-126.  fp16 loses it below 2^-14,
// so there m lies 2^SHIFT below the maximum and the margin ends at 2^15, next to
// fp16's largest value: p is rounded to 2^-11 of itself down to 2^-(14 + SHIFT) of
// the row's greatest and to 2^-(25 + SHIFT) of that below, so that many light
// places next to a heavy one keep their sum.  (SHIFT 11: 8 trees of 16 up to 65536
// in fp16 take 375 us, for 361 with none and a margin of 2^8, 365 with 7 and 385
// with 14; 64 chains up to 16384 453 with any.)
#include "vts_paged.hpp"

namespace vts {

// How a workgroup's waves share the work.
enum Mode : int {
    KEYS = 0,   // four waves, 32 places each of the same rows
    HEADS = 1,  // four waves, a KV head each at the same 32 places
    WIDE2 = 2,  // eight waves: two groups of 32 rows, four times 32 places
    WIDE4 = 4,  // eight waves: four groups of 32 rows, twice 32 places
};

constexpr int threads_of(int mode) { return mode >= WIDE2 ? 512 : NT; }

template <int D, int MT, int MODE>
struct AttendShape {
    static constexpr bool WIDE = MODE >= WIDE2;
    static constexpr int NW = threads_of(MODE) / 64;       // waves
    static constexpr int RG = WIDE ? MODE : 1;             // groups of rows
    static constexpr int KG = WIDE ? NW / RG : MODE == HEADS ? 1 : NW;  // groups of places
    static constexpr int SUBS = MODE == HEADS ? NW : RG;   // blocks of 16 * MT rows
    static constexpr int ROWS = SUBS * 16 * MT;
};

// A wide workgroup's places, K as operands (swizzled) and V in whole rows.
template <int D, int PLACES>
struct WideTiles {
    u32x4 k[2][PLACES * (D / 8)], v[2][PLACES * (D / 8)];
    uint8_t there[2][PLACES];
};

template <int D, int MT, int MODE>
struct AttendShared : AttendShape<D, MT, MODE> {
    using S = AttendShape<D, MT, MODE>;
    u32x4 q[MT > 1 ? S::SUBS * MT * (D / 32) : 1][64];  // query rows as operands, from 32 rows on
    union {
        // a wave's K rows on their way from the order of whole rows to operands
        u32x4 k[S::WIDE ? 1 : WAVES][S::WIDE ? 1 : 32 * (D / 8)];
        WideTiles<D, S::WIDE ? S::KG * 32 : 1> w;
        // outputs of waves to be joined, padded: the 16 rows of a store fall on all banks
        float o[MODE == HEADS ? 1 : S::WIDE ? S::KG - 1 : 2][MODE == HEADS ? 1 : S::ROWS][D + 4];
    };
    float ml[S::KG][S::ROWS][2];
    uint32_t last;
};

template <int DT, int D, int MT, bool SLOTS, int MODE>
struct Attend {
    static constexpr int KS = D / 32;       // steps of the first product
    static constexpr int VB = D / 16 * 2;   // bytes of a V row per lane
    static constexpr int VW = VB / 4;       // words of a V row per lane
    static constexpr int NTILE = D / 16;    // 16-row tiles of the second product
    static constexpr int JOIN = 32;         // parts joined by one workgroup
    using S = AttendShape<D, MT, MODE>;
    static constexpr bool HEAD = MODE == HEADS, WIDE = S::WIDE;
    static constexpr int T = S::NW * 64;    // threads
    // whether a cache row is read once by the whole call, as far as it is known
    // (the slots of two rows may be the same): such loads leave the caches alone.
    // 128 lists of 2048 slots, 64 heads: 112 us without, 104 with.
    static constexpr bool ONCE = HEAD || (SLOTS && !WIDE);
    static constexpr int ROWS = S::ROWS;
    // of m, see above: how far below the maximum it is put, and when it is raised
    static constexpr float SHIFT = DT == F16 ? 11 : 0, RAISE = DT == F16 ? 15 : 8;
    using VRow = typename std::conditional<D == 128, u32x4, u32x2>::type;

    const AttendParams& p;
    AttendShared<D, MT, MODE>& sm;
    int tid, lane, wave, col, grp;
    int rg, kg;  // the wave's group of rows and of places
    uint32_t page_stride, pos_stride;  // of K in lanes 0..31, of V above
    int32_t req, head_unit, mb, t0;  // t0: the row of a slot list
    Places pl;
    static constexpr bool QL = MT > 1;  // query rows in LDS
    static constexpr int CH = D / 8;    // 16-byte chunks of a row
    static constexpr int RPL = 64 / CH; // rows of one load instruction
    // Wide: a thread's chunks of a unit's places, and a wave's rows of them
    static constexpr int LOADS = WIDE ? S::KG * 32 * CH / T : 1;
    static constexpr int MINE = LOADS * RPL;
    u32x4 q[QL ? 1 : KS];
    uint64_t bits[MT];
    f32x4 o[MT][NTILE];
    float m[MT], l[MT];
    // the tile on its way: 32 places to a wave, or the wave's rows of the unit
    u32x4 k[WIDE ? LOADS : 2 * KS];
    VRow v[8];
    u32x4 vw[LOADS];
    const void* kbase;
    const void* vbase;

    __device__ Attend(const AttendParams& p_, AttendShared<D, MT, MODE>& s_, int32_t mb_)
        : p(p_), sm(s_), mb(mb_) {
        fresh();
    }
    // The thread's place, opaque to the compiler: called where a stage begins, so
    // that what one stage computes from it is not kept in registers through the
    // others (70 of them, otherwise, through the walk).
    __device__ __forceinline__ void fresh() {
        tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        lane = tid & 63;
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        col = lane & 15;
        grp = lane >> 4;
        rg = WIDE ? wave % S::RG : 0;
        kg = WIDE ? wave / S::RG : HEAD ? 0 : wave;
    }
    // the block of rows that the wave works on
    __device__ __forceinline__ int sub() const { return HEAD ? wave : rg; }

    // row r of block `sub` (a head's, or a group's): the drafted token and the query head
    __device__ __forceinline__ int32_t row_at(int sub, int r) const {
        return HEAD ? r : (mb * S::SUBS + sub) * 16 * MT + r;
    }
    __device__ __forceinline__ bool row_of(int sub, int r, int32_t& t, int32_t& head) const {
        const int32_t row = row_at(sub, r);
        const int32_t h = HEAD ? head_unit * WAVES + sub : head_unit;
        if (SLOTS) {
            t = t0;
            head = h * p.c.group + row;
        } else {
            t = row / p.c.group;
            head = h * p.c.group + (row - t * p.c.group);
        }
        return row < p.rows;
    }

    __device__ __forceinline__ void begin(int32_t b, int32_t h) {
        fresh();
        head_unit = h;
        if (HEAD) h = h * WAVES + wave;
        const PagedParams& c = p.c;
        if (SLOTS) {
            req = b / c.draft;
            t0 = b - req * c.draft;
            pl.slots = p.slots + (int64_t)b * p.top_k;
        } else {
            req = b;
            t0 = 0;
            pl.slots = nullptr;
        }
        const int32_t n = uniform_len(c, req);
        pl.table = c.table + (int64_t)req * c.table_stride;
        pl.top_k = p.top_k;
        pl.draft_pos = n - c.draft;
        pl.first = SLOTS ? p.top_k : n - c.draft;
        pl.count = place_count<SLOTS>(p, n);
        kbase = (const char*)c.k.base + (((uint64_t)h * c.k.head_stride) << 4);
        vbase = (const char*)c.v.base + (((uint64_t)h * c.v.head_stride) << 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            int32_t t, head;
            const bool ok = row_of(sub(), mt * 16 + col, t, head);
            const char* at = (const char*)p.q +
                             2 * (req * p.q_batch + (ok ? t * p.q_row + head * p.q_head : 0));
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                u32x4 x = {0, 0, 0, 0};
                if (QL && !HEAD && (mt * KS + s) % S::KG != kg) continue;
                if (ok) x = gload((const u32x4*)(at + s * 64 + grp * 16));
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] ^= p.q_sign;
                if constexpr (QL)
                    sm.q[q_at(mt, s)][lane] = x;
                else
                    q[s] = x;
            }
            uint64_t w = 0;
            if (ok) {
                if (p.tree_mask)
                    w = (uint64_t)gload(p.tree_mask + (int64_t)req * c.draft + t);
                else
                    w = t >= 63 ? ~0ull : (2ull << t) - 1;
            }
            bits[mt] = w;
            m[mt] = NEG_INF;
            l[mt] = 0;
#pragma unroll
            for (int n2 = 0; n2 < NTILE; ++n2) o[mt][n2] = f32x4{0, 0, 0, 0};
        }
        if constexpr (QL && !HEAD) __syncthreads();
    }
    __device__ __forceinline__ int q_at(int mt, int s) const {
        return (sub() * MT + mt) * KS + s;
    }

    __device__ __forceinline__ int32_t first_place(int32_t u) const {
        return (u * S::KG + kg) * 32;
    }
    // the place that lane l of a wave looks up: of its own 32, or (wide) of its
    // rows of the unit
    __device__ __forceinline__ Entry issue(int32_t u) const {
        const int l = lane & 31;
        if constexpr (WIDE)
            return issue_entry<SLOTS>(p.c, pl, l < MINE ? u * S::KG * 32 + wide_row(l) : -1);
        return issue_entry<SLOTS>(p.c, pl, first_place(u) + l);
    }
    // row i of the wave's rows of a unit
    __device__ __forceinline__ int wide_row(int i) const {
        return (i / RPL * S::NW + wave) * RPL + i % RPL;
    }
    // K offsets in lanes 0..31, V offsets in lanes 32..63
    __device__ __forceinline__ uint32_t resolve(const Entry& e) const {
        return resolve_entry<SLOTS>(p.c, page_stride, pos_stride, e);
    }
    // K goes through LDS: a load instruction then takes whole rows (as the
    // operand's order it would take 64 bytes of each of 16), which the memory gives
    // 8 % faster (64 requests up to 16384: 454 us for 492).
    __device__ __forceinline__ void load_k(uint32_t off) {
        const uint32_t safe = off == NO_PLACE ? 0 : off;
#pragma unroll
        for (int i = 0; i < (WIDE ? LOADS : 2 * KS); ++i)
            k[i] = row_load<u32x4, ONCE>(kbase, from_lane(safe, i * RPL + lane / CH),
                                         (lane % CH) * 16);
    }
    __device__ __forceinline__ void stage_k() {
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) {
            const int r = i * RPL + lane / CH;
            sm.k[wave][r * CH + ((lane % CH) ^ swizzled<D>(r))] = k[i];
        }
        // the wave's own stores come before its loads; the compiler has to know
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    // A wide workgroup's unit: whole rows of K and V, each once, to half `buf`.
    __device__ __forceinline__ void load_wide(uint32_t off) {
        const uint32_t safe = off == NO_PLACE ? 0 : off;
        load_k(off);
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            vw[i] = row_load<u32x4>(vbase, from_lane(safe, 32 + i * RPL + lane / CH),
                                    (lane % CH) * 16);
    }
    __device__ __forceinline__ void stage_wide(uint32_t off, int buf) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = wide_row(i * RPL + lane / CH);
            const bool there = from_lane(off, i * RPL + lane / CH) != NO_PLACE;
            const u32x4 z = {0, 0, 0, 0};
            sm.w.k[buf][r * CH + ((lane % CH) ^ swizzled<D>(r))] = k[i];
            sm.w.v[buf][r * CH + lane % CH] = there ? vw[i] : z;
            if (lane % CH == 0) sm.w.there[buf][r] = there;
        }
    }
    __device__ __forceinline__ u32x4 operand_k(int h, int s, int buf) const {
        const int r = (WIDE ? kg * 32 : 0) + h * 16 + col;
        const int at = r * CH + ((s * 4 + grp) ^ swizzled<D>(r));
        if constexpr (WIDE) return sm.w.k[buf][at];
        return sm.k[wave][at];
    }
    __device__ __forceinline__ VRow wide_v(int buf, int place, int part) const {
        return *(const VRow*)((const char*)&sm.w.v[buf][(kg * 32 + place) * CH] + part * VB);
    }
    // register j: place 4 * grp + j of the first half, or of the second for j >= 4
    __device__ __forceinline__ int v_place(int j) const {
        return (j >> 2) * 16 + grp * 4 + (j & 3);
    }
    __device__ __forceinline__ void load_v(uint32_t off) {
        const uint32_t safe = off == NO_PLACE ? 0 : off;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = row_load<VRow, ONCE>(vbase, from_lane(safe, 32 + v_place(j)), col * VB);
    }

    // The tile's share of O: V rows turned so that each lane holds eight places
    // of one V column, two of them to a word.
    __device__ __forceinline__ void second_product(const u32x4 (&pv)[MT]) {
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            u32x4 lo, hi;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = __builtin_amdgcn_perm(v[2 * j + 1][w], v[2 * j][w], 0x05040100u);
                hi[j] = __builtin_amdgcn_perm(v[2 * j + 1][w], v[2 * j][w], 0x07060302u);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                o[mt][2 * w] = mfma<DT>(lo, pv[mt], o[mt][2 * w]);
                o[mt][2 * w + 1] = mfma<DT>(hi, pv[mt], o[mt][2 * w + 1]);
            }
        }
    }

    // Where not every row sees every place, an infinity or NaN in a V row would
    // reach rows that do not see it (0 * inf).  Such elements' registers are
    // cleared here, and add_rows adds them to the rows that do.  Returns the
    // places that hold any.
    __device__ __forceinline__ uint32_t clear_not_finite() {
        uint32_t bad = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bool f = false;
#pragma unroll
            for (int w = 0; w < VW; ++w) f = f || not_finite<DT>(v[j][w]);
            const uint64_t any = ballot(f);
            if (any == 0) continue;
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if ((any >> (16 * g)) & 0xFFFFu) bad |= 1u << ((j >> 2) * 16 + g * 4 + (j & 3));
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                if (not_finite<DT>(v[j][w] & 0xFFFFu)) v[j][w] &= 0xFFFF0000u;
                if (not_finite<DT>(v[j][w] >> 16)) v[j][w] &= 0xFFFFu;
            }
        }
        return bad;
    }
    __device__ __forceinline__ void add_rows(uint32_t bad, uint32_t off, int32_t j0, int buf,
                                             const u32x4 (&pv)[MT]) {
#pragma unroll 1
        while (bad) {
            const int kk = __builtin_ctz(bad);
            bad &= bad - 1;
            const uint32_t r = WIDE ? 0 : from_lane(off, 32 + kk);
            VRow x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = WIDE ? wide_v(buf, kk, grp * 4 + e)
                            : row_load<VRow>(vbase, r, (grp * 4 + e) * VB);
            const int src = ((kk & 15) >> 2) * 16 + col;
            const int idx = (kk >> 4) * 4 + (kk & 3);
            const int32_t i = j0 + kk - pl.first;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t pair = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) pair = e == idx >> 1 ? pv[mt][e] : pair;
                pair = from_lane(pair, src);
                const float w = to_float<DT>((pair >> (16 * (idx & 1))) & 0xFFFFu);
                const bool see = i < 0 || ((bits[mt] >> (i & 63)) & 1);
#pragma unroll
                for (int n = 0; n < NTILE; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t raw = (x[e][n >> 1] >> (16 * (n & 1))) & 0xFFFFu;
                        const float y = o[mt][n][e] + w * to_float<DT>(raw);
                        o[mt][n][e] = see && not_finite<DT>(raw) ? y : o[mt][n][e];
                    }
            }
        }
    }

    // One tile: scores, the running softmax, O.  `masked`: some place is missing,
    // or some row does not see some place.  The next tile's K rows are asked for
    // as soon as this tile's are used up, and its V rows after the second
    // product, so one of the two is always on its way.
    __device__ __forceinline__ void tile(uint32_t have, bool drafted, uint32_t off, int32_t j0,
                                         bool more, uint32_t off_next, int buf) {
        const float c = p.scale_log2e;
        const bool masked = have != ~0u || drafted;
        if constexpr (!WIDE) {
            stage_k();
            if (more) load_k(off_next);
        }
        f32x4 s[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) s[mt][h] = f32x4{0, 0, 0, 0};
        // step by step over all rows, so that independent products stand between
        // dependent ones
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const u32x4 k0 = operand_k(0, ks, buf), k1 = operand_k(1, ks, buf);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const u32x4 qq = QL ? sm.q[q_at(mt, ks)][lane] : q[QL ? 0 : ks];
                s[mt][0] = mfma<DT>(k0, qq, s[mt][0]);
                s[mt][1] = mfma<DT>(k1, qq, s[mt][1]);
            }
        }
        if (masked) {
            int g = grp;  // opaque: nothing of this is kept in registers between tiles
            asm volatile("" : "+v"(g));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int kk = (e >> 2) * 16 + g * 4 + (e & 3);
                const int32_t i = j0 + kk - pl.first;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t see = (have >> kk) & (((uint32_t)i >> 31) |
                                                         (uint32_t)(bits[mt] >> (i & 63)));
                    s[mt][e >> 2][e & 3] = (see & 1u) ? s[mt][e >> 2][e & 3] : NEG_INF;
                }
            }
        }
        float top[MT];
        bool past = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            top[mt] = NEG_INF;
#pragma unroll
            for (int e = 0; e < 8; ++e) top[mt] = fmaxf(top[mt], s[mt][e >> 2][e & 3]);
            top[mt] *= c;
            past = past || top[mt] > m[mt] + RAISE;
        }
        if (ballot(past)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float up = fmaxf(top[mt], __shfl_xor(top[mt], 16));
                up = fmaxf(up, __shfl_xor(up, 32));
                // (a row that is not past its maximum keeps it)
                up = up > m[mt] + RAISE ? up - SHIFT : m[mt];
                const float f = up == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(m[mt] - up);
                m[mt] = up;
                l[mt] *= f;
#pragma unroll
                for (int n = 0; n < NTILE; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][n][e] *= f;
            }
        }
        u32x4 pv[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float base = m[mt] == NEG_INF ? 0.0f : m[mt];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a =
                    __builtin_amdgcn_exp2f(fmaf(s[mt][e >> 1][2 * (e & 1)], c, -base));
                const float b =
                    __builtin_amdgcn_exp2f(fmaf(s[mt][e >> 1][2 * (e & 1) + 1], c, -base));
                l[mt] += a + b;
                pv[mt][e] = pack2<DT>(a, b);
            }
        }
        if constexpr (WIDE)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = wide_v(buf, v_place(j), col);
        uint32_t bad = 0;
        if (masked) {
            int g = grp;
            asm volatile("" : "+v"(g));
#pragma unroll
            for (int j = 0; j < (WIDE ? 0 : 8); ++j) {  // (a wide unit's are zero already)
                const uint32_t there = (have >> ((j >> 2) * 16 + g * 4 + (j & 3))) & 1u;
#pragma unroll
                for (int w = 0; w < VW; ++w) v[j][w] = there ? v[j][w] : 0;
            }
            if (drafted) bad = clear_not_finite();
        }
        second_product(pv);
        if (bad) add_rows(bad, off, j0, buf, pv);
        if constexpr (!WIDE) {
            if (more) load_v(off_next);
            // the next tile's stores to sm.k come after these loads
            __builtin_amdgcn_wave_barrier();
        }
    }

    // Units [u0, u1) of the places, this wave's 32 of each.
    __device__ __forceinline__ void walk(int32_t u0, int32_t u1) {
        fresh();
        page_stride = lane < 32 ? p.c.k.page_stride : p.c.v.page_stride;
        pos_stride = lane < 32 ? p.c.k.pos_stride : p.c.v.pos_stride;
        uint32_t off = resolve(issue(u0));
        Entry next = issue(u0 + 1);
        if constexpr (WIDE) {
            load_wide(off);
        } else {
            load_k(off);
            load_v(off);
        }
#pragma unroll 1
        for (int32_t u = u0; u < u1; ++u) {
            const int32_t j0 = first_place(u);
            const int buf = u & 1;
            uint32_t have;
            uint32_t off_next;
            if constexpr (WIDE) {
                // the other half may still be read; this one was done with before
                // the last barrier
                stage_wide(off, buf);
                off_next = resolve(next);
                next = issue(u + 2);
                if (u + 1 < u1) load_wide(off_next);
                __syncthreads();
                have = (uint32_t)ballot(sm.w.there[buf][kg * 32 + (lane & 31)]);
            } else {
                off_next = resolve(next);
                next = issue(u + 2);
                have = (uint32_t)ballot(off != NO_PLACE);
            }
            const bool drafted = j0 + 31 >= pl.first;
            tile(have, drafted, off, j0, u + 1 < u1, off_next, buf);
            off = off_next;
        }
    }

    // o[.] += the rows that another wave left in LDS
    __device__ __forceinline__ void put(int slot) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < NTILE; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sm.o[slot][rg * 16 * MT + mt * 16 + col][(grp * 4 + e) * NTILE + n] = o[mt][n][e];
    }
    __device__ __forceinline__ void take(int slot) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < NTILE; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[mt][n][e] +=
                        sm.o[slot][rg * 16 * MT + mt * 16 + col][(grp * 4 + e) * NTILE + n];
    }

    // Joins the waves of different places.  Four waves: the block's rows are
    // then in sm.o[0], sm.ml[0]; wide: in the registers of the first group's.
    __device__ __forceinline__ void join_waves() {
        fresh();
        const int r0 = rg * 16 * MT + col;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            l[mt] += __shfl_xor(l[mt], 16);
            l[mt] += __shfl_xor(l[mt], 32);
            if (grp == 0) {
                sm.ml[kg][r0 + mt * 16][0] = m[mt];
                sm.ml[kg][r0 + mt * 16][1] = l[mt];
            }
        }
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float top = NEG_INF, sum = 0;
#pragma unroll
            for (int w = 0; w < S::KG; ++w) top = fmaxf(top, sm.ml[w][r0 + mt * 16][0]);
#pragma unroll
            for (int w = 0; w < S::KG; ++w)
                sum += sm.ml[w][r0 + mt * 16][1] * scale_to(sm.ml[w][r0 + mt * 16][0], top);
            const float f = scale_to(m[mt], top);
            m[mt] = top;
            l[mt] = sum;
#pragma unroll
            for (int n = 0; n < NTILE; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][n][e] *= f;
        }
        if constexpr (WIDE) {
            if (kg > 0) put(kg - 1);
            __syncthreads();
            if (kg == 0)
#pragma unroll 1
                for (int w = 0; w < S::KG - 1; ++w) take(w);
            return;
        }
        if (wave >= 2) put(wave - 2);
        __syncthreads();
        if (wave < 2) take(wave);
        __syncthreads();
        if (wave == 1) put(1);
        __syncthreads();
        if (wave == 0) {
            take(1);
            put(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                if (grp == 0) {
                    sm.ml[0][mt * 16 + col][0] = m[mt];
                    sm.ml[0][mt * 16 + col][1] = l[mt];
                }
        }
        __syncthreads();
    }
    // 2^(m - top), 1 where nothing has been seen
    static __device__ __forceinline__ float scale_to(float from, float top) {
        return top == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(from - top);
    }
    // Normalises four outputs of row r and writes them, and its lse.
    __device__ __forceinline__ void write_row(int sub, int r, int d, f32x4 x, float top,
                                              float sum) const {
        int32_t t, head;
        if (!row_of(sub, r, t, head)) return;
        const bool none = sum == 0.0f;  // (then x is NaN where V is no finite number)
        const float inv = 1.0f / sum;
        const int64_t at = ((int64_t)req * p.c.draft + t) * p.c.heads + head;
        u32x2 w;
        w[0] = none ? 0 : pack2<DT>(x[0] * inv, x[1] * inv);
        w[1] = none ? 0 : pack2<DT>(x[2] * inv, x[3] * inv);
        gstore((u32x2*)((char*)p.out + 2 * (at * D + d)), w);
        if (d == 0 && p.lse)
            gstore(p.lse + at, none ? NEG_INF
                                           : (top + SHIFT + log2f(sum * __builtin_exp2f(-SHIFT))) *
                                                 0.6931471805599453f);
    }
    // this lane's outputs 4 * i .. of row mt * 16 + col, and where they begin
    __device__ __forceinline__ f32x4 four(int mt, int i) const {
        f32x4 x;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = o[mt][(4 * i + j) % NTILE][(4 * i + j) / NTILE];
        return x;
    }
    __device__ __forceinline__ int four_at(int i) const { return grp * 4 * NTILE + 4 * i; }

    // A wave with a head of its own: joins the lanes' sums.
    __device__ __forceinline__ void close() {
        fresh();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            l[mt] += __shfl_xor(l[mt], 16);
            l[mt] += __shfl_xor(l[mt], 32);
        }
    }

    // Leaves a wave's rows in its registers (false: in another wave's).
    __device__ __forceinline__ bool own_rows() {
        if constexpr (HEAD)
            close();
        else
            join_waves();
        return kg == 0;
    }

    __device__ __forceinline__ void finish_whole() {
        if constexpr (HEAD || WIDE) {
            if (own_rows())
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < NTILE; ++i)
                        write_row(sub(), mt * 16 + col, four_at(i), four(mt, i), m[mt], l[mt]);
            if constexpr (WIDE) __syncthreads();
        } else {
            join_waves();
            for (int x = tid * 4; x < ROWS * D; x += T * 4) {
                const int r = x / D, d = x % D;
                write_row(0, r, d, *(const f32x4*)&sm.o[0][r][d], sm.ml[0][r][0], sm.ml[0][r][1]);
            }
            __syncthreads();
        }
    }

    // Whether parts are stored through to memory.  A release fence writes all of
    // the XCD's L2 back, about 4 us in which the joiner waits: one list of 4096
    // takes 14.8 us without it for 18, 16 of 1024 25 for 32.  Parts of many rows
    // lie in pieces of 16 bytes, which L2 gathers better: through memory 64 lists
    // of up to 16384 with 16 rows of four heads take 486 us for 456, 8 lists
    // with 128 rows 408 for 385.
    __device__ __forceinline__ bool through() const {
        return MODE == KEYS || (HEAD && MT == 1 && p.rows <= 8);
    }
    template <typename V>
    __device__ __forceinline__ void pstore(V* a, V v) const {
        if (!through()) {
            gstore(a, v);
            return;
        }
        uint32_t w[sizeof(V) / 4];
        __builtin_memcpy(w, &v, sizeof(V));
        if constexpr (sizeof(V) == 4) {
            __hip_atomic_store((VTS_GLOBAL uint32_t*)a, w[0], __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(V) / 8; ++i)
                __hip_atomic_store((VTS_GLOBAL uint64_t*)a + i,
                                   w[2 * i] | (uint64_t)w[2 * i + 1] << 32, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
    }

    // A share of the places: leaves the block's rows in slot `mine`; the
    // last of the workers [w0, w1] to arrive joins all, in their order.
    __device__ __forceinline__ void finish_part(int64_t mine, int32_t w0, int32_t w1,
                                                bool w0_whole_start) {
        float* po = p.part_o + mine * (ROWS * D);
        float* pm = p.part_ml + mine * (ROWS * 2);
        if constexpr (HEAD || WIDE) {
            if (own_rows())
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int r = mt * 16 + col, at = sub() * 16 * MT + r;
                    if (row_at(sub(), r) >= p.rows) continue;
#pragma unroll
                    for (int i = 0; i < NTILE; ++i)
                        pstore((f32x4*)(po + at * D + four_at(i)), four(mt, i));
                    if (grp == 0) {
                        pstore(pm + at * 2, m[mt]);
                        pstore(pm + at * 2 + 1, l[mt]);
                    }
                }
        } else {
            join_waves();
            for (int x = tid * 4; x < ROWS * D; x += T * 4)
                if (row_at(0, x / D) < p.rows)
                    pstore((f32x4*)(po + x), *(const f32x4*)&sm.o[0][x / D][x % D]);
            if (tid < ROWS * 2) pstore(pm + tid, (&sm.ml[0][0][0])[tid]);
        }
        // The parts are joined in blocks of JOIN workers, each by the block's last
        // to arrive, and the blocks by the last of those: with one joiner for
        // all, a list shared by hundreds of workgroups would wait for it.
        const int32_t blocks = (w1 - w0) / JOIN + 1, w = (int32_t)((mine >> 1) - (int64_t)mb * p.workers);
        const int32_t block = (w - w0) / JOIN, wb = w0 + block * JOIN;
        const int32_t members = w1 - wb + 1 < JOIN ? w1 - wb + 1 : JOIN;
        if (members == 1 || last_of(p.tickets + MAX_TICKETS + (int64_t)mb * p.workers + wb, members)) {
            if (blocks == 1 || members > 1)
                join_parts(wb, 1, members, w0, w0_whole_start, blocks == 1);
            if (blocks > 1 && last_of(p.tickets + (int64_t)mb * p.workers + w0, blocks))
                join_parts(w0, JOIN, blocks, w0, w0_whole_start, true);
        }
        __syncthreads();
    }

    // Whether this workgroup is the last of `n` to come here; the parts that the
    // others stored before are then visible.
    __device__ __forceinline__ bool last_of(uint32_t* ticket, int32_t n) {
        // every wave's stores are complete before the barrier: at the device's
        // scope where through(), else thread 0's release fence writes them back
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0);
        asm volatile("" ::: "memory");
        __syncthreads();
        if (tid == 0) {
            if (!through()) __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
            const uint32_t old = __hip_atomic_fetch_add((VTS_GLOBAL uint32_t*)ticket, 1u,
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const bool last = old + 1 == (uint32_t)n;
            if (last) {
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
                gstore(ticket, 0u);  // self-restoring
            }
            sm.last = last;
        }
        __syncthreads();
        return sm.last;
    }

    // Joins the parts of workers first, first + stride, ..: to the outputs, or
    // to the first one's slot.
    __device__ __forceinline__ void join_parts(int32_t first, int32_t stride, int32_t count,
                                               int32_t w0, bool w0_whole_start, bool to_outputs) {
        constexpr int FOURS = (ROWS * D + T * 4 - 1) / (T * 4);  // of elements, a thread
        if (FOURS > 2 && count <= 4)
            join_some<4, 4>(first, stride, count, w0, w0_whole_start, to_outputs);
        else
            join_some<1, 16>(first, stride, count, w0, w0_whole_start, to_outputs);
        if (to_outputs) return;
        const int64_t to = part(first, w0, w0_whole_start);
        __syncthreads();  // everyone has read the slot's maxima and sums
        if (tid < ROWS && row_at(tid / (16 * MT), tid % (16 * MT)) < p.rows) {
            pstore(p.part_ml + to * (ROWS * 2) + tid * 2, sm.ml[0][tid][0]);
            pstore(p.part_ml + to * (ROWS * 2) + tid * 2 + 1, sm.ml[0][tid][1]);
        }
    }

    // Other workgroups' parts come from beyond this XCD, so the loads of a
    // thread's X fours of U parts are issued together, the rows that hold nothing
    // are stepped over and the maximum is a running one: with the maxima in a
    // pass of their own and eight parts at a time, one list of 4096 in 32 parts
    // took 20 us for 18, one after the other 48; and with the empty rows read and
    // one four at a time, 64 lists of up to 16384 under drafts of two 473 us for
    // 456, 64 lists of 1024 under one token 63 for 61.
    template <int X, int U>
    __device__ __forceinline__ void join_some(int32_t first, int32_t stride, int32_t count,
                                              int32_t w0, bool w0_whole_start, bool to_outputs) {
        const int64_t to = part(first, w0, w0_whole_start);
        // rows that hold something: of each head, or the first ones
        const int valid = HEAD || p.rows - row_at(0, 0) < ROWS ? p.rows - row_at(0, 0) : ROWS;
        const int all = (HEAD ? S::SUBS * valid : valid) * D;
        for (int y = tid * 4; y < all; y += T * 4 * X) {
            int r[X], d[X];
            float top[X], sum[X];
            f32x4 acc[X];
#pragma unroll
            for (int j = 0; j < X; ++j) {
                const int at = y + j * T * 4 < all ? y + j * T * 4 : y;
                const int q = at / D, s = HEAD ? q / valid : 0;
                r[j] = HEAD ? s * 16 * MT + q - s * valid : q;
                d[j] = at % D;
                top[j] = NEG_INF;
                sum[j] = 0;
                acc[j] = f32x4{0, 0, 0, 0};
            }
#pragma unroll 1
            for (int32_t i = 0; i < count; i += U) {
                f32x4 o4[X][U];
                float mm[X][U], ll[X][U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int32_t w = first + (i + u < count ? i + u : count - 1) * stride;
                    const int64_t at = part(w, w0, w0_whole_start);
#pragma unroll
                    for (int j = 0; j < X; ++j) {
                        const u32x2 ml =
                            gload((const u32x2*)(p.part_ml + at * (ROWS * 2) + r[j] * 2));
                        o4[j][u] = gload((const f32x4*)(p.part_o + at * (ROWS * D) + r[j] * D + d[j]));
                        const uint32_t m0 = ml[0], l0 = ml[1];
                        mm[j][u] = __builtin_bit_cast(float, m0);
                        ll[j][u] = __builtin_bit_cast(float, l0);
                    }
                }
#pragma unroll
                for (int j = 0; j < X; ++j) {
                    float up = top[j];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        up = fmaxf(up, mm[j][u]);  // (the last one again past count)
                    const float f0 = scale_to(top[j], up);
                    sum[j] *= f0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[j][e] *= f0;
                    top[j] = up;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (i + u < count) {
                            const float f = scale_to(mm[j][u], top[j]);
                            sum[j] += f * ll[j][u];
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[j][e] += f * o4[j][u][e];
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < X; ++j) {
                if (y + j * T * 4 >= all) continue;
                if (to_outputs) {
                    write_row(r[j] / (16 * MT), r[j] % (16 * MT), d[j], acc[j], top[j], sum[j]);
                } else {
                    pstore((f32x4*)(p.part_o + to * (ROWS * D) + r[j] * D + d[j]), acc[j]);
                    if (d[j] == 0) {
                        sm.ml[0][r[j]][0] = top[j];
                        sm.ml[0][r[j]][1] = sum[j];
                    }
                }
            }
        }
    }

    // A worker's slot: its first segment's, or the one of a list that begins
    // inside its share.
    __device__ __forceinline__ int64_t part(int32_t w, int32_t w0, bool w0_whole_start) const {
        return 2 * ((int64_t)mb * p.workers + w) + (w == w0 && !w0_whole_start ? 1 : 0);
    }
};

template <int DT, int D, int MT, bool SLOTS, int MODE>
__global__ __launch_bounds__(threads_of(MODE), MODE >= WIDE2 ? 2 : 1) void attend_kernel(AttendParams p) {
    constexpr bool HEAD = MODE == HEADS;
    constexpr int PLACES = AttendShape<D, MT, MODE>::KG * 32;
    __shared__ AttendShared<D, MT, MODE> sm;
    // the row blocks of one share run next to each other on one XCD
    const int32_t per = 8 * p.row_blocks;
    const int32_t w = (int32_t)(blockIdx.x / per) * 8 + (int32_t)(blockIdx.x & 7);
    const int32_t mb = (int32_t)(blockIdx.x % per) >> 3;
    if (w >= p.workers) return;
    Share sh;
    if constexpr (SLOTS) {
        const int64_t each = (int64_t)units_of<PLACES>(place_count<true>(p, 0)) * head_units<HEAD>(p.c);
        sh.total = p.c.batch * p.c.draft * each;
        sh.workers = sh.total < p.workers ? (int32_t)sh.total : p.workers;
        if (w >= sh.workers) return;
        sh.begin = share_start(sh.total, sh.workers, w);
        sh.end = share_start(sh.total, sh.workers, w + 1);
        sh.b = (int32_t)(sh.begin / each);
        sh.b_unit = sh.b * each;
    } else {
        sh = dense_share<PLACES, HEAD>(p.c, p.workers, w);
        if (w >= sh.workers) return;
    }
    Attend<DT, D, MT, SLOTS, MODE> a(p, sm, mb);
    int64_t x = sh.begin;
    int32_t b = sh.b;
    int64_t b_unit = sh.b_unit;
    while (x < sh.end) {
        const int32_t units =
            units_of<PLACES>(SLOTS ? place_count<true>(p, 0) : uniform_len(p.c, b));
        const int32_t h = (int32_t)((x - b_unit) / units);
        const int64_t g0 = b_unit + (int64_t)h * units, g1 = g0 + units;
        const int64_t x1 = g1 < sh.end ? g1 : sh.end;
        a.begin(b, h);
        a.walk((int32_t)(x - g0), (int32_t)(x1 - g0));
        if (x == g0 && x1 == g1) {
            a.finish_whole();
        } else {
            const int32_t w0 = share_of(sh.total, sh.workers, g0);
            const int32_t w1 = share_of(sh.total, sh.workers, g1 - 1);
            const bool whole_start = share_start(sh.total, sh.workers, w0) == g0;
            a.finish_part(a.part(w, w0, whole_start), w0, w1, whole_start);
        }
        x = x1;
        if (h + 1 == head_units<HEAD>(p.c) && x1 == g1) {
            b_unit = g1;
            ++b;
        }
    }
}

template <int DT, int D, int MT, bool SLOTS, int MODE>
static hipError_t launch_one(const AttendParams& p, hipStream_t stream) {
    const uint32_t grid = (uint32_t)((p.workers + 7) / 8 * 8 * p.row_blocks);
    hipLaunchKernelGGL((attend_kernel<DT, D, MT, SLOTS, MODE>), dim3(grid),
                       dim3(threads_of(MODE)), 0, stream, p);
    return hipGetLastError();
}

template <int DT, int D, bool SLOTS>
static hipError_t launch_mode(const AttendParams& p, hipStream_t stream) {
    if constexpr (!SLOTS) {
        if (p.heads_on_waves)
            return p.rows <= 16 ? launch_one<DT, D, 1, SLOTS, HEADS>(p, stream)
                                : launch_one<DT, D, 2, SLOTS, HEADS>(p, stream);
    }
    switch (p.block_rows) {
        case 16: return launch_one<DT, D, 1, SLOTS, KEYS>(p, stream);
        case 32: return launch_one<DT, D, 2, SLOTS, KEYS>(p, stream);
        case 64: return launch_one<DT, D, 2, SLOTS, WIDE2>(p, stream);
    }
    return launch_one<DT, D, 2, SLOTS, WIDE4>(p, stream);
}

hipError_t launch_attend(int dtype, int head_dim, const AttendParams& p, hipStream_t stream) {
    if (dtype == BF16) {
        if (head_dim == 64)
            return p.slots ? launch_mode<BF16, 64, true>(p, stream)
                           : launch_mode<BF16, 64, false>(p, stream);
        return p.slots ? launch_mode<BF16, 128, true>(p, stream)
                       : launch_mode<BF16, 128, false>(p, stream);
    }
    if (head_dim == 64)
        return p.slots ? launch_mode<F16, 64, true>(p, stream)
                       : launch_mode<F16, 64, false>(p, stream);
    return p.slots ? launch_mode<F16, 128, true>(p, stream)
                   : launch_mode<F16, 128, false>(p, stream);
}

}  // namespace vts
