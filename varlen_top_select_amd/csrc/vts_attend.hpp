// vts_attend.hpp -- attention of drafted tokens over a paged KV cache.
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
//
// A microscaled cache (F 8 or 4 bits to an element, one power of two to 32 of them)
// is turned into 16-bit operands on the way: the conversion takes the scale along and
// every number of the format is one of bf16, and of fp16 within its range.  A wave
// keeps its K and V rows in LDS as they are stored.  K's elements are multiplied in
// an order of their own (lane group g takes the g-th quarter of a row in all steps),
// so that a lane's quarter is one LDS load and, at head size 128, one scale.
#pragma once

#include "vts_paged.hpp"

namespace vts {

// How a workgroup's waves share the work.
enum Mode : int {
    KEYS = 0,   // four waves, 32 places each of the same rows
    HEADS = 1,  // four waves, a KV head each at the same 32 places
    WIDE2 = 2,  // eight waves: two groups of 32 rows, four times 32 places
    WIDE4 = 4,  // eight waves: four groups of 32 rows, twice 32 places
};

// (over a microscaled cache wide workgroups have four waves, and two of them share a
// compute unit: eight that wait for each other have all their products at the same time)
constexpr int threads_of(int mode, int f) { return mode >= WIDE2 && f == 16 ? 512 : NT; }

template <int D, int MT, int MODE, int F>
struct AttendShape {
    static constexpr bool WIDE = MODE >= WIDE2;
    static constexpr int NW = threads_of(MODE, F) / 64;    // waves
    static constexpr int RG = WIDE ? MODE : 1;             // groups of rows
    static constexpr int KG = WIDE ? NW / RG : MODE == HEADS ? 1 : NW;  // groups of places
    static constexpr int PLACES = WIDE && F != 16 ? 64 : KG * 32;  // of a unit
    static constexpr int SUBS = MODE == HEADS ? NW : RG;   // blocks of 16 * MT rows
    static constexpr int ROWS = SUBS * 16 * MT;
    // a cache row in memory
    static constexpr int RB = D * F / 8;    // bytes
    static constexpr int CHF = RB / 16;     // 16-byte chunks
    // a wave's microscaled rows in LDS, padded: the four lane groups of a V load
    // take their part of rows 4 apart from banks of their own
    static constexpr int PAD = RB + (RB == 128 ? 32 : 16);
};

// A wide workgroup's places, K as operands (swizzled) and V in whole rows.
template <int D, int PLACES>
struct WideTiles {
    u32x4 k[2][PLACES * (D / 8)], v[2][PLACES * (D / 8)];
    uint8_t there[2][PLACES];
};

template <int D, int MT, int MODE, int F>
struct AttendShared : AttendShape<D, MT, MODE, F> {
    using S = AttendShape<D, MT, MODE, F>;
    // query rows as operands, from 32 rows on
    u32x4 q[MT > 1 && !(S::WIDE && F != 16) ? S::SUBS * MT * (D / 32) : 1][64];
    union {
        // a wave's K rows on their way from the order of whole rows to operands
        u32x4 k[S::WIDE || F != 16 ? 1 : WAVES][S::WIDE || F != 16 ? 1 : 32 * (D / 8)];
        // the same of a microscaled cache, K and V
        u32x4 packed[S::WIDE || F == 16 ? 1 : WAVES][S::WIDE || F == 16 ? 1 : 2 * 32 * S::PAD / 16];
        WideTiles<D, S::WIDE ? S::PLACES : 1> w;
        // outputs of waves to be joined, padded: the 16 rows of a store fall on all banks
        float o[MODE == HEADS || S::KG == 1 ? 1 : S::WIDE ? S::KG - 1 : 2][MODE == HEADS ? 1 : S::ROWS][D + 4];
    };
    // 16 rows of a wave on their way to whole rows of a part (waves do not wait for each
    // other, so it is no wave's tile; from 32 rows on, where its query rows were)
    f32x4 turn[F != 16 && MODE == HEADS && MT == 1 ? WAVES : 1][16 * D / 4];
    float ml[S::KG][S::ROWS][2];
    uint32_t last;
};

template <int DT, int D, int MT, bool SLOTS, int MODE, int F>
struct Attend {
    static constexpr int KS = D / 32;       // steps of the first product
    static constexpr int VB = D / 16 * 2;   // bytes of a V row per lane
    static constexpr int VW = VB / 4;       // words of a V row per lane
    static constexpr int NTILE = D / 16;    // 16-row tiles of the second product
    static constexpr int JOIN = 32;         // parts joined by one workgroup
    using S = AttendShape<D, MT, MODE, F>;
    static constexpr bool MICRO = F != 16;
    // a lane multiplies the elements of its quarter of a row, and not its eight of each 32
    static constexpr bool PERMUTED = MICRO && !S::WIDE;
    // A wide workgroup over a microscaled cache: a wave's 32 rows are one block of the 32x32x16
    // product.  It takes two thirds of the LDS loads that two blocks of the 16x16x32 one take,
    // and two workgroups of four waves to a compute unit have products and softmax at the
    // same time (8 trees of 16 up to 65536: 280 us for 433).
    static constexpr bool BLOCK = MICRO && S::WIDE;
    static constexpr int KB = D / 16, OB = D / 32;  // steps and tiles of its products
    static constexpr int PB = BLOCK ? S::PLACES / 32 / S::KG : 1;  // 32 places of a wave in a unit
    static constexpr bool HEAD = MODE == HEADS, WIDE = S::WIDE;
    static constexpr int T = S::NW * 64;    // threads
    // whether a cache row is read once by the whole call, as far as it is known
    // (the slots of two rows may be the same): such loads leave the caches alone.
    // 128 lists of 2048 slots, 64 heads: 112 us without, 104 with.  (Microscaled rows
    // that are no whole cache line share one with another head's.)
    static constexpr bool ONCE = (HEAD || (SLOTS && !WIDE)) && S::RB >= 128;
    static constexpr int ROWS = S::ROWS;
    // of m, see above: how far below the maximum it is put, and when it is raised
    static constexpr float SHIFT = DT == F16 ? 11 : 0, RAISE = DT == F16 ? 15 : 8;
    using VRow = typename std::conditional<D == 128, u32x4, u32x2>::type;

    const AttendParams& p;
    AttendShared<D, MT, MODE, F>& sm;
    int tid, lane, wave, col, grp;
    int bcol, half;  // (BLOCK) the lane's row, and its half of a product's places
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
    // Microscaled: a wave's loads of each of K and V, or (wide) a thread's chunks of both
    static constexpr int CHF = S::CHF, RB = S::RB, PAD = S::PAD;
    static constexpr int BLOCKS = D / 32;  // scales of a row
    static constexpr int HALF = S::PLACES * CHF;  // (wide) chunks of K in a unit, and of V
    static constexpr int LOADSF = !WIDE ? CHF / 2 : HALF >= T ? 2 * HALF / T : 1;
    // Microscaled tiles (wide: units) on their way, as many as the registers hold beside
    // two waves of a SIMD: with one of 4 KB a wave waits for memory most of the time (64
    // requests up to 16384 over a 4-bit cache 224 us with one and 187 with two).
    static constexpr int AHEAD = !MICRO          ? 1
                                 : WIDE          ? (D == 64 || F == 4 ? 2 : 1)
                                 : D == 64       ? 3
                                 : MT > 1        ? 1
                                 : F == 4        ? 2
                                 : HEAD && SLOTS ? 1
                                                 : 2;
    using Scales = typename std::conditional<D == 128, uint32_t, uint16_t>::type;
    u32x4 q[BLOCK ? KB : QL ? 1 : KS];
    uint64_t bits[MT];
    f32x4 o[BLOCK ? 1 : MT][NTILE];
    float m[MT], l[MT];
    f32x16 ob[BLOCK ? OB : 1];
    // the tile on its way: 32 places to a wave, or the wave's rows of the unit
    u32x4 k[MICRO ? LOADSF * AHEAD : WIDE ? LOADS : 2 * KS];
    VRow v[8];
    u32x4 vw[MICRO ? LOADSF * AHEAD : LOADS];
    const void* kbase;
    const void* vbase;
    // Microscaled: the scales on their way (K's of place l in lane l, V's in lane
    // 32 + l; wide: of the thread's chunks) and of the tile at hand
    uint32_t sc_next[WIDE ? LOADSF * AHEAD : AHEAD], sc;
    bool here[WIDE ? LOADSF * AHEAD : 1];  // (wide) whether the chunks' places are there
    // of the scales: K's in lanes 0..31, V's above
    const char* sbase;
    uint32_t scale_page, scale_pos;
    bool cleared;  // something that is not finite was taken out of a tile's V
    // Which of the lane's probabilities are 0 or NaN, of the last tiles that hold drafted
    // tokens, eight bits to a tile and the last one's low (three hold 64 tokens)
    uint32_t none[MT];

    __device__ Attend(const AttendParams& p_, AttendShared<D, MT, MODE, F>& s_, int32_t mb_)
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
        bcol = lane & 31;
        half = lane >> 5;
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
        if constexpr (MICRO && !WIDE) {
            const ScaleView& s = lane < 32 ? p.k_scale : p.v_scale;
            sbase = (const char*)s.base + (uint64_t)h * s.head_stride * BLOCKS;
        }
        if constexpr (BLOCK) {
            begin_block();
            return;
        }
#pragma unroll
        for (int mt = 0; mt < (BLOCK ? 0 : MT); ++mt) {
            int32_t t, head;
            const bool ok = row_of(sub(), mt * 16 + col, t, head);
            const char* at = (const char*)p.q +
                             2 * (req * p.q_batch + (ok ? t * p.q_row + head * p.q_head : 0));
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                u32x4 x = {0, 0, 0, 0};
                if (QL && !HEAD && (mt * KS + s) % S::KG != kg) continue;
                if (ok) x = gload((const u32x4*)(at + (PERMUTED ? (grp * KS + s) * 16 : s * 64 + grp * 16)));
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
    __device__ __forceinline__ void begin_block() {
        int32_t t, head;
        const bool ok = row_of(sub(), bcol, t, head);
        const char* at = (const char*)p.q + 2 * (req * p.q_batch + (ok ? t * p.q_row + head * p.q_head : 0));
#pragma unroll
        for (int s = 0; s < KB; ++s) {
            u32x4 x = {0, 0, 0, 0};
            if (ok) x = gload((const u32x4*)at + s * 2 + half);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] ^= p.q_sign;
            q[s] = x;
        }
        bits[0] = !ok           ? 0
                  : p.tree_mask ? (uint64_t)gload(p.tree_mask + (int64_t)req * p.c.draft + t)
                  : t >= 63     ? ~0ull
                                : (2ull << t) - 1;
        m[0] = NEG_INF;
        l[0] = 0;
#pragma unroll
        for (int i = 0; i < OB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) ob[i][e] = 0;
        cleared = false;
    }
    __device__ __forceinline__ int q_at(int mt, int s) const {
        return (sub() * MT + mt) * KS + s;
    }

    __device__ __forceinline__ int32_t first_place(int32_t u) const {
        return BLOCK ? u * S::PLACES + kg * 32 : (u * S::KG + kg) * 32;
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
    // ---- a microscaled cache

    // eight numbers of the format with their scale's power of two, as an operand
    static __device__ __forceinline__ u32x4 widen(uint32_t lo, uint32_t hi, float scale) {
        u32x4 x;
        if constexpr (F == 4) {
            x[0] = widen4<DT, 0>(lo, scale);
            x[1] = widen4<DT, 1>(lo, scale);
            x[2] = widen4<DT, 2>(lo, scale);
            x[3] = widen4<DT, 3>(lo, scale);
        } else {
            x[0] = widen8<DT, false>(lo, scale);
            x[1] = widen8<DT, true>(lo, scale);
            x[2] = widen8<DT, false>(hi, scale);
            x[3] = widen8<DT, true>(hi, scale);
        }
        return x;
    }
    // scale number i of a row's
    static __device__ __forceinline__ float scale_at(uint32_t scales, int i) {
        return scale_of((scales >> (8 * i)) & 0xFFu);
    }
    // The rows of a wave's tile, as they lie in memory, and their scales: K's of
    // place l in lane l, V's in lane 32 + l, one load for both.
    // Returns whether the lane's place is there.
    __device__ __forceinline__ bool load_micro(int to, const Lookup& e) {
        const Spot at = resolve_lookup<SLOTS>(p.c, e);
        const uint32_t off = spot_offset(at, page_stride, pos_stride);
#pragma unroll
        for (int i = 0; i < LOADSF; ++i) {
            const int r = i * (64 / CHF) + lane / CHF;
            k[to * LOADSF + i] = row_load<u32x4, ONCE>(kbase, from_lane(off, r), (lane % CHF) * 16);
            vw[to * LOADSF + i] = row_load<u32x4, ONCE>(vbase, from_lane(off, 32 + r), (lane % CHF) * 16);
        }
        sc_next[to] = *(const VTS_GLOBAL Scales*)((const VTS_GLOBAL char*)sbase +
                                                  (uint64_t)spot_offset(at, scale_page, scale_pos) * BLOCKS);
        return at.there;
    }
    __device__ __forceinline__ char* packed_row(int which, int r) const {
        return (char*)sm.packed[wave] + (which * 32 + r) * PAD;
    }
    __device__ __forceinline__ void stage_micro(int from) {
#pragma unroll
        for (int i = 0; i < LOADSF; ++i) {
            const int r = i * (64 / CHF) + lane / CHF;
            *(u32x4*)(packed_row(0, r) + (lane % CHF) * 16) = k[from * LOADSF + i];
            *(u32x4*)(packed_row(1, r) + (lane % CHF) * 16) = vw[from * LOADSF + i];
        }
        sc = sc_next[from];
        // the wave's own stores come before its loads; the compiler has to know
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    // K row h * 16 + col, the lane's quarter, as the operands of all steps
    __device__ __forceinline__ void micro_k(int h, u32x4 (&x)[KS]) const {
        constexpr int WORDS = RB / 16;  // of a quarter
        uint32_t w[WORDS];
        __builtin_memcpy(w, __builtin_assume_aligned(packed_row(0, h * 16 + col) + grp * (RB / 4), RB / 4 < 16 ? RB / 4 : 16), RB / 4);
        const float scale = scale_at(from_lane(sc, h * 16 + col), D == 128 ? grp : grp >> 1);
#pragma unroll
        for (int s = 0; s < KS; ++s)
            x[s] = F == 4 ? widen(w[s], 0, scale) : widen(w[(2 * s) % WORDS], w[(2 * s + 1) % WORDS], scale);
    }
    // second_product over V as it is stored: word by word of the lane's elements, so that
    // few converted ones are held at a time.
    __device__ __forceinline__ void micro_product(uint32_t have, bool masked, bool drafted,
                                                  const u32x4 (&pv)[MT]) {
        constexpr int B = RB / 16;  // bytes of the lane's part of a row
        uint32_t raw[8][B == 8 ? 2 : 1];
        float scale[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const char* at = packed_row(1, v_place(j)) + col * B;
            if constexpr (B == 2)
                raw[j][0] = *(const uint16_t*)at;
            else
                __builtin_memcpy(raw[j], __builtin_assume_aligned(at, B), B);
            scale[j] = scale_at(from_lane(sc, 32 + v_place(j)), col / (16 / BLOCKS));
        }
        if (masked) {
            int g = grp;
            asm volatile("" : "+v"(g));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t there = (have >> ((j >> 2) * 16 + g * 4 + (j & 3))) & 1u;
#pragma unroll
                for (int w = 0; w < (B == 8 ? 2 : 1); ++w) raw[j][w] = there ? raw[j][w] : 0;
                scale[j] = there ? scale[j] : 1.0f;
            }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            uint32_t x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (F == 4)
                    x[j] = w == 0   ? widen4<DT, 0>(raw[j][0], scale[j])
                           : w == 1 ? widen4<DT, 1>(raw[j][0], scale[j])
                           : w == 2 ? widen4<DT, 2>(raw[j][0], scale[j])
                                    : widen4<DT, 3>(raw[j][0], scale[j]);
                else
                    x[j] = w & 1 ? widen8<DT, true>(raw[j][w / 2], scale[j])
                                 : widen8<DT, false>(raw[j][w / 2], scale[j]);
            }
            if (drafted) {  // see clear_not_finite
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (ballot(not_finite<DT>(x[j])) == 0) continue;
                    cleared = true;
                    if (not_finite<DT>(x[j] & 0xFFFFu)) x[j] &= 0xFFFF0000u;
                    if (not_finite<DT>(x[j] >> 16)) x[j] &= 0xFFFFu;
                }
            }
            u32x4 lo, hi;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x05040100u);
                hi[j] = __builtin_amdgcn_perm(x[2 * j + 1], x[2 * j], 0x07060302u);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                o[mt][2 * w] = mfma<DT>(lo, pv[mt], o[mt][2 * w]);
                o[mt][2 * w + 1] = mfma<DT>(hi, pv[mt], o[mt][2 * w + 1]);
            }
        }
    }
    // weightless of a tile's eight, as bits
    static __device__ __forceinline__ uint32_t weightless_of(u32x4 pv) {
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) x |= weightless<DT>(e & 1 ? pv[e / 2] >> 16 : pv[e / 2] & 0xFFFFu) << e;
        return x;
    }
    // (BLOCK) The same of 32 places of a unit, sixteen bits, their scores computed again: the K
    // rows of the walk's last two units, which hold all drafted tokens, are still in LDS.
    __device__ __forceinline__ uint32_t weightless_block(int32_t u, int b) const {
        f32x16 s;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0;
        const int r = (kg + b) * 32 + bcol;
#pragma unroll
        for (int ks = 0; ks < KB; ++ks)
            s = mfma32<DT>(sm.w.k[u & 1][r * CH + ((2 * ks + half) ^ swizzled<D>(r))], q[ks], s);
        const float base = m[0] == NEG_INF ? 0.0f : m[0];
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x |= weightless<DT>(pack2<DT>(__builtin_amdgcn_exp2f(fmaf(s[e], p.scale_log2e, -base)), 0.0f) & 0xFFFFu) << e;
        return x;
    }
    // What was cleared of V in the wave's tiles of units [u0, u1), from memory to the rows that
    // see it (all of them, where it is of the prefix or the list, whose end such a tile holds):
    // rare, and apart from the walk, whose registers it would take.  Each wave adds what its
    // own places hold, for in the join its outputs meet those of waves that saw more or less
    // of a row (0 * inf).  An infinity of any weight is the infinity; of none (a score of
    // -inf) it is NaN, as the products of other tiles give it.
    __device__ __forceinline__ void add_cleared(int32_t u0, int32_t u1) {
        fresh();
        constexpr int SPAN = BLOCK ? PB * 32 : 32;
        uint32_t of_block = 0;
#pragma unroll 1
        for (int32_t u = u0; u < u1; ++u) {
            const int32_t j0 = first_place(u);
            // (a wide unit is cleared as a whole)
            if ((BLOCK ? u * S::PLACES + S::PLACES : j0 + SPAN) <= pl.first) continue;
#pragma unroll 1
            for (int kk = 0; kk < SPAN; ++kk) {
                if constexpr (BLOCK)
                    if ((kk & 31) == 0) of_block = weightless_block(u, kk >> 5);
                const int32_t i = j0 + kk - pl.first;
                const Spot at = resolve_lookup<SLOTS>(p.c, issue_lookup<SLOTS>(p.c, pl, j0 + kk));
                if (!at.there) continue;
                const uint32_t off = spot_offset(at, p.c.v.page_stride, p.c.v.pos_stride);
                const uint32_t soff = spot_offset(at, p.v_scale.page_stride, p.v_scale.pos_stride);
                const int32_t h = HEAD ? head_unit * WAVES + wave : head_unit;
                const uint8_t* codes = p.v_scale.base + ((uint64_t)soff + (uint64_t)h * p.v_scale.head_stride) * BLOCKS;
                const VTS_GLOBAL char* row = (const VTS_GLOBAL char*)vbase + ((uint64_t)off << 4);
                if constexpr (BLOCK) {
                    const uint32_t n = from_lane(of_block, (kk >> 2 & 1) * 32 + bcol);
                    add_to_block(codes, row, i, n >> ((kk >> 3 & 3) * 4 + (kk & 3)) & 1);
                    continue;
                }
                const int src = ((kk & 15) >> 2) * 16 + col, bit = 8 * (u1 - 1 - u) + (kk >> 4) * 4 + (kk & 3);
                uint32_t weighs_nothing[MT];
#pragma unroll
                for (int mt = 0; mt < (BLOCK ? 0 : MT); ++mt) weighs_nothing[mt] = from_lane(none[mt], src) >> bit & 1;
#pragma unroll
                for (int e4 = 0; e4 < (BLOCK ? 0 : 4); ++e4) {
                    constexpr int B = RB / 16;
                    const int part = grp * 4 + e4;
                    const float scale = scale_of(gload(codes + part / (16 / BLOCKS)));
                    uint32_t w[2] = {0, 0};
                    const VTS_GLOBAL char* x4 = row + part * B;
                    if constexpr (B == 2) {
                        w[0] = *(const VTS_GLOBAL uint16_t*)x4;
                    } else {
                        w[0] = *(const VTS_GLOBAL uint32_t*)x4;
                        if constexpr (B == 8) w[1] = *(const VTS_GLOBAL uint32_t*)(x4 + 4);
                    }
                    const u32x4 x = widen(w[0], w[1], scale);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const bool see = i < 0 || ((bits[mt] >> (i & 63)) & 1);
#pragma unroll
                        for (int n = 0; n < NTILE; ++n) {
                            const uint32_t half = (x[n >> 1] >> (16 * (n & 1))) & 0xFFFFu;
                            const float y = o[mt][n][e4] + (weighs_nothing[mt] ? NOT_A_NUMBER : to_float<DT>(half));
                            o[mt][n][e4] = see && not_finite<DT>(half) ? y : o[mt][n][e4];
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    }
    // The same of one place's row (place < 0: of the prefix or the list), to the lane's elements
    // 32 i + 8 n + 4 half ..
    __device__ __forceinline__ void add_to_block(const uint8_t* codes, const VTS_GLOBAL char* row, int32_t place,
                                                 bool weighs_nothing) {
        const bool see = place < 0 || ((bits[0] >> (place & 63)) & 1);
#pragma unroll
        for (int i = 0; i < OB; ++i) {
            const float scale = scale_of(gload(codes + i));
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const VTS_GLOBAL char* at = row + (32 * i + 8 * n + 4 * half) * F / 8;
                u32x4 x;
                if constexpr (F == 4)
                    x = widen(*(const VTS_GLOBAL uint16_t*)at, 0, scale);
                else
                    x = widen(*(const VTS_GLOBAL uint32_t*)at, 0, scale);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t one = (x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                    const float y = ob[i][4 * n + e] + (weighs_nothing ? NOT_A_NUMBER : to_float<DT>(one));
                    ob[i][4 * n + e] = see && not_finite<DT>(one) ? y : ob[i][4 * n + e];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    // A wave's 32 rows and its places of a unit, 32 or all 64: as tile(), in blocks.
    __device__ __forceinline__ void tile_block(const uint32_t (&have)[PB], bool masked, int32_t j0, int buf) {
        const float c = p.scale_log2e;
        f32x16 s[PB];
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = 0;
#pragma unroll
        for (int ks = 0; ks < KB; ++ks)
#pragma unroll
            for (int b = 0; b < PB; ++b) {
                const int r = (kg + b) * 32 + bcol;
                s[b] = mfma32<DT>(sm.w.k[buf][r * CH + ((2 * ks + half) ^ swizzled<D>(r))], q[ks], s[b]);
            }
        if (masked) {
            int h = half;  // opaque: nothing of this is kept in registers between tiles
            asm volatile("" : "+v"(h));
#pragma unroll
            for (int b = 0; b < PB; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int kk = key_of(e) + 4 * h;
                    const int32_t i = j0 + b * 32 + kk - pl.first;
                    const uint32_t see =
                        (have[b] >> kk) & (((uint32_t)i >> 31) | (uint32_t)(bits[0] >> (i & 63)));
                    s[b][e] = (see & 1u) ? s[b][e] : NEG_INF;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
        top *= c;
        if (ballot(top > m[0] + RAISE)) {
            float up = fmaxf(top, __shfl_xor(top, 32));
            up = up > m[0] + RAISE ? up - SHIFT : m[0];
            const float f = up == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(m[0] - up);
            m[0] = up;
            l[0] *= f;
#pragma unroll
            for (int i = 0; i < OB; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) ob[i][e] *= f;
        }
        const float base = m[0] == NEG_INF ? 0.0f : m[0];
        u32x4 pv[2 * PB];
#pragma unroll
        for (int b = 0; b < PB; ++b)
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[b][e], c, -base));
                const float y = __builtin_amdgcn_exp2f(fmaf(s[b][e + 1], c, -base));
                l[0] += x + y;
                pv[2 * b + (e >> 3)][(e >> 1) & 3] = pack2<DT>(x, y);
            }
#pragma unroll
        for (int step = 0; step < 2 * PB; ++step)
#pragma unroll
            for (int i = 0; i < OB; ++i)
                ob[i] = mfma32<DT>(turned_v<D>(sm.w.v[buf], lane, kg * 32 + 16 * step, i), pv[step], ob[i]);
    }
    // Wide: the thread's chunks of a unit.  PAIRS of the same place and number of K and of V,
    // or, where the unit's K has fewer chunks than there are threads, one of K or of V.
    static constexpr int PAIRS = HALF >= T ? HALF / T : 0;
    __device__ __forceinline__ int place_of(int i) const { return (i * T + tid) % HALF / CHF; }
    __device__ __forceinline__ bool thread_v() const { return PAIRS == 0 && tid >= HALF; }
    __device__ __forceinline__ void load_chunk(int to, const Spot& at, bool is_v) {
        const CacheView& view = is_v ? p.c.v : p.c.k;
        const ScaleView& s = is_v ? p.v_scale : p.k_scale;
        const int chunk = tid % CHF;
        here[to] = at.there;
        k[to] = row_load<u32x4>(is_v ? vbase : kbase, spot_offset(at, view.page_stride, view.pos_stride), chunk * 16);
        sc_next[to] = ((const VTS_GLOBAL uint8_t*)s.base)
            [((uint64_t)spot_offset(at, s.page_stride, s.pos_stride) + (uint64_t)head_unit * s.head_stride) * BLOCKS +
             chunk * BLOCKS / CHF];
    }
    static_assert(!BLOCK || (T % CHF == 0 && (PAIRS == 0 ? 2 * HALF == T : HALF % T == 0)), "chunks of a thread");
    static constexpr int LOOKUPS = PAIRS ? PAIRS : 1;  // places of a thread's chunks
    __device__ __forceinline__ void issue_wide(Lookup (&e)[LOOKUPS], int32_t u) const {
#pragma unroll
        for (int i = 0; i < LOOKUPS; ++i)
            e[i] = issue_lookup<SLOTS>(p.c, pl, u * S::PLACES + place_of(i));
    }
    __device__ __forceinline__ void load_wide_micro(int to, const Lookup (&e)[LOOKUPS]) {
#pragma unroll
        for (int i = 0; i < LOOKUPS; ++i) {
            const Spot at = resolve_lookup<SLOTS>(p.c, e[i]);
            if constexpr (PAIRS) {
                load_chunk(to * LOADSF + 2 * i, at, false);
                load_chunk(to * LOADSF + 2 * i + 1, at, true);
            } else {
                load_chunk(to, at, thread_v());
            }
        }
    }
    // clear: some rows of the unit do not see some places; what is not finite in V goes to
    // them by add_cleared
    __device__ __forceinline__ void stage_wide_micro(int from, int buf, bool clear) {
        constexpr int OUT = CH / CHF;  // 16-byte chunks of operands from one
#pragma unroll
        for (int i = 0; i < LOADSF; ++i) {
            const bool is_v = PAIRS ? i & 1 : thread_v();
            const int r = place_of(PAIRS ? i / 2 : 0), chunk = tid % CHF;
            const float scale = scale_of(sc_next[from * LOADSF + i]);
#pragma unroll
            for (int e = 0; e < OUT; ++e) {
                u32x4 y = F == 4 ? widen(k[from * LOADSF + i][e % 4], 0, scale)
                                 : widen(k[from * LOADSF + i][2 * e % 4], k[from * LOADSF + i][(2 * e + 1) % 4], scale);
                const int c = chunk * OUT + e;
                if (is_v) {
                    const u32x4 z = {0, 0, 0, 0};
                    if (!here[from * LOADSF + i]) y = z;
                    if (clear) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            cleared = cleared || not_finite<DT>(y[x]);
                            y[x] = finite_part<DT>(y[x]);
                        }
                    }
                    sm.w.v[buf][v_chunk<D>(r, c)] = y;
                } else {
                    sm.w.k[buf][r * CH + (c ^ swizzled<D>(r))] = y;
                }
            }
            if (!is_v && chunk == 0) sm.w.there[buf][r] = here[from * LOADSF + i];
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
            for (int e = 0; e < 4; ++e) {
                if constexpr (WIDE)
                    x[e] = wide_v(buf, kk, grp * 4 + e);
                else
                    x[e] = row_load<VRow>(vbase, r, (grp * 4 + e) * VB);
            }
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
        if constexpr (!MICRO && !WIDE) {
            stage_k();
            if (more) load_k(off_next);
        }
        f32x4 s[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) s[mt][h] = f32x4{0, 0, 0, 0};
        if constexpr (PERMUTED) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 kx[KS];
                micro_k(h, kx);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        s[mt][h] = mfma<DT>(kx[ks], QL ? sm.q[q_at(mt, ks)][lane] : q[QL ? 0 : ks], s[mt][h]);
            }
        }
        // step by step over all rows, so that independent products stand between
        // dependent ones
#pragma unroll
        for (int ks = 0; ks < (PERMUTED ? 0 : KS); ++ks) {
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
        if constexpr (PERMUTED) {
            if (drafted) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) none[mt] = none[mt] << 8 | weightless_of(pv[mt]);
            }
            micro_product(have, masked, drafted, pv);
        } else if (masked) {
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
        if constexpr (!PERMUTED) second_product(pv);
        if constexpr (!PERMUTED)
            if (bad) add_rows(bad, off, j0, buf, pv);
        if constexpr (!WIDE) {
            if constexpr (!MICRO)
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
        if constexpr (MICRO) {
            if constexpr (WIDE)
                walk_wide_micro(u0, u1);
            else
                walk_micro(u0, u1);
            return;
        }
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
    // The same over a microscaled cache, AHEAD tiles on their way.
    __device__ __forceinline__ void walk_micro(int32_t u0, int32_t u1) {
        cleared = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) none[mt] = 0;
        scale_page = lane < 32 ? p.k_scale.page_stride : p.v_scale.page_stride;
        scale_pos = lane < 32 ? p.k_scale.pos_stride : p.v_scale.pos_stride;
        const auto look = [&](int32_t u) { return issue_lookup<SLOTS>(p.c, pl, first_place(u) + (lane & 31)); };
        bool there[AHEAD];
        Lookup e[AHEAD + 1];
#pragma unroll
        for (int i = 0; i <= AHEAD; ++i) e[i] = look(u0 + i);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) there[i] = load_micro(i, e[i]);
        Lookup next = e[AHEAD];
#pragma unroll 1
        for (int32_t u = u0; u < u1; u += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (u + i >= u1) break;
                const int32_t j0 = first_place(u + i);
                const uint32_t have = (uint32_t)ballot(there[i]);
                stage_micro(i);
                const Lookup now = next;
                // (before the rows: waiting for it waits for all loads before it)
                next = look(u + i + AHEAD + 1);
                there[i] = load_micro(i, now);
                tile(have, j0 + 31 >= pl.first, 0, j0, false, 0, 0);
            }
        }
        if (cleared) add_cleared(u0, u1);
    }
    // A wide workgroup's.
    __device__ __forceinline__ void walk_wide_micro(int32_t u0, int32_t u1) {
        Lookup e[AHEAD + 1][LOOKUPS];
#pragma unroll
        for (int i = 0; i <= AHEAD; ++i) issue_wide(e[i], u0 + i);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load_wide_micro(i, e[i]);
        Lookup next[LOOKUPS];
#pragma unroll
        for (int i = 0; i < LOOKUPS; ++i) next[i] = e[AHEAD][i];
#pragma unroll 1
        for (int32_t u2 = u0; u2 < u1; u2 += AHEAD) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int32_t u = u2 + i;
                if (u >= u1) break;
                const int32_t j0 = first_place(u);
                const int buf = u & 1;
                stage_wide_micro(i, buf, (u + 1) * S::PLACES > pl.first);
                Lookup now[LOOKUPS];
#pragma unroll
                for (int x = 0; x < LOOKUPS; ++x) now[x] = next[x];
                issue_wide(next, u + AHEAD + 1);  // (before the rows, as in walk_micro)
                load_wide_micro(i, now);
                __syncthreads();
                uint32_t have[PB];
                bool masked = j0 + PB * 32 > pl.first;
#pragma unroll
                for (int b = 0; b < PB; ++b) {
                    have[b] = (uint32_t)ballot(sm.w.there[buf][(kg + b) * 32 + (lane & 31)]);
                    masked = masked || have[b] != ~0u;
                }
                tile_block(have, masked, j0, buf);
            }
        }
        if (u1 * S::PLACES > pl.first) {  // (the same in all waves)
            if (tid == 0) sm.last = 0;
            __syncthreads();
            if (cleared) sm.last = 1;
            __syncthreads();
            if (sm.last) add_cleared(u0, u1);
            __syncthreads();
        }
    }

    // (BLOCK) the lane's outputs, four by four, and where they begin
    static constexpr int NFOUR = BLOCK ? 4 * OB : 0;
    __device__ __forceinline__ f32x4 block_four(int i) const {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ob[i / 4][4 * (i % 4) + e];
        return x;
    }
    __device__ __forceinline__ int block_at(int i) const { return 32 * (i / 4) + 8 * (i % 4) + 4 * half; }
    // the same of waves of different places: left in the registers of the first group's
    __device__ __forceinline__ void join_blocks() {
        fresh();
        l[0] += __shfl_xor(l[0], 32);
        const int r = rg * 32 + bcol;
        if (half == 0) {
            sm.ml[kg][r][0] = m[0];
            sm.ml[kg][r][1] = l[0];
        }
        __syncthreads();
        float top = NEG_INF, sum = 0;
#pragma unroll
        for (int w = 0; w < S::KG; ++w) top = fmaxf(top, sm.ml[w][r][0]);
#pragma unroll
        for (int w = 0; w < S::KG; ++w) sum += sm.ml[w][r][1] * scale_to(sm.ml[w][r][0], top);
        const float f = scale_to(m[0], top);
        m[0] = top;
        l[0] = sum;
#pragma unroll
        for (int i = 0; i < OB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) ob[i][e] *= f;
        if (kg > 0) put(kg - 1);
        __syncthreads();
        if (kg == 0)
#pragma unroll 1
            for (int w = 0; w < S::KG - 1; ++w) take(w);
    }

    // o[.] += the rows that another wave left in LDS
    __device__ __forceinline__ void put(int slot) {
        if constexpr (BLOCK) {
#pragma unroll
            for (int i = 0; i < NFOUR; ++i)
                *(f32x4*)&sm.o[slot][rg * 32 + bcol][block_at(i)] = block_four(i);
            return;
        }
#pragma unroll
        for (int mt = 0; mt < (BLOCK ? 0 : MT); ++mt)
#pragma unroll
            for (int n = 0; n < NTILE; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sm.o[slot][rg * 16 * MT + mt * 16 + col][(grp * 4 + e) * NTILE + n] = o[mt][n][e];
    }
    __device__ __forceinline__ void take(int slot) {
        if constexpr (BLOCK) {
#pragma unroll
            for (int i = 0; i < NFOUR; ++i) {
                const f32x4 x = *(const f32x4*)&sm.o[slot][rg * 32 + bcol][block_at(i)];
#pragma unroll
                for (int e = 0; e < 4; ++e) ob[i / 4][4 * (i % 4) + e] += x[e];
            }
            return;
        }
#pragma unroll
        for (int mt = 0; mt < (BLOCK ? 0 : MT); ++mt)
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
        if constexpr (BLOCK) {
            join_blocks();
            return;
        }
        fresh();
        const int r0 = rg * 16 * MT + col;
#pragma unroll
        for (int mt = 0; mt < (BLOCK ? 0 : MT); ++mt) {
            l[mt] += __shfl_xor(l[mt], 16);
            l[mt] += __shfl_xor(l[mt], 32);
            if (grp == 0) {
                sm.ml[kg][r0 + mt * 16][0] = m[mt];
                sm.ml[kg][r0 + mt * 16][1] = l[mt];
            }
        }
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < (BLOCK ? 0 : MT); ++mt) {
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
        if constexpr (BLOCK) {
            if (own_rows())
#pragma unroll
                for (int i = 0; i < NFOUR; ++i) write_row(sub(), bcol, block_at(i), block_four(i), m[0], l[0]);
            __syncthreads();
        } else if constexpr (HEAD || WIDE) {
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

    // four outputs of row r on their way, in an order that spreads a column over the banks
    __device__ __forceinline__ f32x4& turned(int r, int c) const {
        f32x4* base = MT == 1 ? sm.turn[MT == 1 ? wave : 0] : (f32x4*)sm.q[MT == 1 ? 0 : wave * MT * KS];
        return base[r * (D / 4) + (c ^ r)];
    }

    // Whether parts are stored through to memory.  A release fence writes all of
    // the XCD's L2 back, about 4 us in which the joiner waits: one list of 4096
    // takes 14.8 us without it for 18, 16 of 1024 25 for 32.  Parts of many rows
    // lie in pieces of 16 bytes, which L2 gathers better: through memory 64 lists
    // of up to 16384 with 16 rows of four heads take 486 us for 456, 8 lists
    // with 128 rows 408 for 385.
    __device__ __forceinline__ bool through() const {
        return MODE == KEYS || (HEAD && (MICRO || (MT == 1 && p.rows <= 8)));
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
        if constexpr (HEAD && MICRO) {
            close();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int i = 0; i < NTILE; ++i) turned(col, grp * NTILE + i) = four(mt, i);
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                const int r0 = mt * 16, at = wave * 16 * MT + r0;
                for (int x = lane * 4; x < 16 * D; x += 256)
                    if (r0 + x / D < p.rows)
                        pstore((f32x4*)(po + at * D + x), turned(x / D, x % D / 4));
                if (grp == 0 && r0 + col < p.rows) {
                    pstore(pm + (at + col) * 2, m[mt]);
                    pstore(pm + (at + col) * 2 + 1, l[mt]);
                }
                // the next rows' stores come after these loads
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        } else if constexpr (BLOCK) {
            if (own_rows() && row_at(sub(), bcol) < p.rows) {
                const int at = sub() * 32 + bcol;
#pragma unroll
                for (int i = 0; i < NFOUR; ++i) pstore((f32x4*)(po + at * D + block_at(i)), block_four(i));
                if (half == 0) {
                    pstore(pm + at * 2, m[0]);
                    pstore(pm + at * 2 + 1, l[0]);
                }
            }
        } else if constexpr (HEAD || WIDE) {
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

template <int DT, int D, int MT, bool SLOTS, int MODE, int F>
__global__ __launch_bounds__(threads_of(MODE, F), MODE >= WIDE2 || F != 16 ? 2 : 1) void attend_kernel(AttendParams p) {
    constexpr bool HEAD = MODE == HEADS;
    constexpr int PLACES = AttendShape<D, MT, MODE, F>::PLACES;
    __shared__ AttendShared<D, MT, MODE, F> sm;
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
        // (four heads' parts: 64 requests up to 1024 over a 4-bit cache 48 us with shares of any
        // size, 35 with these)
        sh = dense_share<PLACES, HEAD, HEAD && F != 16 ? 12 : 1>(p.c, p.workers, w);
        if (w >= sh.workers) return;
    }
    Attend<DT, D, MT, SLOTS, MODE, F> a(p, sm, mb);
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
            // (opaque: its reciprocal is not kept from the shares above to here, in the one form that
            // has no register left for it; dividing anew takes 1.7 us)
            int32_t workers = sh.workers;
            if constexpr (F != 16 && SLOTS && MODE == WIDE4) asm volatile("" : "+s"(workers));
            const int32_t w0 = share_of(sh.total, workers, g0);
            const int32_t w1 = share_of(sh.total, workers, g1 - 1);
            const bool whole_start = share_start(sh.total, workers, w0) == g0;
            a.finish_part(a.part(w, w0, whole_start), w0, w1, whole_start);
        }
        x = x1;
        if (h + 1 == head_units<HEAD>(p.c) && x1 == g1) {
            b_unit = g1;
            ++b;
        }
    }
}

template <int DT, int D, int MT, bool SLOTS, int MODE, int F>
static hipError_t launch_one(const AttendParams& p, hipStream_t stream) {
    const uint32_t grid = (uint32_t)((p.workers + 7) / 8 * 8 * p.row_blocks);
    hipLaunchKernelGGL((attend_kernel<DT, D, MT, SLOTS, MODE, F>), dim3(grid),
                       dim3(threads_of(MODE, F)), 0, stream, p);
    return hipGetLastError();
}

template <int DT, int D, bool SLOTS, int F>
static hipError_t launch_mode(const AttendParams& p, hipStream_t stream) {
    if constexpr (!SLOTS || F != 16) {
        if (p.heads_on_waves)
            return p.rows <= 16 ? launch_one<DT, D, 1, SLOTS, HEADS, F>(p, stream)
                                : launch_one<DT, D, 2, SLOTS, HEADS, F>(p, stream);
    }
    switch (p.block_rows) {
        case 16: return launch_one<DT, D, 1, SLOTS, KEYS, F>(p, stream);
        case 32: return launch_one<DT, D, 2, SLOTS, KEYS, F>(p, stream);
        case 64: return launch_one<DT, D, 2, SLOTS, WIDE2, F>(p, stream);
    }
    return launch_one<DT, D, 2, SLOTS, WIDE4, F>(p, stream);
}

}  // namespace vts
