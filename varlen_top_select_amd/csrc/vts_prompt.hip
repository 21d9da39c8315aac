// vts_prompt.hip -- attention of whole prompts, packed one after the other.
//
//   o_i = sum_j p_ij v_j,  p_i = softmax_j(scale * q_i . k_j)
//
// over the keys j of i's sequence, up to i's own (its queries are the last of its
// keys).  One pass with a running maximum and sum per row, as in vts_attend.hpp.
//
// The rows of a workgroup are tokens times the query heads of one KV head, so that K
// and V are read once for a whole group and a tile of 128 rows spans few tokens: its
// masked corner is small, and a sequence of one token still fills `group` rows.  A wave
// has 32 rows; K and V tiles of 64 keys go through LDS for all waves.  With K rows
// as A and query rows as B of the 32x32x16 product, lane l gets scores of row l % 32
// at keys 8 * (e / 4) + 4 * (l / 32) + e % 4: its sixteen probabilities are already
// its B operands of the second product, with V's keys taken in the same order by
// transposing LDS loads.  m is raised only when a score passes it by a margin, and p is
// rounded to the type of V for the second product, whose operands it takes (at most half
// a step, 2^-8 of a bf16 p and 2^-11 of an fp16 one, which average out over the keys; the
// margins are those of vts_attend.hpp); l sums the unrounded p, and all else is 32-bit.
//
// Where there are few tiles and long contexts, several workgroups take parts of a tile's
// keys, and a second kernel joins them.
#include "vts_cache.h"
#include "vts_paged.hpp"

namespace vts {

constexpr int PROMPT_WAVES = PROMPT_ROWS / 32;
constexpr int PROMPT_NT = PROMPT_WAVES * 64;
constexpr int PROMPT_KEYS = 64;  // of a tile

template <int D>
struct PromptShared {
    u32x4 k[2][PROMPT_KEYS * (D / 8)], v[2][PROMPT_KEYS * (D / 8)];
    int32_t bad[2];  // 1 + the first key of the last tile there whose V held something not finite
};

// A workgroup's tile: its sequence, the first of its rows, and the lengths.
struct PromptTile {
    int32_t q0, k0, lq, lk, row0;
    bool found;
};

__device__ __forceinline__ int32_t cu_at(const int32_t* cu, int32_t i, int32_t total) {
    const int32_t n = gload(cu + i);
    return n < 0 ? 0 : n > total ? total : n;
}

// Tile t of all sequences' tiles.  Every wave finds it by itself, 64 sequences at a time.
__device__ __forceinline__ PromptTile find_tile(const PromptParams& p, int32_t t) {
    PromptTile r;
    r.found = false;
    const int lane = lane_id();
    int32_t base = 0;
    for (int32_t b0 = 0; b0 < p.batch; b0 += 64) {
        const int32_t b = b0 + lane;
        int32_t q0 = 0, len = 0, k0 = 0, keys = 0;
        if (b < p.batch) {
            q0 = cu_at(p.cu_q, b, p.total_q);
            k0 = cu_at(p.cu_k, b, p.total_k);
            len = cu_at(p.cu_q, b + 1, p.total_q) - q0;
            keys = cu_at(p.cu_k, b + 1, p.total_k) - k0;
            if (len < 0) len = 0;
            if (keys < 0) keys = 0;
        }
        if (p.longest_first) {
            // each sequence to the lane of its place in the order of falling lengths
            int32_t place = 0;
            for (int32_t i = 0; i < p.batch; ++i) {
                const int32_t n = __builtin_amdgcn_readlane(keys, i);
                place += n > keys || (n == keys && i < lane) ? 1 : 0;
            }
            place = lane < p.batch ? place : lane;
            q0 = __builtin_amdgcn_ds_permute(place << 2, q0);
            k0 = __builtin_amdgcn_ds_permute(place << 2, k0);
            len = __builtin_amdgcn_ds_permute(place << 2, len);
            keys = __builtin_amdgcn_ds_permute(place << 2, keys);
        }
        const int32_t mine = (len * p.group + PROMPT_ROWS - 1) / PROMPT_ROWS;
        int32_t inc = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        const uint64_t past = ballot(t < base + inc);
        if (past) {
            const int at = __builtin_ctzll(past);
            r.found = true;
            r.q0 = __builtin_amdgcn_readlane(q0, at);
            r.lq = __builtin_amdgcn_readlane(len, at);
            const int32_t tiles = __builtin_amdgcn_readlane(mine, at);
            const int32_t first = base + __builtin_amdgcn_readlane(inc, at) - tiles;
            // the sequence's last tile, which sees the most, comes first
            r.row0 = (tiles - 1 - (t - first)) * PROMPT_ROWS;
            r.k0 = __builtin_amdgcn_readlane(k0, at);
            r.lk = __builtin_amdgcn_readlane(keys, at);
            return r;
        }
        base += __builtin_amdgcn_readlane(inc, 63);
    }
    return r;
}

template <int DT, int D>
struct Prompt {
    static constexpr int CH = D / 8;     // 16-byte chunks of a row
    static constexpr int KS = D / 16;    // steps of the first product
    static constexpr int MT = D / 32;    // tiles of the second
    static constexpr int LOADS = PROMPT_KEYS * CH / PROMPT_NT;
    static constexpr float SHIFT = DT == F16 ? 11 : 0, RAISE = DT == F16 ? 15 : 8;

    const PromptParams& p;
    PromptShared<D>& sm;
    PromptTile t;
    int32_t kv;
    int tid, lane, wave, col, half;
    int32_t limit;  // the last key that the lane's row sees, -1: none
    bool valid;
    int64_t row_out;  // the row's place in lse, and out
    u32x4 q[KS];
    f32x16 o[MT];
    float m, l;
    u32x4 kr[LOADS], vr[LOADS];  // the tile on its way

    __device__ __forceinline__ Prompt(const PromptParams& p_, PromptShared<D>& s_, const PromptTile& t_, int32_t kv_)
        : p(p_), sm(s_), t(t_), kv(kv_) {
        tid = threadIdx.x;
        lane = tid & 63;
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        col = lane & 31;
        half = lane >> 5;
        const int32_t row = t.row0 + wave * 32 + col;
        const int32_t token = row / p.group, head = kv * p.group + (row - token * p.group);
        valid = token < t.lq;
        limit = !valid ? -1 : p.causal ? token + t.lk - t.lq : t.lk - 1;
        row_out = (int64_t)(t.q0 + token) * p.heads + head;
        const char* at = (const char*)p.q +
                         2 * (valid ? (int64_t)(t.q0 + token) * p.q_token + head * p.q_head : 0);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            u32x4 x = {0, 0, 0, 0};
            if (valid) x = gload((const u32x4*)at + s * 2 + half);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] ^= p.q_sign;
            q[s] = x;
        }
        m = NEG_INF;
        l = 0;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] = 0;
    }

    static __device__ __forceinline__ int k_at(int r, int c) {
        return r * CH + (c ^ (D == 128 ? r & 15 : (r >> 1) & 7));
    }
    __device__ __forceinline__ void load(int32_t j0) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int x = i * PROMPT_NT + tid, c = x % CH;
            int32_t j = j0 + x / CH;
            if (j >= t.lk) j = t.lk - 1;
            const int64_t row = t.k0 + j;
            kr[i] = gload((const u32x4*)((const char*)p.k + 2 * (row * p.k_token + kv * p.k_head)) + c);
            vr[i] = gload((const u32x4*)((const char*)p.v + 2 * (row * p.v_token + kv * p.v_head)) + c);
        }
    }
    __device__ __forceinline__ void stage(int buf) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int x = i * PROMPT_NT + tid, r = x / CH, c = x % CH;
            sm.k[buf][k_at(r, c)] = kr[i];
            sm.v[buf][v_chunk<D>(r, c)] = vr[i];
        }
    }
    template <bool MASKED>
    __device__ __forceinline__ void tile(int32_t j0, int buf) {
        const float c = p.scale_log2e;
        f32x16 s[2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                s[b] = mfma32<DT>(sm.k[buf][k_at(32 * b + col, 2 * ks + half)], q[ks], s[b]);
        if constexpr (MASKED) {
            const int32_t last = limit - j0 - 4 * half;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[b][e] = 32 * b + key_of(e) <= last ? s[b][e] : NEG_INF;
        }
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
        top *= c;
        if (ballot(top > m + RAISE)) {
            float up = fmaxf(top, __shfl_xor(top, 32));
            up = up > m + RAISE ? up - SHIFT : m;
            const float f = up == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[i][e] *= f;
        }
        const float base = m == NEG_INF ? 0.0f : m;
        u32x4 pv[4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(s[b][e], c, -base));
                const float y = __builtin_amdgcn_exp2f(fmaf(s[b][e + 1], c, -base));
                l += x + y;
                pv[2 * b + (e >> 3)][(e >> 1) & 3] = pack2<DT>(x, y);
            }
#pragma unroll
        for (int step = 0; step < 4; ++step)
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i] = mfma32<DT>(turned_v<D>(sm.v[buf], lane, 16 * step, i), pv[step], o[i]);
    }

    // Where not every row sees every key, an infinity or NaN in V would reach rows that
    // do not see it (0 * inf).  Such a tile's are cleared on the way to LDS, and what rows
    // see of them is added after the tile's products, from memory: rare, and kept apart from
    // the tile on its way, whose registers it would take (45 spilled): that is loaded again.
    __device__ __forceinline__ void clear_not_finite(int32_t j0, int buf) {
        bool f = false;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = vr[i][e];
                f = f || not_finite<DT>(w);
                vr[i][e] = finite_part<DT>(w);
            }
        if (f) sm.bad[buf] = j0 + 1;
    }
    // Which of the lane's probabilities of 32 keys in half `buf` are 0 or NaN: sixteen bits, their
    // scores computed again.
    __device__ __forceinline__ uint32_t weightless_block(int buf, int b) const {
        f32x16 s;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            s = mfma32<DT>(sm.k[buf][k_at(32 * b + col, 2 * ks + half)], q[ks], s);
        const float base = m == NEG_INF ? 0.0f : m;
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x |= weightless<DT>(pack2<DT>(__builtin_amdgcn_exp2f(fmaf(s[e], p.scale_log2e, -base)), 0.0f) & 0xFFFFu) << e;
        return x;
    }
    // An infinity of any weight is the infinity; of none (a score of -inf) it is NaN, as the
    // products of other tiles give it.
    __device__ __forceinline__ void add_not_finite(int32_t j0, int32_t end, int buf) {
        uint32_t none = 0;
#pragma unroll 1
        for (int32_t j = j0; j < end; ++j) {
            const int kk = j - j0;
            if ((kk & 31) == 0) none = weightless_block(buf, kk >> 5);
            const char* at = (const char*)p.v + 2 * ((int64_t)(t.k0 + j) * p.v_token + kv * p.v_head);
            const bool see = j <= limit;
            const int bit = (kk >> 3 & 3) * 4 + (kk & 3);
            const bool weighs_nothing = from_lane(none, (kk >> 2 & 1) * 32 + col) >> bit & 1;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const u32x2 four = gload((const u32x2*)(at + 2 * (32 * i + key_of(e) + 4 * half)));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t raw = (four[x >> 1] >> (16 * (x & 1))) & 0xFFFFu;
                        const float y = o[i][e + x] + (weighs_nothing ? NOT_A_NUMBER : to_float<DT>(raw));
                        o[i][e + x] = see && not_finite<DT>(raw) ? y : o[i][e + x];
                    }
                }
        }
    }

    // The row as a part of its keys gives it: outputs that are not divided, maximum and sum.
    __device__ __forceinline__ void write_part(int64_t part) {
        l += __shfl_xor(l, 32);
        if (!valid) return;
        const int64_t at = part * PROMPT_ROWS + wave * 32 + col;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                gstore((f32x4*)(p.part_o + at * D + 32 * i + key_of(e) + 4 * half),
                       f32x4{o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3]});
        if (half == 0) {
            gstore(p.part_ml + 2 * at, m);
            gstore(p.part_ml + 2 * at + 1, l);
        }
    }
    __device__ __forceinline__ void write() {
        l += __shfl_xor(l, 32);
        if (!valid) return;
        const bool none = l == 0.0f;  // (then o is NaN where V is no finite number)
        const float inv = 1.0f / l;
        char* at = (char*)p.out + 2 * row_out * D;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                u32x2 w;
                w[0] = none ? 0 : pack2<DT>(o[i][e] * inv, o[i][e + 1] * inv);
                w[1] = none ? 0 : pack2<DT>(o[i][e + 2] * inv, o[i][e + 3] * inv);
                gstore((u32x2*)(at + 2 * (32 * i + key_of(e) + 4 * half)), w);
            }
        if (half == 0 && p.lse)
            gstore(p.lse + row_out, none ? NEG_INF
                                         : (m + SHIFT + log2f(l * __builtin_exp2f(-SHIFT))) *
                                               0.6931471805599453f);
    }

    // A tile that every row sees, from memory to half `buf` without the way through
    // registers (32 of them, which the products' operands take).  LDS gets a wave's chunks
    // one after the other, so a lane reads the chunk that lies at its place.
    __device__ __forceinline__ void load_direct(int32_t j0, int buf) {
        const int r = tid / CH, c = tid % CH;  // (of 256 chunks; the next ones are as many rows on)
        const uint32_t ko = 2 * (uint32_t)(r * p.k_token) + 16 * (c ^ (D == 128 ? r & 15 : (r >> 1) & 7));
        const uint32_t vo = 2 * (uint32_t)(r * p.v_token) + 16 * (c ^ v_swizzle<D>(r));
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int64_t row = t.k0 + j0 + i * (PROMPT_NT / CH);
            to_lds(&sm.k[buf][i * PROMPT_NT + wave * 64], (const char*)p.k + 2 * (row * p.k_token + kv * p.k_head), ko);
            to_lds(&sm.v[buf][i * PROMPT_NT + wave * 64], (const char*)p.v + 2 * (row * p.v_token + kv * p.v_head), vo);
        }
    }
    static __device__ __forceinline__ void to_lds(u32x4* to, const char* base, uint32_t offset) {
        __builtin_amdgcn_global_load_lds((const VTS_GLOBAL void*)((const VTS_GLOBAL char*)base + offset),
                                         (__attribute__((address_space(3))) void*)to, 16, 0, 0);
    }
    // the tile at j0 to LDS, and the next one on its way
    __device__ __forceinline__ void next(int32_t j0, int32_t end, int buf) {
        clear_not_finite(j0, buf);
        // the other half may still be read; this one was done with before the last barrier
        stage(buf);
        if (j0 + PROMPT_KEYS < end) load(j0 + PROMPT_KEYS);
        __syncthreads();
    }
    // Part `split` of the keys.
    __device__ __forceinline__ void run(int32_t split) {
        // the keys that the last token of the tile sees, and those that all rows see
        const int32_t rows = t.lq * p.group;
        const int32_t last_row = t.row0 + PROMPT_ROWS < rows ? t.row0 + PROMPT_ROWS - 1 : rows - 1;
        int32_t end = !p.causal ? t.lk : last_row / p.group + 1 + t.lk - t.lq;
        int32_t all = !p.causal ? t.lk : t.row0 / p.group + 1 + t.lk - t.lq;
        int32_t j0 = 0;
        if (p.splits > 1 && end > 0) {
            const int64_t tiles = (end + PROMPT_KEYS - 1) / PROMPT_KEYS;
            j0 = (int32_t)(tiles * split / p.splits) * PROMPT_KEYS;
            const int32_t to = (int32_t)(tiles * (split + 1) / p.splits) * PROMPT_KEYS;
            if (to < end) end = to;
            if (to < all) all = to;
        }
        if (j0 < end) {
            if (tid < 2) sm.bad[tid] = 0;
            int buf = 0;
            if (p.direct && j0 + PROMPT_KEYS <= all) {
                load_direct(j0, 0);
#pragma unroll 1
                for (; j0 + PROMPT_KEYS <= all; j0 += PROMPT_KEYS, buf ^= 1) {
                    // this wave's part of the tile is there, and after the barrier everyone's;
                    // all have done with the other half
                    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    __syncthreads();
                    if (j0 + 2 * PROMPT_KEYS <= all) load_direct(j0 + PROMPT_KEYS, buf ^ 1);
                    tile<false>(j0, buf);
                }
            }
            if (j0 < end) load(j0);
            __syncthreads();
#pragma unroll 1
            for (; j0 < end; j0 += PROMPT_KEYS, buf ^= 1) {
                next(j0, end, buf);
                tile<true>(j0, buf);
                if (sm.bad[buf] == j0 + 1) {
                    add_not_finite(j0, j0 + PROMPT_KEYS < end ? j0 + PROMPT_KEYS : end, buf);
                    if (j0 + PROMPT_KEYS < end) load(j0 + PROMPT_KEYS);
                }
            }
        }
    }
};

// (Heads of 64: three workgroups to a compute unit, packed prompts 342 us for 375 with two.)
template <int DT, int D>
__global__ __launch_bounds__(PROMPT_NT, D == 64 ? 3 : 2) void prompt_kernel(PromptParams p) {
    __shared__ PromptShared<D> sm;
    const int32_t work = p.tiles * p.kv_heads * p.splits;
    if ((int32_t)blockIdx.x >= work) {
        // rows of no sequence, before the first and behind the last
        const int32_t a = p.batch > 0 ? cu_at(p.cu_q, 0, p.total_q) : 0;
        const int32_t b = p.batch > 0 ? cu_at(p.cu_q, p.batch, p.total_q) : 0;
        const int64_t per = (int64_t)p.heads * (D / 8), all = ((int64_t)a + p.total_q - b) * per;
        const int64_t step = (int64_t)(gridDim.x - work) * PROMPT_NT;
        for (int64_t x = (int64_t)(blockIdx.x - work) * PROMPT_NT + threadIdx.x; x < all; x += step) {
            const int64_t y = x < a * per ? x : x + (int64_t)(b - a) * per;
            gstore((u32x4*)p.out + y, u32x4{0, 0, 0, 0});
            if (p.lse && y % (D / 8) == 0) gstore(p.lse + y / (D / 8), NEG_INF);
        }
        return;
    }
    const int32_t kv = (int32_t)blockIdx.x % p.kv_heads, x = (int32_t)blockIdx.x / p.kv_heads;
    const int32_t n = x / p.splits, split = x - n * p.splits;
    const PromptTile t = find_tile(p, n);
    if (!t.found) return;
    Prompt<DT, D> a(p, sm, t, kv);
    a.run(split);
    if (p.splits > 1)
        a.write_part(((int64_t)n * p.kv_heads + kv) * p.splits + split);
    else
        a.write();
}

// The parts of a tile's rows joined, in their order: 32 rows to a workgroup.
constexpr int JOIN_ROWS = 32;
template <int DT, int D>
__global__ __launch_bounds__(PROMPT_NT) void prompt_join_kernel(PromptParams p) {
    constexpr float SHIFT = DT == F16 ? 11 : 0;
    constexpr int PER = PROMPT_ROWS / JOIN_ROWS;
    const int32_t x = (int32_t)blockIdx.x / PER, first = (int32_t)blockIdx.x % PER * JOIN_ROWS;
    const int32_t kv = x % p.kv_heads, n = x / p.kv_heads;
    const PromptTile t = find_tile(p, n);
    if (!t.found) return;
    for (int32_t y = (int32_t)threadIdx.x * 4; y < JOIN_ROWS * D; y += PROMPT_NT * 4) {
        const int32_t r = first + y / D, d = y % D, row = t.row0 + r, token = row / p.group;
        if (token >= t.lq) continue;
        const int64_t part = ((int64_t)n * p.kv_heads + kv) * p.splits;
        float top = NEG_INF, sum = 0;
        f32x4 o = {0, 0, 0, 0};
        for (int32_t s = 0; s < p.splits; ++s) {
            const int64_t at = (part + s) * PROMPT_ROWS + r;
            const float m = gload(p.part_ml + 2 * at), l = gload(p.part_ml + 2 * at + 1);
            const f32x4 v = gload((const f32x4*)(p.part_o + at * D + d));
            const float up = fmaxf(top, m);
            const float f = up == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(top - up);
            const float g = up == NEG_INF ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            top = up;
            sum = sum * f + l * g;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = o[e] * f + v[e] * g;
        }
        const bool none = sum == 0.0f;
        const float inv = 1.0f / sum;
        const int64_t out = (int64_t)(t.q0 + token) * p.heads + kv * p.group + (row - token * p.group);
        u32x2 w;
        w[0] = none ? 0 : pack2<DT>(o[0] * inv, o[1] * inv);
        w[1] = none ? 0 : pack2<DT>(o[2] * inv, o[3] * inv);
        gstore((u32x2*)((char*)p.out + 2 * (out * D + d)), w);
        if (d == 0 && p.lse)
            gstore(p.lse + out, none ? NEG_INF
                                     : (top + SHIFT + log2f(sum * __builtin_exp2f(-SHIFT))) * 0.6931471805599453f);
    }
}

template <int DT, int D>
static hipError_t start(const PromptParams& p, hipStream_t stream) {
    const uint32_t grid = (uint32_t)(p.tiles * p.kv_heads * p.splits + (p.clear ? 64 : 0));
    hipLaunchKernelGGL((prompt_kernel<DT, D>), dim3(grid), dim3(PROMPT_NT), 0, stream, p);
    if (p.splits > 1)
        hipLaunchKernelGGL((prompt_join_kernel<DT, D>), dim3(p.tiles * p.kv_heads * (PROMPT_ROWS / JOIN_ROWS)),
                           dim3(PROMPT_NT), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_prompt(int dtype, int head_dim, const PromptParams& p, hipStream_t stream) {
    if (dtype == BF16) return head_dim == 64 ? start<BF16, 64>(p, stream) : start<BF16, 128>(p, stream);
    return head_dim == 64 ? start<F16, 64>(p, stream) : start<F16, 128>(p, stream);
}

}  // namespace vts
