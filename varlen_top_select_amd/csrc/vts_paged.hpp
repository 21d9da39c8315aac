// vts_paged.hpp -- device building blocks of the kernels that read a paged KV
// cache with matrix instructions.
//
// A wave works on 32 cached positions at a time.  With K rows as the A operand
// of the 16x16x32 matrix product and query rows as B, lane l gets the scores
// of query row l % 16 at positions 4 * (l / 16) + {0..3} of each 16-position
// half: a query row's softmax state is one lane's scalar (replicated in four
// lanes), and the eight probabilities a lane holds are already its B operand
// of the second product, with V rows taken in the same order of positions.
#pragma once

#include "vts_decode.h"
#include "vts_device.hpp"

namespace vts {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float NOT_A_NUMBER = __builtin_nanf("");

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The 32x32x16 product, of 32 query rows: with K rows as A, lane l gets the scores of query
// row l % 32 at places key_of(e) + 4 * (l / 32), and its probabilities are in order its B
// operands of the second product, of sixteen places each.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
template <int DT>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
    if constexpr (DT == BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ constexpr int key_of(int e) { return 8 * (e >> 2) + (e & 3); }

// V rows in LDS, whole, for transposing loads: each takes 32 bytes of four rows for 16
// lanes, so a row's chunks (16 bytes) are moved by 64 bytes from row to row and the four
// lie in different banks; and by one chunk within them, so that a store of one chunk in
// four to several rows meets in no bank either.
template <int D>
__device__ __forceinline__ int v_swizzle(int r) {
    return D == 128 ? (r & 3) * 5 : ((r >> 1) & 1) << 2 | ((r >> 1) & 3);
}
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
    return r * (D / 8) + (c ^ v_swizzle<D>(r));
}
// The second product's A operand of places r0 + 16 .. and elements 32 * i ..: eight places
// in the order of the lane's probabilities.
template <int D>
__device__ __forceinline__ u32x4 turned_v(const u32x4* v, int lane, int r0, int i) {
    const int g = lane >> 4, n = lane & 15;
    u32x4 x;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int r = r0 + 8 * w + 4 * (g >> 1) + (n >> 2);
        const int c = 4 * i + 2 * (g & 1) + ((n & 3) >> 1);
        const char* at = (const char*)&v[v_chunk<D>(r, c)] + 8 * (n & 1);
        const u32x2 y = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at));
        x[2 * w] = y[0];
        x[2 * w + 1] = y[1];
    }
    return x;
}

// two floats rounded to nearest even, the first in the low half
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f32x2 v = {a, b};
    if constexpr (DT == BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

template <int DT>
__device__ __forceinline__ float to_float(uint32_t raw16) {
    if constexpr (DT == BF16)
        return __builtin_bit_cast(float, raw16 << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (uint16_t)raw16);
}

// ---- microscaled rows: one power of two (E8M0) per 32 elements of 8 bits (E4M3) or
// 4 (E2M1, the first of two in the low half of a byte)

// The scale as the conversions take it: a float's exponent.  They read 0 as 2^-127 and
// the infinity that 255 gives as NaN.
__device__ __forceinline__ float scale_of(uint32_t code) {
    return __builtin_bit_cast(float, code << 23);
}
// the two numbers in byte I of x
template <int DT, int I>
__device__ __forceinline__ uint32_t widen4(uint32_t x, float scale) {
    if constexpr (DT == BF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, I));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(x, scale, I));
}
// the two numbers in the low or high half of x
template <int DT, bool HI>
__device__ __forceinline__ uint32_t widen8(uint32_t x, float scale) {
    if constexpr (DT == BF16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, scale, HI));
}

template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t pair) {
    constexpr uint32_t E = DT == BF16 ? 0x7F80u : 0x7C00u;
    return (pair & E) == E || ((pair >> 16) & E) == E;
}
// the pair with zeros in place of what is not finite
template <int DT>
__device__ __forceinline__ uint32_t finite_part(uint32_t pair) {
    return (not_finite<DT>(pair & 0xFFFFu) ? 0 : pair & 0xFFFFu) |
           (not_finite<DT>(pair >> 16) ? 0 : pair & 0xFFFF0000u);
}

// Whether a probability as the products take it (0 or more) is 0 or NaN.
template <int DT>
__device__ __forceinline__ uint32_t weightless(uint32_t half) {
    return half - 1u >= (DT == BF16 ? 0x7F80u : 0x7C00u) ? 1 : 0;
}

// One request's (or, with slot lists, one row's) positions: a list of `count`
// places, those from `first` on being the drafted tokens.
struct Places {
    int32_t count, first;
    const int32_t* table;  // the request's page-table row
    const int32_t* slots;  // the row's slot list, or null
    int32_t top_k;
    int32_t draft_pos;     // position of the first drafted token (may be negative)
};

__device__ __forceinline__ int32_t clamped_len(const PagedParams& c, int32_t b) {
    const int32_t n = gload(c.seq_lens + b);
    return n < 0 ? 0 : n > c.capacity ? c.capacity : n;
}
// the same of a request that is the same in every lane, as a scalar
__device__ __forceinline__ int32_t uniform_len(const PagedParams& c, int32_t b) {
    return __builtin_amdgcn_readfirstlane(clamped_len(c, b));
}

template <bool SLOTS>
__device__ __forceinline__ int32_t place_count(const AttendParams& p, int32_t n) {
    if constexpr (SLOTS) return p.top_k + (p.tree_mask ? p.c.draft : 0);
    return n;
}

// A lookup in flight: a slot of the row's list, or the page-table entry of a
// position.  (Two members, for one load through a selected pointer would keep
// the caller's state in scratch memory.)
struct Entry {
    int32_t slot;   // < 0: none
    int32_t entry;  // < 0: none
    int32_t pos;
};

template <bool SLOTS>
__device__ __forceinline__ Entry issue_entry(const PagedParams& c, const Places& pl, int32_t j) {
    Entry e;
    e.slot = -1;
    e.entry = -1;
    e.pos = j;
    if constexpr (SLOTS) {
        if (j >= 0 && j < pl.top_k) e.slot = gload(pl.slots + j);
        e.pos = j < pl.top_k ? -1 : pl.draft_pos + (j - pl.top_k);
    }
    if (j < pl.count && e.pos >= 0 && e.pos < c.capacity) {
        const int32_t page = c.page_shift >= 0 ? e.pos >> c.page_shift : e.pos / c.page_size;
        e.entry = gload(pl.table + page);
    }
    return e;
}

constexpr uint32_t NO_PLACE = 0xFFFFFFFFu;

// The row's offset in 16-byte vectors, or NO_PLACE.
template <bool SLOTS>
__device__ __forceinline__ uint32_t resolve_entry(const PagedParams& c, uint32_t page_stride,
                                                  uint32_t pos_stride, const Entry& e) {
    int32_t page = e.entry, at = e.pos;
    if constexpr (SLOTS) {
        if (e.slot >= 0) {
            page = c.page_shift >= 0 ? e.slot >> c.page_shift : e.slot / c.page_size;
            at = e.slot;
        }
    }
    if (page < 0 || page >= c.num_pages) return NO_PLACE;
    at = c.page_shift >= 0 ? at & (c.page_size - 1) : at % c.page_size;
    return (uint32_t)page * page_stride + (uint32_t)at * pos_stride;
}

// A lookup in flight that loads in any case, from the first entry where there is none to
// look up: with loads in branches the compiler does not know how many are on their way,
// and waits for all of them where it needs the first.
struct Lookup {
    int32_t slot, entry;  // as loaded
    int32_t pos;          // of the entry, -1: none
    bool listed;          // the slot is the place's
};
struct Spot {
    uint32_t page, at;
    bool there;
};

template <bool SLOTS>
__device__ __forceinline__ Lookup issue_lookup(const PagedParams& c, const Places& pl, int32_t j) {
    Lookup e;
    e.slot = -1;
    e.listed = false;
    int32_t pos = j;
    if constexpr (SLOTS) {
        e.listed = j >= 0 && j < pl.top_k;
        e.slot = gload(pl.slots + (e.listed ? j : 0));
        pos = e.listed ? -1 : pl.draft_pos + (j - pl.top_k);
    }
    e.pos = j < pl.count && pos >= 0 && pos < c.capacity ? pos : -1;
    const int32_t at = e.pos < 0 ? 0 : e.pos;
    e.entry = gload(pl.table + (c.page_shift >= 0 ? at >> c.page_shift : at / c.page_size));
    return e;
}
template <bool SLOTS>
__device__ __forceinline__ Spot resolve_lookup(const PagedParams& c, const Lookup& e) {
    int32_t page = e.pos < 0 ? -1 : e.entry, at = e.pos;
    if constexpr (SLOTS) {
        if (e.listed) {
            at = e.slot;
            page = at < 0 ? -1 : c.page_shift >= 0 ? at >> c.page_shift : at / c.page_size;
        }
    }
    Spot s;
    s.there = page >= 0 && page < c.num_pages;
    s.page = s.there ? (uint32_t)page : 0;
    s.at = !s.there ? 0 : (uint32_t)(c.page_shift >= 0 ? at & (c.page_size - 1) : at % c.page_size);
    return s;
}
__device__ __forceinline__ uint32_t spot_offset(const Spot& s, uint32_t page_stride, uint32_t pos_stride) {
    return s.page * page_stride + s.at * pos_stride;
}

__device__ __forceinline__ uint32_t from_lane(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_ds_bpermute(lane << 2, (int)v);
}

template <class V, bool ONCE = false>
__device__ __forceinline__ V row_load(const void* base, uint32_t off16, uint32_t byte) {
    const VTS_GLOBAL V* at =
        (const VTS_GLOBAL V*)((const VTS_GLOBAL char*)base + ((uint64_t)off16 << 4) + byte);
    if constexpr (ONCE) return __builtin_nontemporal_load(at);  // read by nobody else
    return *at;
}

// K rows on their way from the order of whole rows to operands, in LDS: chunk c
// (16 bytes) of row r lies at chunk c ^ swizzled(r) of the row, so that neither
// the stores (whole rows) nor the loads (one chunk of 16 rows) meet in a bank.
template <int D>
__device__ __forceinline__ int swizzled(int r) {
    return D == 128 ? r & 15 : (r >> 1) & 7;
}

// ---- shares of the work: units of PLACES places, in order of request and KV
// head (or four heads); worker w of W takes units [w * total / W,
// (w + 1) * total / W).

__device__ __forceinline__ int64_t share_start(int64_t total, int32_t workers, int32_t w) {
    return total * w / workers;
}
// the worker whose share holds unit x (total >= workers)
__device__ __forceinline__ int32_t share_of(int64_t total, int32_t workers, int64_t x) {
    return (int32_t)(((x + 1) * workers - 1) / total);
}

template <int PLACES>
__device__ __forceinline__ int32_t units_of(int32_t count) {
    return count <= 0 ? 1 : (count + PLACES - 1) / PLACES;
}
// units that differ by KV head alone
template <bool HEADS>
__device__ __forceinline__ int32_t head_units(const PagedParams& c) {
    return HEADS ? c.kv_heads / WAVES : c.kv_heads;
}

// Where a worker's share begins: request, KV head, unit, and the totals.
struct Share {
    int64_t total, begin, end;
    int32_t b;       // request of unit `begin`
    int64_t b_unit;  // first unit of request b
    int32_t workers;
};

// a value that is the same in every lane, as a scalar
__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = first_lane_value((uint32_t)v), hi = first_lane_value((uint32_t)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Shares over the batch's dense lengths; with LEAST, of that many units where this leaves
// 256 of them or more.  Every wave finds the same by itself, four requests to a lane and 256
// at a time.
template <int PLACES, bool HEADS, int LEAST = 1>
__device__ __forceinline__ Share dense_share(const PagedParams& c, int32_t workers, int32_t w) {
    constexpr int PER = 4, STEP = 64 * PER;
    const int32_t heads = head_units<HEADS>(c);
    const int lane = lane_id();
    int64_t u[PER];
    // the lane's units, their sum over the lanes up to this one, and over all
    const auto scan = [&](int32_t b0, int64_t& all) -> int64_t {
        int64_t inc = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int32_t b = b0 + lane * PER + i;
            u[i] = b < c.batch ? (int64_t)units_of<PLACES>(clamped_len(c, b)) * heads : 0;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) inc += u[i];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        all = uniform64(__shfl(inc, 63));
        return inc;
    };
    Share s;
    s.total = 0;
    int64_t all, inc = 0;
    for (int32_t b0 = 0; b0 < c.batch; b0 += STEP) {
        inc = scan(b0, all);
        s.total += all;
    }
    int64_t most = s.total;
    if (LEAST > 1 && most > 256) most = most / LEAST > 256 ? most / LEAST : 256;
    s.workers = most < workers ? (int32_t)most : workers;
    s.begin = s.end = s.b_unit = 0;
    s.b = 0;
    if (w >= s.workers) return s;
    s.begin = share_start(s.total, s.workers, w);
    s.end = share_start(s.total, s.workers, w + 1);
    int64_t base = 0;
    for (int32_t b0 = 0; b0 < c.batch; b0 += STEP) {
        if (c.batch > STEP) inc = scan(b0, all);  // (of one step the first scan is at hand)
        const uint64_t past = ballot(s.begin < base + inc);
        if (past) {
            const int at = __builtin_ctzll(past);
            // within that lane's requests
            int64_t start = base + inc;
#pragma unroll
            for (int i = 0; i < PER; ++i) start -= u[i];
            int32_t b = b0 + lane * PER;
#pragma unroll
            for (int i = 0; i < PER - 1; ++i)
                if (s.begin >= start + u[i] && b == b0 + lane * PER + i) {
                    start += u[i];
                    ++b;
                }
            s.b = __builtin_amdgcn_readfirstlane(__shfl(b, at));
            s.b_unit = uniform64(__shfl(start, at));
            return s;
        }
        base += all;
    }
    return s;
}

}  // namespace vts
