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

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
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
