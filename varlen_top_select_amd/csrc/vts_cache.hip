// vts_cache.hip -- tokens' keys and values into a paged cache, and out of it.
//
// write:  q and k are normalised per head (x / sqrt(mean x^2 + eps) * w), turned by
// their position's angles ((a, b) -> (a c - b s, b c + a s) for each pair of a row) and
// q goes to an output, k and v to the cache, in 16 bits or microscaled: e is the least
// exponent with which the block's largest magnitude, divided by 2^e, rounds to a number
// of the format, and the elements are x / 2^e rounded to nearest even.  One pass: a row
// is held by D / 8 lanes, its pairs meet by one exchange of raw elements, and norm, weight
// and angle are one product and one fused product to an element, with factors that a
// wave makes once for its token.
//
// q, and k for a 16-bit cache, are computed in 32 bits and rounded once.  A microscaled
// k is computed in 64: an element next to the border of two 4-bit numbers goes to the
// same one whatever the order of the sums, and the time is the memory's (64-bit products
// are issued at half the 32-bit rate, and only k's rows take them).
//
// read:  the rows of listed slots, widened exactly.
#include "vts_cache.h"
#include "vts_paged.hpp"

namespace vts {

constexpr int CACHE_NT = 256;

__device__ __forceinline__ void slot_place(const SlotCache& c, int32_t slot, uint32_t& page,
                                           uint32_t& at) {
    if (c.page_shift >= 0) {
        page = (uint32_t)slot >> c.page_shift;
        at = (uint32_t)slot & (uint32_t)(c.page_size - 1);
    } else {
        page = (uint32_t)slot / (uint32_t)c.page_size;
        at = (uint32_t)slot % (uint32_t)c.page_size;
    }
}
// where a slot's row of head 0 begins, in 16-byte vectors and in rows of scales
__device__ __forceinline__ uint32_t slot_row(const CacheView& v, uint32_t page, uint32_t at) {
    return page * v.page_stride + at * v.pos_stride;
}
__device__ __forceinline__ uint32_t slot_scale(const ScaleView& v, uint32_t page, uint32_t at) {
    return page * v.page_stride + at * v.pos_stride;
}

template <int DT>
__device__ __forceinline__ void unpack8(u32x4 raw, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = to_float<DT>(raw[i] & 0xFFFFu);
        x[2 * i + 1] = to_float<DT>(raw[i] >> 16);
    }
}
template <int DT>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pack2<DT>(x[2 * i], x[2 * i + 1]);
    return y;
}

// A 64-bit value to 32 bits such that a later rounding to fewer sees on which side of
// a border it lies: towards zero, with the last bit set if anything was lost.
__device__ __forceinline__ float to_odd(double d) {
    const float f = (float)d;
    const double back = f;
    if (back == d) return f;
    uint32_t u = __builtin_bit_cast(uint32_t, f);
    if (__builtin_fabs(back) > __builtin_fabs(d)) u -= 1;
    return __builtin_bit_cast(float, u | 1u);
}
__device__ __forceinline__ float to_odd(float f) { return f; }

// v of the lane `x` lanes away (by exclusive or), for the sums over a row's lanes
__device__ __forceinline__ float other(float v, int x) { return __shfl_xor(v, x); }
__device__ __forceinline__ double other(double v, int x) { return __shfl_xor(v, x); }

// The scale of a block whose largest magnitude has these bits: the exponent plus 127,
// 255 for a block that is not finite.
template <int BITS>
__device__ __forceinline__ uint32_t scale_code(uint32_t top) {
    // the largest number is 1.75 * 2^8 (1.5 * 2^2); up to 1.8125 * 2^8 (below 1.75 * 2^2)
    // rounds to it
    constexpr uint32_t EMAX = BITS == 8 ? 8 : 2, PAST = BITS == 8 ? 0x680001u : 0x600000u;
    const uint32_t e = (top >> 23) + ((top & 0x7FFFFFu) >= PAST ? 1 : 0);
    if (top >= 0x7F800000u) return 255;
    return e > EMAX ? e - EMAX : 0;
}

// Eight elements of a row, four lanes to a block of 32: the lane's bytes, and the
// block's scale.
template <int BITS>
__device__ __forceinline__ u32x2 quantise8(const float (&x)[8], uint32_t& code) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __builtin_bit_cast(uint32_t, x[i]) & 0x7FFFFFFFu;  // (NaN above infinity)
        top = u > top ? u : top;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
        const uint32_t u = (uint32_t)__shfl_xor((int)top, d);
        top = u > top ? u : top;
    }
    code = scale_code<BITS>(top);
    const float scale = scale_of(code);
    u32x2 w = {0, 0};
    if constexpr (BITS == 4) {
        uint32_t y = 0;
        y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[0], x[1], scale, 0);
        y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[2], x[3], scale, 1);
        y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[4], x[5], scale, 2);
        y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[6], x[7], scale, 3);
        w[0] = y;
    } else {
        typedef short s16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s16x2 y = {0, 0};
            y = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(y, x[4 * i], x[4 * i + 1], scale, false);
            y = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(y, x[4 * i + 2], x[4 * i + 3], scale, true);
            w[i] = __builtin_bit_cast(uint32_t, y);
        }
    }
    if (code == 255) w = u32x2{0, 0};
    return w;
}

template <int DT, int D, int BITS>
struct Writer {
    static constexpr int LANES = D / 8;        // of a row
    static constexpr int ROWS = 64 / LANES;    // of a wave
    using KT = typename std::conditional<BITS == 16, float, double>::type;

    const WriteParams& p;
    int lane, c, sub;  // c: the lane's eight elements of its row
    int32_t token;
    bool valid, kept;
    // the angle's factors of the lane's elements and of their partners; src: the lane
    // that holds these (its own for neighbouring pairs), turned: whether there are any
    float cosine[8], sine[8];
    int src;
    bool turned;

    __device__ __forceinline__ Writer(const WriteParams& p_, int32_t token_) : p(p_), token(token_) {
        lane = threadIdx.x & 63;
        c = lane % LANES;
        sub = lane / LANES;
    }

    __device__ __forceinline__ void angles() {
        valid = true;
        turned = p.rot > 0 && c * 8 < p.rot;
        src = lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cosine[i] = 1;
            sine[i] = 0;
        }
        if (p.rot == 0) return;
        const int32_t pos = gload(p.positions + token);
        valid = pos >= 0 && pos < p.max_position;
        if (!valid || !turned) return;
        const float* row = p.rotary + (int64_t)pos * p.rot;
        if (p.interleaved) {
            const f32x4 a = gload((const f32x4*)(row + c * 4));
            const f32x4 b = gload((const f32x4*)(row + p.rot / 2 + c * 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cosine[i] = a[i / 2];
                sine[i] = i & 1 ? b[i / 2] : -b[i / 2];
            }
        } else {
            const int half = p.rot / 16;
            const bool first = c < half;
            const int at = (first ? c : c - half) * 8;
            src = first ? lane + half : lane - half;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 a = gload((const f32x4*)(row + at + 4 * i));
                const f32x4 b = gload((const f32x4*)(row + p.rot / 2 + at + 4 * i));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    cosine[4 * i + j] = a[j];
                    sine[4 * i + j] = first ? -b[j] : b[j];
                }
            }
        }
    }

    // The factors of a row's elements and of their partners: the norm's weights times
    // the angle's.
    template <typename T>
    __device__ __forceinline__ void factors(const void* w, T (&own)[8], T (&partner)[8]) const {
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = b[i] = 1;
        if (w != nullptr) {
            weights(w, c, a);
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) b[i] = a[i ^ 1];
            } else {
                weights(w, c + src - lane, b);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            own[i] = (T)a[i] * (T)cosine[i];
            partner[i] = (T)b[i] * (T)sine[i];
        }
    }
    __device__ __forceinline__ void weights(const void* w, int chunk, float (&x)[8]) const {
        if (p.norm_f32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 a = gload((const f32x4*)w + chunk * 2 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * i + j] = a[j];
            }
        } else {
            unpack8<DT>(gload((const u32x4*)w + chunk), x);
        }
    }

    // A row's elements normalised and turned.  Every lane of the wave takes part.
    template <typename T>
    __device__ __forceinline__ void turn(u32x4 raw, bool norm, const T (&own)[8],
                                         const T (&partner)[8], T (&y)[8]) const {
        float x[8], z[8];
        unpack8<DT>(raw, x);
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = x[i ^ 1];
        } else {
            u32x4 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = from_lane(raw[i], src);
            unpack8<DT>(r, z);
        }
        T inv = 1;
        if (norm) {
            T sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += (T)x[i] * (T)x[i];
#pragma unroll
            for (int d = 1; d < LANES; d <<= 1) sum += other(sum, d);
            inv = (T)1 / sqrt(sum * ((T)1 / D) + (T)p.eps);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            T a = (T)x[i] * own[i];
            // (nothing is added where there is no partner: 0 * inf)
            if (turned) a += (T)z[i] * partner[i];
            y[i] = a * inv;
        }
    }

    // The inputs are read once, and leave the caches alone: 16384 tokens of 64 and 8 heads
    // into a 4-bit cache and back take 160 us for 169, and 156 with such stores of q_out too
    // (4.8 TB/s; 163 on a slower card, 4.6.  A copy of 4 GiB: 4.7 to 4.95).
    __device__ __forceinline__ u32x4 load(const void* base, int64_t token_stride, int64_t head_stride,
                                          int32_t head, int32_t heads) const {
        u32x4 x = {0, 0, 0, 0};
        if (head < heads)
            x = __builtin_nontemporal_load(
                (const VTS_GLOBAL u32x4*)((const char*)base + 2 * (token * token_stride + head * head_stride)) + c);
        return x;
    }

    // a row into the cache
    __device__ __forceinline__ void store(const CacheView& view, const ScaleView& scale, uint32_t row,
                                          uint32_t scale_row, int32_t head, bool ok, u32x4 half,
                                          const float (&x)[8]) const {
        char* at = (char*)view.base + ((uint64_t)(row + (uint32_t)head * view.head_stride) << 4);
        if constexpr (BITS == 16) {
            if (ok) gstore((u32x4*)at + c, half);
        } else {
            uint32_t code;
            const u32x2 w = quantise8<BITS>(x, code);
            if (!ok) return;
            if constexpr (BITS == 8)
                gstore((u32x2*)at + c, w);
            else
                gstore((uint32_t*)at + c, w[0]);
            if ((c & 3) == 0)
                gstore((uint8_t*)scale.base + (uint64_t)(scale_row + (uint32_t)head * scale.head_stride) * (D / 32) +
                           c / 4,
                       (uint8_t)code);
        }
    }

    __device__ __forceinline__ void run(int32_t part) {
        const int32_t kv = p.c.kv_heads;
        const int32_t q_end = (p.heads + ROWS - 1) / ROWS, each = (kv + ROWS - 1) / ROWS;
        angles();
        const int32_t slot = gload(p.slots + token);
        kept = valid && slot >= 0 && slot < p.c.num_slots;
        uint32_t page = 0, at = 0;
        if (kept) slot_place(p.c, slot, page, at);
        int32_t it = part;
        if (it < q_end) {
            float own[8], partner[8];
            factors<float>(p.q_norm, own, partner);
            u32x4 next = load(p.q, p.q_token, p.q_head, it * ROWS + sub, p.heads);
#pragma unroll 1
            for (; it < q_end; it += p.parts) {
                const u32x4 raw = next;
                const int32_t head = it * ROWS + sub;
                if (it + p.parts < q_end)
                    next = load(p.q, p.q_token, p.q_head, head + p.parts * ROWS, p.heads);
                float y[8];
                turn<float>(raw, p.q_norm != nullptr, own, partner, y);
                u32x4 out = pack8<DT>(y);
                if (!valid) out = u32x4{0, 0, 0, 0};
                if (head < p.heads) {
                    u32x4* at = (u32x4*)((char*)p.q_out + 2 * ((int64_t)token * p.heads + head) * D) + c;
                    // (where there are many tokens; what reads the queries of a few finds them
                    // in the caches)
                    if (p.parts == 1)
                        __builtin_nontemporal_store(out, (VTS_GLOBAL u32x4*)at);
                    else
                        gstore(at, out);
                }
            }
        }
        if (it < q_end + each) {
            KT own[8], partner[8];
            factors<KT>(p.k_norm, own, partner);
            const uint32_t row = slot_row(p.c.k, page, at), srow = slot_scale(p.c.k_scale, page, at);
#pragma unroll 1
            for (; it < q_end + each; it += p.parts) {
                const int32_t head = (it - q_end) * ROWS + sub;
                const u32x4 raw = load(p.k, p.k_token, p.k_head, head, kv);
                KT y[8];
                turn<KT>(raw, p.k_norm != nullptr, own, partner, y);
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = to_odd(y[i]);
                u32x4 out = {0, 0, 0, 0};
                if (BITS == 16 || p.k_out != nullptr) out = pack8<DT>(x);
                if (!valid) out = u32x4{0, 0, 0, 0};
                if (p.k_out != nullptr && head < kv)
                    gstore((u32x4*)((char*)p.k_out + 2 * ((int64_t)token * kv + head) * D) + c, out);
                store(p.c.k, p.c.k_scale, row, srow, head, kept && head < kv, out, x);
            }
        }
        const uint32_t row = slot_row(p.c.v, page, at), srow = slot_scale(p.c.v_scale, page, at);
#pragma unroll 1
        for (; it < q_end + 2 * each; it += p.parts) {
            const int32_t head = (it - q_end - each) * ROWS + sub;
            const u32x4 raw = load(p.v, p.v_token, p.v_head, head, kv);
            float x[8];
            unpack8<DT>(raw, x);
            store(p.c.v, p.c.v_scale, row, srow, head, kept && head < kv, raw, x);
        }
    }
};

template <int DT, int D, int BITS>
__global__ __launch_bounds__(CACHE_NT) void write_kernel(WriteParams p) {
    const int32_t wave = (int32_t)blockIdx.x * (CACHE_NT / 64) +
                         __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int32_t token = wave / p.parts;
    if (token >= p.tokens) return;
    Writer<DT, D, BITS> w(p, token);
    w.run(wave - token * p.parts);
}

// ---- read

constexpr int READ_EACH = 4;  // chunks of a thread

template <int DT, int D, int BITS>
__global__ __launch_bounds__(CACHE_NT) void read_kernel(ReadParams p) {
    using Raw = typename std::conditional<
        BITS == 16, u32x4, typename std::conditional<BITS == 8, u32x2, uint32_t>::type>::type;
    constexpr int CH = D / 8;
    const int64_t first = (int64_t)blockIdx.x * (CACHE_NT * READ_EACH) + threadIdx.x;
    Raw raw[READ_EACH][2];
    uint32_t code[READ_EACH][2];
    bool there[READ_EACH];
#pragma unroll
    for (int i = 0; i < READ_EACH; ++i) {
        const int64_t x = first + i * CACHE_NT;
        there[i] = false;
        if (x >= p.chunks) continue;
        const int64_t n = x / p.per_slot;
        const int32_t slot = gload(p.slots + n);
        there[i] = slot >= 0 && slot < p.c.num_slots;
        if (!there[i]) continue;
        const int32_t y = (int32_t)(x - n * p.per_slot), head = y / CH, c = y % CH;
        uint32_t page, at;
        slot_place(p.c, slot, page, at);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const CacheView& view = w ? p.c.v : p.c.k;
            const ScaleView& scale = w ? p.c.v_scale : p.c.k_scale;
            const uint32_t row = slot_row(view, page, at) + (uint32_t)head * view.head_stride;
            raw[i][w] = gload((const Raw*)((const char*)view.base + ((uint64_t)row << 4)) + c);
            if constexpr (BITS != 16) {
                const uint32_t srow = slot_scale(scale, page, at) + (uint32_t)head * scale.head_stride;
                code[i][w] = gload(scale.base + (uint64_t)srow * (D / 32) + c / 4);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < READ_EACH; ++i) {
        const int64_t x = first + i * CACHE_NT;
        if (x >= p.chunks) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            u32x4 y = {0, 0, 0, 0};
            if (there[i]) {
                if constexpr (BITS == 16) {
                    y = raw[i][w];
                } else {
                    const float scale = scale_of(code[i][w]);
                    if constexpr (BITS == 8) {
                        y[0] = widen8<DT, false>(raw[i][w][0], scale);
                        y[1] = widen8<DT, true>(raw[i][w][0], scale);
                        y[2] = widen8<DT, false>(raw[i][w][1], scale);
                        y[3] = widen8<DT, true>(raw[i][w][1], scale);
                    } else {
                        y[0] = widen4<DT, 0>(raw[i][w], scale);
                        y[1] = widen4<DT, 1>(raw[i][w], scale);
                        y[2] = widen4<DT, 2>(raw[i][w], scale);
                        y[3] = widen4<DT, 3>(raw[i][w], scale);
                    }
                }
            }
            gstore((u32x4*)(w ? p.v_out : p.k_out) + x, y);
        }
    }
}

// ---- launches

template <int DT, int D, int BITS>
static hipError_t start(const WriteParams& p, hipStream_t stream) {
    const uint32_t waves = (uint32_t)((int64_t)p.tokens * p.parts);
    hipLaunchKernelGGL((write_kernel<DT, D, BITS>), dim3((waves + CACHE_NT / 64 - 1) / (CACHE_NT / 64)),
                       dim3(CACHE_NT), 0, stream, p);
    return hipGetLastError();
}
template <int DT, int D, int BITS>
static hipError_t start(const ReadParams& p, hipStream_t stream) {
    const int64_t each = CACHE_NT * READ_EACH;
    hipLaunchKernelGGL((read_kernel<DT, D, BITS>), dim3((uint32_t)((p.chunks + each - 1) / each)),
                       dim3(CACHE_NT), 0, stream, p);
    return hipGetLastError();
}

template <int DT, int D, class P>
static hipError_t start_bits(int bits, const P& p, hipStream_t stream) {
    switch (bits) {
        case 4: return start<DT, D, 4>(p, stream);
        case 8: return start<DT, D, 8>(p, stream);
    }
    return start<DT, D, 16>(p, stream);
}
template <class P>
static hipError_t start_any(int dtype, int head_dim, int bits, const P& p, hipStream_t stream) {
    if (dtype == BF16)
        return head_dim == 64 ? start_bits<BF16, 64>(bits, p, stream) : start_bits<BF16, 128>(bits, p, stream);
    return head_dim == 64 ? start_bits<F16, 64>(bits, p, stream) : start_bits<F16, 128>(bits, p, stream);
}

hipError_t launch_write(int dtype, int head_dim, int bits, const WriteParams& p, hipStream_t stream) {
    return start_any(dtype, head_dim, bits, p, stream);
}
hipError_t launch_read(int dtype, int head_dim, int bits, const ReadParams& p, hipStream_t stream) {
    return start_any(dtype, head_dim, bits, p, stream);
}

}  // namespace vts
