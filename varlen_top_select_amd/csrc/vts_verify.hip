// vts_verify.hip -- verification of drafted tokens from given random numbers.
//
// At a node with target distribution p and draft distribution q, its children
// are tried in index order; child c, which drafted token x, is accepted if
//   u_c q(x) < r_i(x),    r_0 = p,  r_{i+1} = max(r_i - q, 0) / (its sum),
// i counting the rejected siblings.  In closed form
//   r_i = max(p - a_i q, 0) / S_i,  a_0 = 0, S_0 = 1,
//   a_{i+1} = a_i + S_i,            S_i = sum_v max(p - a_i q, 0),
// so a rejection costs one sum over the vocabulary and no vector is stored.
// Where no child is accepted, the next token is drawn from the residual: the
// first v whose running sum passes u S.  Sums are held in 64 bits: the token is
// a whole number that must not depend on how the sum is split.
//
// Each request has `slices` workgroups.  All of them walk the tree as far as it
// goes without a sum, which is a few dozen scalars and gives all the same
// state, and sum one slice each; the last to arrive joins the sums in order,
// finishes the walk, and scans the one slice that the token lies in.
#include "vts_paged.hpp"

namespace vts {

struct VerifyShared {
    float p[MAX_DRAFT], q[MAX_DRAFT], u[MAX_DRAFT];
    int32_t token[MAX_DRAFT], parent[MAX_DRAFT], path[MAX_DRAFT];
    double sum[WAVES];
    uint32_t last;
    int32_t found;
};

__device__ __forceinline__ float prob(float x) { return x > 0.0f ? x : 0.0f; }  // NaN: 0

template <int DT>
__device__ __forceinline__ float load_prob(const void* row, int64_t i) {
    if constexpr (DT == F32)
        return prob(gload((const float*)row + i));
    else
        return prob(to_float<DT>(gload((const uint16_t*)row + i)));
}

// The walk's state at a node.
struct Walk {
    int32_t cur;      // the last accepted node, -1 at the root
    int32_t next;     // the next node to look at
    int32_t steps;    // accepted so far
    double a, mass;   // of the residual
    uint64_t gone;    // rejected children (chosen drafts: their tokens leave p)
};

template <int DT>
struct Verify {
    const VerifyParams& p;
    VerifyShared& sm;
    const int32_t b;
    const char* target;
    const char* drafts;

    __device__ Verify(const VerifyParams& p_, VerifyShared& s_, int32_t b_)
        : p(p_), sm(s_), b(b_) {
        constexpr int64_t E = DT == F32 ? 4 : 2;
        target = (const char*)p.target + b * p.target_batch * E;
        drafts = p.draft_probs ? (const char*)p.draft_probs + b * p.draft_batch * E : nullptr;
    }
    __device__ __forceinline__ const void* target_row(int32_t cur) const {
        return target + (cur + 1) * p.target_row * (DT == F32 ? 4 : 2);
    }
    __device__ __forceinline__ const void* draft_row(int32_t cur) const {
        return drafts + (cur + 1) * p.draft_row * (DT == F32 ? 4 : 2);
    }

    // what the walk needs of every node: its token's probabilities under its parent
    __device__ __forceinline__ void gather() {
        const int32_t t = threadIdx.x;
        if (t < p.draft) {
            const int64_t at = (int64_t)b * p.draft + t;
            const int32_t x = gload(p.tokens + at);
            int32_t parent = p.parents ? gload(p.parents + at) : t - 1;
            if (parent < -1 || parent >= t) parent = -2;  // no such node: never reached
            const bool ok = parent >= -1 && x >= 0 && x < p.vocab;
            sm.token[t] = ok ? x : -1;
            sm.parent[t] = parent;
            sm.p[t] = ok ? load_prob<DT>(target_row(parent), x) : 0.0f;
            sm.q[t] = !drafts ? 1.0f : ok ? load_prob<DT>(draft_row(parent), x) : 0.0f;
            sm.u[t] = gload(p.uniforms + (int64_t)b * (p.draft + 1) + t);
        }
        __syncthreads();
    }

    // Goes on until a sum is needed (true: a sibling was rejected and the
    // residual has to be summed before the walk goes on) or the walk ends.
    __device__ __forceinline__ bool advance(Walk& k) const {
        for (int32_t t = k.next; t < p.draft; ++t) {
            if (sm.parent[t] != k.cur) continue;
            const double pt = sm.p[t];
            bool yes;
            if (drafts) {
                const double r = fmax(pt - k.a * (double)sm.q[t], 0.0);
                yes = r > 0 && (double)sm.u[t] * (double)sm.q[t] * k.mass < r;
            } else {
                yes = pt > 0 && !is_gone(k.gone, sm.token[t]) && (double)sm.u[t] * k.mass < pt;
            }
            if (yes) {
                if (threadIdx.x == 0) sm.path[k.steps] = t;
                ++k.steps;
                k.cur = t;
                k.a = 0;
                k.mass = 1;
                k.gone = 0;
                continue;
            }
            if (drafts) {
                k.a += k.mass;
                // the sum matters to a later sibling, or to the draw at the end
                k.next = t + 1;
                return true;
            }
            if (!is_gone(k.gone, sm.token[t])) k.mass -= pt;
            k.gone |= 1ull << t;
        }
        k.next = p.draft;
        return false;
    }
    __device__ __forceinline__ bool is_gone(uint64_t gone, int32_t x) const {
        while (gone) {
            const int i = __builtin_ctzll(gone);
            gone &= gone - 1;
            if (sm.token[i] == x) return true;
        }
        return false;
    }

    __device__ __forceinline__ double residual(const Walk& k, const void* pr, const void* qr,
                                               int32_t v) const {
        const double x = load_prob<DT>(pr, v);
        if (k.a > 0) return fmax(x - k.a * (double)load_prob<DT>(qr, v), 0.0);
        return k.gone && is_gone(k.gone, v) ? 0.0 : x;
    }

    __device__ __forceinline__ int32_t slice_begin(int32_t s) const {
        return (int32_t)((int64_t)p.vocab * s / p.slices);
    }

    // The residual's sum over [v0, v1), the same in every thread.
    __device__ __forceinline__ double sum(const Walk& k, int32_t v0, int32_t v1) {
        const void* pr = target_row(k.cur);
        const void* qr = k.a > 0 ? draft_row(k.cur) : nullptr;
        double s = 0;
        for (int32_t v = v0 + (int32_t)threadIdx.x; v < v1; v += NT) s += residual(k, pr, qr, v);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
        __syncthreads();
        if (lane_id() == 0) sm.sum[threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += sm.sum[w];
        return s;
    }

    // First v of [v0, v1) with start + (running sum) > bar; if none, the last v
    // of positive mass, or -1.
    __device__ __forceinline__ int32_t search(const Walk& k, int32_t v0, int32_t v1, double start,
                                              double bar) {
        const void* pr = target_row(k.cur);
        const void* qr = k.a > 0 ? draft_row(k.cur) : nullptr;
        int32_t fallback = -1;
        for (int32_t x0 = v0; x0 < v1; x0 += NT) {
            const int32_t v = x0 + (int32_t)threadIdx.x;
            const double r = v < v1 ? residual(k, pr, qr, v) : 0.0;
            double inc = r;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_up(inc, d);
                if ((int)lane_id() >= d) inc += o;
            }
            __syncthreads();
            if (lane_id() == 63) sm.sum[threadIdx.x >> 6] = inc;
            if (threadIdx.x == 0) sm.found = INT32_MAX, sm.last = 0;
            __syncthreads();
            double before = start;
            for (int w = 0; w < (int)(threadIdx.x >> 6); ++w) before += sm.sum[w];
            if (r > 0 && before + inc > bar) atomicMin(&sm.found, v);
            if (r > 0) atomicMax(&sm.last, (uint32_t)v + 1);
            for (int w = 0; w < WAVES; ++w) start += sm.sum[w];
            __syncthreads();
            if (sm.found != INT32_MAX) return sm.found;
            if (sm.last) fallback = (int32_t)sm.last - 1;
        }
        return fallback;
    }

    __device__ __forceinline__ void run(int32_t slice) {
        gather();
        Walk k;
        k.cur = -1;
        k.next = 0;
        k.steps = 0;
        k.a = 0;
        k.mass = 1;
        k.gone = 0;
        bool more = advance(k);
        if (p.slices > 1) {
            const double mine = sum(k, slice_begin(slice), slice_begin(slice + 1));
            if (threadIdx.x == 0) {
                gstore(p.sums + (int64_t)b * p.slices + slice, mine);
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
                const uint32_t old =
                    __hip_atomic_fetch_add((VTS_GLOBAL uint32_t*)(p.tickets + b), 1u,
                                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                const bool last = old + 1 == (uint32_t)p.slices;
                if (last) {
                    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
                    gstore(p.tickets + b, 0u);  // self-restoring
                }
                sm.last = last;
            }
            __syncthreads();
            if (!sm.last) return;
        }
        // Slice sums of the state at hand, in sums[]; whether they are current.
        double* sums = p.sums + (int64_t)b * p.slices;
        bool current = p.slices > 1;
        double total = 0;
        for (;;) {
            if (!current) {
                for (int32_t s = 0; s < p.slices; ++s) {
                    const double x = sum(k, slice_begin(s), slice_begin(s + 1));
                    if (threadIdx.x == 0) gstore(sums + s, x);
                }
                __syncthreads();
            }
            total = 0;
            for (int32_t s = 0; s < p.slices; ++s) total += gload(sums + s);
            if (!more) break;
            k.mass = total;
            const Walk was = k;
            more = advance(k);
            current = !more && k.cur == was.cur && k.a == was.a;
        }
        if (total == 0 && (k.a > 0 || k.gone)) {  // nothing left of p: draw from p itself
            k.a = 0;
            k.gone = 0;
            __syncthreads();
            for (int32_t s = 0; s < p.slices; ++s) {
                const double x = sum(k, slice_begin(s), slice_begin(s + 1));
                if (threadIdx.x == 0) gstore(sums + s, x);
                total += x;
            }
            __syncthreads();
        }
        const double bar =
            (double)gload(p.uniforms + (int64_t)b * (p.draft + 1) + p.draft) * total;
        int32_t token = -1;
        double start = 0;
        int32_t at = -1;
        double at_start = 0;
        for (int32_t s = 0; s < p.slices; ++s) {  // the slice the running sum passes the bar in
            const double x = gload(sums + s);
            if (x > 0) {
                at = s;
                at_start = start;
                if (start + x > bar) break;
            }
            start += x;
        }
        if (at >= 0) token = search(k, slice_begin(at), slice_begin(at + 1), at_start, bar);
        if (threadIdx.x == 0) {
            gstore(p.token + b, token);
            gstore(p.count + b, k.steps);
        }
        __syncthreads();
        if ((int32_t)threadIdx.x < p.draft)
            gstore(p.path + (int64_t)b * p.draft + threadIdx.x,
                   (int32_t)threadIdx.x < k.steps ? sm.path[threadIdx.x] : -1);
    }
};

template <int DT>
__global__ __launch_bounds__(NT) void verify_kernel(VerifyParams p) {
    __shared__ VerifyShared sm;
    // a request's slices run on the XCDs in turn
    const int32_t b = (int32_t)(blockIdx.x / p.slices), slice = (int32_t)(blockIdx.x % p.slices);
    Verify<DT> v(p, sm, b);
    v.run(slice);
}

hipError_t launch_verify(int dtype, const VerifyParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)p.batch * (uint32_t)p.slices), block(NT);
    switch (dtype) {
        case F32: hipLaunchKernelGGL((verify_kernel<F32>), grid, block, 0, stream, p); break;
        case BF16: hipLaunchKernelGGL((verify_kernel<BF16>), grid, block, 0, stream, p); break;
        default: hipLaunchKernelGGL((verify_kernel<F16>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

}  // namespace vts
