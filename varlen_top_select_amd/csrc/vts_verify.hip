// vts_verify.hip -- verification of drafted tokens from given random numbers.
//
// At a node with target distribution p and draft distribution q, its children
// are tried in index order; child c, which drafted token x, is accepted if
//   u_c q(x) < r_i(x),    r_0 = p,  r_{i+1} = max(r_i - q, 0) / (its sum),
// i counting the rejected siblings.  In closed form
//   r_i = max(p - a_i q, 0) / S_i,  a_0 = 0, S_0 = 1,
//   a_{i+1} = a_i + S_i,            S_i = sum_v max(p - a_i q, 0),
// so a rejection costs one sum over the vocabulary and no vector is stored.  A
// chosen token (q is 1 at it) takes its own p away and leaves the others': r is p
// without the rejected tokens over what they leave.  That is the row's sum
// without any of the node's children, plus the p of those not yet rejected: one
// sum a node, of positive terms only (1 - p of the rejected would be off by the
// row's whole rounding, which in 16 bits passes what a few tokens leave).
// Where no child is accepted, the next token is drawn from the residual: the
// first v whose running sum passes u S.  Sums are held in 64 bits: the token is
// a whole number that must not depend on how the sum is split.
//
// Each request has `slices` workgroups of 16 waves.  All of them walk the tree
// as far as it goes without a sum, which is a few dozen scalars and gives all
// the same state, and every wave sums one segment of the vocabulary; the last
// workgroup to arrive joins the sums in order, finishes the walk, and scans the
// one segment that the token lies in.  A chain needs no other sum, and a tree of
// chosen tokens one for each node where a child was rejected and another follows,
// the later ones by the last workgroup alone (16 trees of 24: 42 us).  In a tree of drawn tokens a rejection's sum decides
// over the next sibling, so there the walk goes in ROUNDS launches that each end
// with a sum by all workgroups, and a last one of one workgroup per request that
// takes what sums are left alone, a sixteenth of the row to a wave (10 us for
// 100003 bf16; with all but the first sum taken so, 16 trees of 24 took 80 us).
#include "vts_paged.hpp"

namespace vts {

constexpr int VT = 1024;  // threads
constexpr int VW = VT / 64;
// launches of a tree's walk that end with a sum by all (16 trees over 100003 bf16:
// of 24 tokens 56 us with 2, 51 with 3, 49 with 5, 52 with 7; of 4 tokens, whose
// walk seldom needs so many, 27, 30, 34 and 37)
constexpr int ROUNDS = 5;

// a 16-byte load from any element's address
typedef u32x4 Unaligned __attribute__((aligned(2)));

struct VerifyShared {
    float p[MAX_DRAFT], q[MAX_DRAFT], u[MAX_DRAFT];
    int32_t token[MAX_DRAFT], parent[MAX_DRAFT], path[MAX_DRAFT];
    double sums[VT];  // of the segments
    double scan[VW];
    uint32_t last;
    int32_t found, tail;
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
    // chosen drafts: once a child was rejected, all children, whose tokens are not
    // in `mass`
    uint64_t gone;
};

// DRAWN: with draft probabilities.  The two walks have kernels of their own: code
// that runs once waits for its own instructions (in one kernel a single chosen
// token takes 17.0 us for 14.9, a drawn tree of 24 57.7 for 48.6).
template <int DT, bool DRAWN>
struct Verify {
    static constexpr int VE = DT == F32 ? 4 : 8;  // elements of a 16-byte vector
    const VerifyParams& p;
    VerifyShared& sm;
    const int32_t b;
    const char* target;
    const char* drafts;

    __device__ Verify(const VerifyParams& p_, VerifyShared& s_, int32_t b_)
        : p(p_), sm(s_), b(b_) {
        constexpr int64_t E = DT == F32 ? 4 : 2;
        target = (const char*)p.target + b * p.target_batch * E;
        drafts = DRAWN ? (const char*)p.draft_probs + b * p.draft_batch * E : nullptr;
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
            sm.q[t] = !DRAWN ? 1.0f : ok ? load_prob<DT>(draft_row(parent), x) : 0.0f;
            sm.u[t] = gload(p.uniforms + (int64_t)b * (p.draft + 1) + t);
        }
        __syncthreads();
    }

    // Goes on until a sum is needed (true: a sibling was rejected, of chosen ones
    // the first, and the residual has to be summed before the walk goes on) or the
    // walk ends.
    __device__ __forceinline__ bool advance(Walk& k) const {
        for (int32_t t = k.next; t < p.draft; ++t) {
            // (where there is no token none was drawn, so nothing leaves the residual)
            if (sm.parent[t] != k.cur || sm.token[t] < 0) continue;
            const double pt = sm.p[t];
            bool yes;
            if constexpr (DRAWN) {
                const double r = fmax(pt - k.a * (double)sm.q[t], 0.0);
                yes = r > 0 && (double)sm.u[t] * (double)sm.q[t] * k.mass < r;
            } else {
                yes = pt > 0 && !is_token_of(before(k.gone, t), sm.token[t]) &&
                      (double)sm.u[t] * left(k, t) < pt;
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
            if constexpr (DRAWN) {
                k.a += k.mass;
                // the sum matters to a later sibling, or to the draw at the end
                k.next = t + 1;
                return true;
            } else {
                if (k.gone) continue;
                for (int32_t c = t; c < p.draft; ++c)
                    if (sm.parent[c] == k.cur && sm.token[c] >= 0) k.gone |= 1ull << c;
                if (k.gone == 1ull << t) break;  // there is no later sibling
                k.next = t + 1;
                return true;
            }
        }
        k.next = p.draft;
        return false;
    }
    static __device__ __forceinline__ uint64_t before(uint64_t nodes, int32_t t) {
        return nodes & ((1ull << t) - 1);
    }
    __device__ __forceinline__ bool is_token_of(uint64_t nodes, int32_t x) const {
        for (; nodes; nodes &= nodes - 1)
            if (sm.token[__builtin_ctzll(nodes)] == x) return true;
        return false;
    }
    // Chosen drafts: the mass that the children before t leave.  Before the first
    // rejection that is the row as it is given; then `mass` and the later
    // children's tokens, each once.
    __device__ __forceinline__ double left(const Walk& k, int32_t t) const {
        double m = k.mass;
        uint64_t seen = before(k.gone, t);
        for (uint64_t g = k.gone & ~seen; g; g &= g - 1) {
            const int i = __builtin_ctzll(g);
            if (!is_token_of(seen, sm.token[i])) m += (double)sm.p[i];
            seen |= 1ull << i;
        }
        return m;
    }

    // A vector of values from element v of a row on, past the vocabulary 0.
    // Rows need no alignment beyond their element's.
    __device__ __forceinline__ void load(const void* row, int32_t v, float (&x)[VE]) const {
        constexpr int E = DT == F32 ? 4 : 2;
        if (v + VE <= p.vocab) {
            const Unaligned w = *(const VTS_GLOBAL Unaligned*)((const VTS_GLOBAL char*)row + (int64_t)v * E);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                if constexpr (DT == F32) {
                    const uint32_t bits = w[i];  // (a bit cast of w[i] itself takes element 0)
                    x[i] = __builtin_bit_cast(float, bits);
                } else
                    x[i] = to_float<DT>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
            }
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] = v + i < p.vocab ? load_prob<DT>(row, v + i) : 0.0f;
        }
    }
    // The residual at elements v .. v + VE - 1.
    struct Pair {
        float x[VE], y[VE];
    };
    __device__ __forceinline__ Pair fetch(const Walk& k, const void* pr, const void* qr,
                                          int32_t v) const {
        Pair f;
        load(pr, v, f.x);
        if (DRAWN && k.a > 0) load(qr, v, f.y);
        return f;
    }
    __device__ __forceinline__ void residual(const Walk& k, const Pair& f, int32_t v,
                                             double (&r)[VE]) const {
        if (DRAWN && k.a > 0) {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                r[i] = fmax((double)f.x[i] - k.a * (double)prob(f.y[i]), 0.0);  // NaN: 0
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) r[i] = prob(f.x[i]);
            if constexpr (!DRAWN)
                for (uint64_t g = k.gone; g; g &= g - 1) {
                    const int32_t x = sm.token[__builtin_ctzll(g)] - v;
#pragma unroll
                    for (int i = 0; i < VE; ++i) r[i] = x == i ? 0.0 : r[i];
                }
        }
    }

    // This wave's lanes' sum over [v0, v1) (v0 a multiple of VE), in every lane.
    __device__ __forceinline__ double wave_sum(const Walk& k, int32_t v0, int32_t v1) const {
        constexpr int U = DT == F32 ? 4 : 2;  // vectors in flight per lane and row
        const void* pr = target_row(k.cur);
        const void* qr = DRAWN && k.a > 0 ? draft_row(k.cur) : nullptr;
        double s = 0;
        for (int32_t v = v0 + (int32_t)lane_id() * VE; v < v1; v += 64 * VE * U) {
            Pair f[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + u * 64 * VE < v1) f[u] = fetch(k, pr, qr, v + u * 64 * VE);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v + u * 64 * VE < v1) {
                    double r[VE];
                    residual(k, f[u], v + u * 64 * VE, r);
#pragma unroll
                    for (int i = 0; i < VE; ++i) s += r[i];
                }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
        return s;
    }

    // Elements per segment when the row is cut in `n`.
    __device__ __forceinline__ int32_t segment(int32_t n) const {
        return ((p.vocab + n - 1) / n + VE - 1) / VE * VE;
    }
    __device__ __forceinline__ double sum_segment(const Walk& k, int32_t n, int32_t g) const {
        const int64_t len = segment(n), v0 = g * len;
        const int64_t v1 = v0 + len < p.vocab ? v0 + len : p.vocab;
        return v0 < v1 ? wave_sum(k, (int32_t)v0, (int32_t)v1) : 0.0;
    }
    // The whole row by this workgroup alone, VW segments.
    __device__ __forceinline__ void sum_alone(const Walk& k) {
        const int wave = threadIdx.x >> 6;
        const double s = sum_segment(k, VW, wave);
        __syncthreads();
        if (lane_id() == 0) sm.sums[wave] = s;
        __syncthreads();
    }

    // Inclusive sums over the workgroup's threads, and the whole.
    __device__ __forceinline__ double block_scan(double v, double& total) {
        double inc = v;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double o = __shfl_up(inc, d);
            if ((int)lane_id() >= d) inc += o;
        }
        const int wave = threadIdx.x >> 6;
        __syncthreads();
        if (lane_id() == 63) sm.scan[wave] = inc;
        __syncthreads();
        double before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            if (w < wave) before += sm.scan[w];
            total += sm.scan[w];
        }
        return before + inc;
    }

    // First v of [v0, v1) with start + (running sum) > bar; if none, the last v
    // of positive mass, or -1.
    __device__ __forceinline__ int32_t search(const Walk& k, int32_t v0, int32_t v1, double start,
                                              double bar) {
        const void* pr = target_row(k.cur);
        const void* qr = DRAWN && k.a > 0 ? draft_row(k.cur) : nullptr;
        int32_t tail = -1;
        for (int32_t x0 = v0; x0 < v1; x0 += VT * VE) {
            const int32_t v = x0 + (int32_t)threadIdx.x * VE;
            double r[VE], s = 0, total;
#pragma unroll
            for (int i = 0; i < VE; ++i) r[i] = 0;
            if (v < v1) residual(k, fetch(k, pr, qr, v), v, r);
#pragma unroll
            for (int i = 0; i < VE; ++i) s += r[i];
            if (threadIdx.x == 0) sm.found = INT32_MAX, sm.tail = -1;
            const double inc = start + block_scan(s, total);
            if (s > 0) {
                if (inc > bar) atomicMin(&sm.found, (int32_t)threadIdx.x);
                int32_t mine = 0;
#pragma unroll
                for (int i = 0; i < VE; ++i) mine = r[i] > 0 ? i : mine;
                atomicMax(&sm.tail, v + mine);
            }
            __syncthreads();
            if (sm.found != INT32_MAX) {
                const bool me = sm.found == (int32_t)threadIdx.x;
                __syncthreads();
                if (me) {
                    double run = inc - s;
                    int32_t at = 0;
                    bool hit = false;
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        run += r[i];
                        if (!hit && r[i] > 0) at = i, hit = run > bar;
                    }
                    sm.found = v + at;
                }
                __syncthreads();
                return sm.found;
            }
            if (sm.tail >= 0) tail = sm.tail;
            start += total;
            __syncthreads();
        }
        return tail;
    }

    static __device__ __forceinline__ Walk root() {
        Walk k;
        k.cur = -1;
        k.next = 0;
        k.steps = 0;
        k.a = 0;
        k.mass = 1;
        k.gone = 0;
        return k;
    }

    __device__ __forceinline__ void run(int32_t slice) {
        gather();
        Walk k = root();
        const bool more = advance(k);
        const int wave = threadIdx.x >> 6;
        const int32_t segments = p.slices * VW;
        if (p.slices > 1) {
            double* sums = p.sums + (int64_t)b * segments;
            const double mine = sum_segment(k, segments, slice * VW + wave);
            if (lane_id() == 0) gstore(sums + slice * VW + wave, mine);
            // every wave's store is complete before the barrier, which does not
            // wait for it; thread 0's release fence then covers the workgroup's
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0);
            asm volatile("" ::: "memory");
            __syncthreads();
            if (threadIdx.x == 0) {
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
            if ((int32_t)threadIdx.x < segments)
                sm.sums[threadIdx.x] = gload(sums + threadIdx.x);
        } else {
            sum_alone(k);
        }
        finish(k, more, segments);
    }

    // Round `r` of the walk: its state and sums come from the round before (of
    // the other parity) and go to the next.
    __device__ __forceinline__ void round(int32_t slice, int32_t r) {
        const int wave = threadIdx.x >> 6;
        const int32_t segments = p.slices * VW;
        Walk k = root();
        bool more;
        VerifyState* to = p.states + 2 * b + (r & 1);
        if (r == 0) {
            gather();
            more = advance(k);
        } else {
            const VerifyState* from = p.states + 2 * b + (~r & 1);
            if (!gload(&from->more)) {  // ended: the state goes on as it is
                if (slice == 0 && threadIdx.x < sizeof(VerifyState) / 4)
                    gstore((uint32_t*)to + threadIdx.x, gload((const uint32_t*)from + threadIdx.x));
                return;
            }
            gather();
            more = load_state(k, from);
            double total;
            block_scan((int32_t)threadIdx.x < segments ? sm.sums[threadIdx.x] : 0.0, total);
            const int32_t cur = k.cur;
            const double a = k.a;
            k.mass = total;
            more = advance(k);
            if (!more && k.cur == cur && k.a == a) {  // ended, with the sums at hand
                if (slice == 0) store_state(k, more, gload(&from->sums), to);
                return;
            }
        }
        double* sums = p.sums + ((int64_t)(r & 1) * p.batch + b) * segments;
        const double mine = sum_segment(k, segments, slice * VW + wave);
        if (lane_id() == 0) gstore(sums + slice * VW + wave, mine);
        if (slice == 0) store_state(k, more, r & 1, to);
    }
    __device__ __forceinline__ void last_round(int32_t rounds) {
        gather();
        Walk k = root();
        const bool more = load_state(k, p.states + 2 * b + (~rounds & 1));
        finish(k, more, p.slices * VW);
    }
    __device__ __forceinline__ bool load_state(Walk& k, const VerifyState* from) {
        k.cur = gload(&from->cur);
        k.next = gload(&from->next);
        k.steps = gload(&from->steps);
        k.a = gload(&from->a);
        k.mass = gload(&from->mass);
        if (threadIdx.x < MAX_DRAFT) sm.path[threadIdx.x] = gload(from->path + threadIdx.x);
        const int32_t segments = p.slices * VW;
        const double* sums = p.sums + ((int64_t)gload(&from->sums) * p.batch + b) * segments;
        if ((int32_t)threadIdx.x < segments) sm.sums[threadIdx.x] = gload(sums + threadIdx.x);
        __syncthreads();
        return gload(&from->more) != 0;
    }
    __device__ __forceinline__ void store_state(const Walk& k, bool more, int32_t sums,
                                                VerifyState* to) {
        __syncthreads();
        if (threadIdx.x < MAX_DRAFT) gstore(to->path + threadIdx.x, sm.path[threadIdx.x]);
        if (threadIdx.x == 0) {
            gstore(&to->cur, k.cur);
            gstore(&to->next, k.next);
            gstore(&to->steps, k.steps);
            gstore(&to->more, more ? 1 : 0);
            gstore(&to->sums, sums);
            gstore(&to->a, k.a);
            gstore(&to->mass, k.mass);
        }
    }

    // From the sums of the state at hand (`segments` of them in sm.sums) to the
    // outputs.
    __device__ __forceinline__ void finish(Walk k, bool more, int32_t segments) {
        double total, inc;
        for (;;) {
            __syncthreads();
            inc = block_scan((int32_t)threadIdx.x < segments ? sm.sums[threadIdx.x] : 0.0, total);
            if (more) {
                const int32_t cur = k.cur;
                const double a = k.a;
                k.mass = total;
                more = advance(k);
                if (!more && k.cur == cur && k.a == a) continue;  // the same residual
            } else if (total == 0 && (k.a > 0 || k.gone)) {
                k.a = 0;  // nothing is left of p: draw from p itself
                k.gone = 0;
            } else {
                break;
            }
            sum_alone(k);
            segments = VW;
        }
        const double bar =
            (double)gload(p.uniforms + (int64_t)b * (p.draft + 1) + p.draft) * total;
        // the first segment whose running sum passes the bar, or the last of any mass
        const double x = (int32_t)threadIdx.x < segments ? sm.sums[threadIdx.x] : 0.0;
        if (threadIdx.x == 0) sm.found = INT32_MAX, sm.tail = -1;
        __syncthreads();
        if (x > 0) {
            if (inc > bar) atomicMin(&sm.found, (int32_t)threadIdx.x);
            atomicMax(&sm.tail, (int32_t)threadIdx.x);
        }
        __syncthreads();
        const int32_t at = sm.found != INT32_MAX ? sm.found : sm.tail;
        if ((int32_t)threadIdx.x == at) sm.scan[0] = inc - x;
        __syncthreads();
        int32_t token = -1;
        if (at >= 0) {
            const double start = sm.scan[0];
            const int64_t len = segment(segments), v0 = at * len;
            const int64_t v1 = v0 + len < p.vocab ? v0 + len : p.vocab;
            token = search(k, (int32_t)v0, (int32_t)v1, start, bar);
        }
        if (threadIdx.x == 0) {
            gstore(p.token + b, token);
            gstore(p.count + b, k.steps);
        }
        if ((int32_t)threadIdx.x < p.draft)
            gstore(p.path + (int64_t)b * p.draft + threadIdx.x,
                   (int32_t)threadIdx.x < k.steps ? sm.path[threadIdx.x] : -1);
    }
};

template <int DT, bool DRAWN>
__global__ __launch_bounds__(VT) void verify_kernel(VerifyParams p) {
    __shared__ VerifyShared sm;
    const int32_t b = (int32_t)(blockIdx.x / p.slices), slice = (int32_t)(blockIdx.x % p.slices);
    Verify<DT, DRAWN> v(p, sm, b);
    v.run(slice);
}

template <int DT>
__global__ __launch_bounds__(VT) void verify_round_kernel(VerifyParams p, int32_t r) {
    __shared__ VerifyShared sm;
    const int32_t b = (int32_t)(blockIdx.x / p.slices), slice = (int32_t)(blockIdx.x % p.slices);
    Verify<DT, true> v(p, sm, b);
    v.round(slice, r);
}

template <int DT>
__global__ __launch_bounds__(VT) void verify_last_kernel(VerifyParams p, int32_t rounds) {
    __shared__ VerifyShared sm;
    Verify<DT, true> v(p, sm, (int32_t)blockIdx.x);
    v.last_round(rounds);
}

template <int DT>
static hipError_t launch_dt(const VerifyParams& p, hipStream_t stream) {
    const dim3 grid((uint32_t)p.batch * (uint32_t)p.slices), block(VT);
    // a drawn token's rejected siblings make the walk wait for a sum each
    if (!p.draft_probs || !p.parents || p.draft == 1 || p.slices == 1) {
        if (p.draft_probs)
            hipLaunchKernelGGL((verify_kernel<DT, true>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((verify_kernel<DT, false>), grid, block, 0, stream, p);
        return hipGetLastError();
    }
    for (int32_t r = 0; r < ROUNDS; ++r)
        hipLaunchKernelGGL((verify_round_kernel<DT>), grid, block, 0, stream, p, r);
    hipLaunchKernelGGL((verify_last_kernel<DT>), dim3((uint32_t)p.batch), block, 0, stream, p,
                       ROUNDS);
    return hipGetLastError();
}

hipError_t launch_verify(int dtype, const VerifyParams& p, hipStream_t stream) {
    switch (dtype) {
        case F32: return launch_dt<F32>(p, stream);
        case BF16: return launch_dt<BF16>(p, stream);
    }
    return launch_dt<F16>(p, stream);
}

}  // namespace vts
