// logprob.hip -- log probabilities of given tokens under rows of logits, with the logarithm of the
// sum, the entropy and the likeliest tokens, and their gradient:
//   lse = log sum exp(scale x),   logprob = scale x_t - lse,   H = lse - sum p scale x
//   dx_j = scale (dlogprob (1[j = t] - p_j) + dlse p_j - dH p_j (log p_j + H))
// One pass over a row keeps its running maximum m, s = sum e^(d) and w = sum e^d d with
// d = scale (x - m) (in base 2): the difference is taken before the scale, so that rows of the
// type's lowest value neither overflow nor vanish, and m starts at the lowest finite value, so
// that a row of -inf ends with s = 0 (probabilities 0, no entropy, no gradient).
//
// HBM bounds it: one read forward, one read and one write backward, against about 12 and 14 VALU
// slots per element, 4 of them the exp.
//
// The likeliest tokens, by value and then by index: about the k / 4-th largest of a wavefront's
// lane maxima is reached by k / 4 of its elements, so that k elements of the block's reach the
// least of its 4 wavefronts' bounds.  The row's second reading (from the caches, or registers)
// keeps only the elements at or above it, less than 2 k of them as a rule, and each kept element's
// rank is counted. (Bounds that k elements of one wavefront reach, the largest of them taken, keep
// some 5 k of them for k = 20 and 1000 for k = 64.)  Rows with more ties than the list holds are
// searched once per token, and so are rows whose mask leaves fewer lanes with a token than the
// bound needs, since all masked columns tie (64 x 50257 fp32 with 40 tokens left, kernels: 20
// likeliest 43 us, 15 without a mask; 64 likeliest 110).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block_kernels.hpp"
#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

constexpr float kLowest = -3.402823466e38f;
// A scale for powers of 2; finite for every finite scale, since it multiplies differences of 0.
__device__ __forceinline__ float base2(float scale) { return fminf(scale * kLog2e, -kLowest); }
constexpr int kThreads = 256;
constexpr int kCandidates = 1024;
constexpr unsigned kMaxBlocks = 1u << 22;  // a grid has fewer than 2^32 threads
// beyond it an fp32 lse has fewer than 13 bits behind the point: the backward sums the row again
constexpr float kBigLse = 1024.0f;

// ---- reductions over teams of 4, 16 or 64 lanes ----------------------------------------------

constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int TEAM, typename Op>
__device__ __forceinline__ float team_reduce(float v, Op op) {
    v = op(v, dpp<kQuadXor1, 0xf>(v, v));
    v = op(v, dpp<kQuadXor2, 0xf>(v, v));
    if constexpr (TEAM >= 16) {
        v = op(v, dpp<kHalfMirror, 0xf>(v, v));
        v = op(v, dpp<kMirror, 0xf>(v, v));
    }
    if constexpr (TEAM >= 64) {
        v = op(v, __shfl_xor(v, 16));
        v = op(v, __shfl_xor(v, 32));
    }
    return v;
}
struct Max {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Add {
    __device__ float operator()(float a, float b) const { return a + b; }
};

// Keys in the order of the tokens: by value (a NaN first, the zeros equal), then the lowest index.
// No key is ~0, which stands above all of them.
typedef unsigned long long Key;
constexpr uint32_t kNanKey = 0xfffffffeu;
__device__ __forceinline__ Key key_of(float x, int col) {
    uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
    u = x != x ? kNanKey : (u ^ (u >> 31 ? 0xffffffffu : 0x80000000u));
    return (static_cast<Key>(u) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ int col_of(Key k) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k));
}
__device__ __forceinline__ float value_of(Key k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    if (u == kNanKey) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ Key shfl_xor_key(Key k, int m) {
    const uint32_t lo = __shfl_xor(static_cast<uint32_t>(k), m);
    const uint32_t hi = __shfl_xor(static_cast<uint32_t>(k >> 32), m);
    return (static_cast<Key>(hi) << 32) | lo;
}
template <int TEAM>
__device__ __forceinline__ Key team_max_key(Key k) {
#pragma unroll
    for (int m = 1; m < TEAM; m *= 2) {
        const Key o = shfl_xor_key(k, m);
        k = o > k ? o : k;
    }
    return k;
}

// ---- a row's sums ------------------------------------------------------------------------------

// max is the row's largest value itself (-inf if it has no other); m, where the sums stand, is at
// least the lowest finite value.
struct Sums {
    float max, s, w;
    __device__ __forceinline__ float m() const { return fmaxf(max, kLowest); }
};

// e^d and e^d d, both 0 far below (where d may be -inf); a NaN stays.
__device__ __forceinline__ void add_term(float x, float m, float k2, float& s, float& w) {
    const float d = (x - m) * k2;
    const float e = exp2_hw(d);
    s += e;
    w = fmaf(e, fmaxf(d, -200.0f), w);
}

// The sums moved to stand at m.  Rounded as they are written: fused with the first addition of a
// reduction over lanes, the products would round differently in each of two lanes that add theirs.
__device__ __forceinline__ void rebase(Sums& a, float m, float k2) {
#pragma clang fp contract(off)
    const float d = (a.m() - m) * k2;
    const float c = exp2_hw(d);
    a.w = c * fmaf(a.s, fmaxf(d, -200.0f), a.w);
    a.s *= c;
}

__device__ __forceinline__ Sums join(Sums a, Sums b, float k2) {
    const float top = fmaxf(a.max, b.max), m = fmaxf(top, kLowest);
    rebase(a, m, k2);
    rebase(b, m, k2);
    return {top, a.s + b.s, a.w + b.w};
}

__device__ __forceinline__ Sums wave_join(Sums a, float k2) {
    const float top = team_reduce<64>(a.max, Max());
    rebase(a, fmaxf(top, kLowest), k2);
    return {top, team_reduce<64>(a.s, Add()), team_reduce<64>(a.w, Add())};
}

// What a row's sums give.
struct RowOut {
    float m, log_s, lse, entropy;
    bool dead;
    __device__ __forceinline__ RowOut(const Sums& t, float scale) {
        m = t.m();
        dead = t.s == 0.0f;
        log_s = logf(t.s);
        lse = dead ? -INFINITY : fmaf(m, scale, log_s);
        entropy = dead ? 0.0f : log_s - kLn2 * t.w / t.s;
    }
    __device__ __forceinline__ float logprob(float x, float scale) const {
        return dead ? -INFINITY : fmaf(x - m, scale, -log_s);
    }
};

// The token asked for in a row, -1 where there is none in range.
__device__ __forceinline__ int token_of(const void* ids, int ids64, int64_t row, int64_t rows,
                                        int V) {
    if (ids == nullptr) return -1;
    const int64_t at = MSEL_IDX(row, rows);
    const int64_t t = ids64 ? static_cast<const int64_t*>(ids)[at]
                            : static_cast<const int32_t*>(ids)[at];
    return t >= 0 && t < V ? static_cast<int>(t) : -1;
}

template <typename T>
__device__ __forceinline__ void write_row(const LogprobParams& p, const T* row, int64_t r,
                                          const RowOut& o) {
    if (p.lse != nullptr) p.lse[MSEL_IDX(r, p.rows)] = o.lse;
    if (p.entropy != nullptr) p.entropy[MSEL_IDX(r, p.rows)] = o.entropy;
    if (p.logprob != nullptr) {
        const int t = token_of(p.ids, p.ids64, r, p.rows, p.V);
        const float x = t >= 0 ? Elem<T>::load1(row + MSEL_IDX(t, p.V)) : 0.0f;
        p.logprob[MSEL_IDX(r, p.rows)] = t >= 0 ? o.logprob(x, p.scale) : 0.0f;
    }
}

__device__ __forceinline__ void write_top(const LogprobParams& p, int64_t r, int rank, Key k,
                                          const RowOut& o) {
    const int64_t at = MSEL_IDX(r * p.top + rank, p.rows * p.top);
    p.top_ids[at] = col_of(k);
    p.top_logprobs[at] = o.logprob(value_of(k), p.scale);
}

// ---- narrow rows: TEAM lanes hold a row in registers, N vectors each ----------------------------

template <typename T, int TEAM, int NV>
struct NarrowRow {
    static constexpr int VE = 16 / static_cast<int>(sizeof(T));
    static constexpr int N = NV;
    float x[N * VE];  // columns past the end are -inf
    __device__ __forceinline__ static int col(int l, int k) {
        return ((k / VE) * TEAM + l) * VE + k % VE;
    }
    __device__ __forceinline__ NarrowRow(const T* row, int l, int V) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = (j * TEAM + l) * VE;
            float v[VE];
#pragma unroll
            for (int k = 0; k < VE; ++k) v[k] = -INFINITY;
            if (c + VE <= V) {
                to_f32<T, VE>(ld_raw<T, VE>(row + MSEL_SPAN(c, VE, V)), v);
            } else if (c < V) {
#pragma unroll
                for (int k = 0; k < VE; ++k)
                    if (c + k < V) v[k] = Elem<T>::load1(row + c + k);
            }
#pragma unroll
            for (int k = 0; k < VE; ++k) x[j * VE + k] = v[k];
        }
    }
    __device__ __forceinline__ Sums sums(float k2) const {
        float m = x[0];
#pragma unroll
        for (int k = 1; k < N * VE; ++k) m = fmaxf(m, x[k]);
        Sums t{team_reduce<TEAM>(m, Max()), 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < N * VE; ++k) add_term(x[k], t.m(), k2, t.s, t.w);
        t.s = team_reduce<TEAM>(t.s, Add());
        t.w = team_reduce<TEAM>(t.w, Add());
        return t;
    }
};

template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(kThreads) void narrow_fwd_kernel(LogprobParams p) {
    using Row = NarrowRow<T, TEAM, NV>;
    const int l = threadIdx.x % TEAM;
    const float k2 = base2(p.scale);
    constexpr int kTeams = kThreads / TEAM;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kTeams; r0 < p.rows;
         r0 += static_cast<int64_t>(gridDim.x) * kTeams) {
        const int64_t mine = r0 + threadIdx.x / TEAM;
        const bool live = mine < p.rows;
        const int64_t r = live ? mine : p.rows - 1;  // lanes without a row repeat the last one
        const T* row = static_cast<const T*>(p.logits) + MSEL_IDX(r, p.rows) * p.stride;
        const Row v(row, l, p.V);
        const RowOut o(v.sums(k2), p.scale);
        if (live && l == 0) write_row<T>(p, row, r, o);
        Key below = ~Key(0);  // a rank's key is the largest one below the rank's before
        for (int k = 0; k < p.top; ++k) {
            Key best = 0;
#pragma unroll
            for (int j = 0; j < Row::N * Row::VE; ++j) {
                const int c = Row::col(l, j);
                const Key q = key_of(v.x[j], c);
                if (c < p.V && q < below && q > best) best = q;
            }
            below = team_max_key<TEAM>(best);
            if (live && l == 0) write_top(p, r, k, below, o);
        }
    }
}

// What the gradient of a row needs.
struct RowGrad {
    float lse, cp, ch, h, dt, k2;  // p = 2^(x k2 - lse); dx = scale (p (cp - ch (log p + h)) + dt)
    float m;                       // with the sums formed again: p = 2^((x - m) k2 - lse)
    int t;
    bool dead;
    __device__ __forceinline__ RowGrad(const LogprobParams& p, int64_t r) {
        t = token_of(p.ids, p.ids64, r, p.rows, p.V);
        const int64_t at = MSEL_IDX(r, p.rows);
        dt = t >= 0 && p.dlogprob != nullptr ? p.dlogprob[at] : 0.0f;
        cp = (p.dlse != nullptr ? p.dlse[at] : 0.0f) - dt;
        ch = p.dentropy != nullptr ? p.dentropy[at] : 0.0f;
        h = p.dentropy != nullptr ? p.in_entropy[at] : 0.0f;
        k2 = base2(p.scale);
        m = 0.0f;
        lse = p.in_lse[at] * kLog2e;
        dead = false;
    }
    __device__ __forceinline__ bool again() const { return !(fabsf(lse) < kBigLse * kLog2e); }
    __device__ __forceinline__ void stand_at(const Sums& s) {
        m = s.m();
        lse = log2_hw(s.s);
        dead = s.s == 0.0f;
    }
    __device__ __forceinline__ float at(float x, float scale) const {
        const float lp = fmaf(x - m, k2, -lse);
        const float e = exp2_hw(lp);
        return scale * e * fmaf(-ch, fmaf(fmaxf(lp, -200.0f), kLn2, h), cp);
    }
};

template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(kThreads) void narrow_bwd_kernel(LogprobParams p) {
    using Row = NarrowRow<T, TEAM, NV>;
    constexpr int VE = Row::VE;
    constexpr int kTeams = kThreads / TEAM;
    const int l = threadIdx.x % TEAM;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kTeams; r0 < p.rows;
         r0 += static_cast<int64_t>(gridDim.x) * kTeams) {
        const int64_t mine = r0 + threadIdx.x / TEAM;
        const bool live = mine < p.rows;
        const int64_t r = live ? mine : p.rows - 1;
        const Row v(static_cast<const T*>(p.logits) + MSEL_IDX(r, p.rows) * p.stride, l, p.V);
        RowGrad g(p, r);
        if (__ballot(g.again()) != 0) {  // whole wavefronts: the teams' lanes are all there
            const Sums s = v.sums(g.k2);
            if (g.again()) g.stand_at(s);
        }
        T* out = static_cast<T*>(p.dlogits) + MSEL_IDX(r, p.rows) * p.dstride;
#pragma unroll
        for (int j = 0; j < Row::N; ++j) {
            const int c = (j * TEAM + l) * VE;
            float d[VE];
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                d[k] = g.at(v.x[j * VE + k], p.scale);
                if (c + k == g.t) d[k] = fmaf(g.dt, p.scale, d[k]);
                if (g.dead) d[k] = 0.0f;
            }
            if (live && c < p.V) {
                const RawVec<T, VE> q = from_f32<T, VE>(d);
                if (c + VE <= p.V)
                    st_raw<T, VE>(out + MSEL_SPAN(c, VE, p.V), q);
                else
                    st_part<T, VE>(out + c, q, p.V - c);
            }
        }
    }
}

// ---- wide rows: a block per row, or per slice of one -------------------------------------------

constexpr int kUnroll = 4;

// Columns before c0 of the line of 128 bytes that c0 lies in: the vectors start with it, since a
// wavefront's vectors across the lines of an odd row take one line more each (16384 rows of 50257
// in bf16: 352 us forward, 286 with this).
template <typename T>
__device__ __forceinline__ int before_line(const T* row, int c0) {
    return static_cast<int>((reinterpret_cast<uintptr_t>(row + c0) & 127) / sizeof(T));
}

// The values of a vector's columns in [c0, c1), -inf in place of others.
template <typename T, int VE>
__device__ __forceinline__ RawVec<T, VE> ld_between(const T* row, int c, int c0, int c1) {
    if (c >= c0 && c + VE <= c1) return ld_raw<T, VE>(row + MSEL_SPAN(c, VE, c1));
    float v[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k)
        v[k] = c + k >= c0 && c + k < c1 ? Elem<T>::load1(row + c + k) : -INFINITY;
    return from_f32<T, VE>(v);
}

// Calls each(x values of some vectors, first column, columns from a vector to the next, number of
// vectors) for the vectors of columns [c0, c1) that are this thread's, kUnroll of them loaded at
// once.  Columns outside are -inf.
template <typename T, typename Fn>
__device__ __forceinline__ void each_vector(const T* row, int c0, int c1, Fn each) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int kRound = kThreads * VE;
    int c = c0 - before_line(row, c0) + static_cast<int>(threadIdx.x) * VE;
    const auto one = [&] {
        float v[VE];
        to_f32<T, VE>(ld_between<T, VE>(row, c, c0, c1), v);
        each(v, c, kRound, std::integral_constant<int, 1>());
        c += kRound;
    };
    if (c < c0) {
        if (c + VE > c0)
            one();
        else
            c += kRound;
    }
    for (; c + (kUnroll - 1) * kRound + VE <= c1; c += kUnroll * kRound) {
        RawVec<T, VE> raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            raw[u] = ld_raw<T, VE>(row + MSEL_SPAN(c + u * kRound, VE, c1));
        float v[kUnroll * VE];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float x[VE];
            to_f32<T, VE>(raw[u], x);
#pragma unroll
            for (int k = 0; k < VE; ++k) v[u * VE + k] = x[k];
        }
        each(v, c, kRound, std::integral_constant<int, kUnroll>());
    }
    while (c < c1) one();
}

// The terms of some values added to sums that may have to be moved for them.
template <bool ENTROPY, typename V>
__device__ __forceinline__ void add_vector(Sums& t, const V& v, float k2) {
    constexpr int n = sizeof(v) / sizeof(v[0]);
    float m = v[0];
#pragma unroll
    for (int k = 1; k < n; ++k) m = fmaxf(m, v[k]);
    if (m > t.max) {
        rebase(t, fmaxf(m, kLowest), k2);
        t.max = m;
    }
    const float at = t.m();
#pragma unroll
    for (int k = 0; k < n; ++k) {
        if constexpr (ENTROPY)
            add_term(v[k], at, k2, t.s, t.w);
        else
            t.s += exp2_hw((v[k] - at) * k2);
    }
}

// A thread's sums over its columns.
template <typename T, bool ENTROPY>
__device__ __forceinline__ Sums thread_sums(const T* row, int c0, int c1, float k2) {
    Sums t{-INFINITY, 0.0f, 0.0f};
    each_vector<T>(row, c0, c1,
                   [&](const auto& v, int, int, auto) { add_vector<ENTROPY>(t, v, k2); });
    return t;
}

// Joined over the block, in every thread; part: one per wavefront.
__device__ __forceinline__ Sums block_join(const Sums& mine, float k2, Sums* part) {
    const Sums w = wave_join(mine, k2);
    if (lane_id() == 0) part[threadIdx.x >> 6] = w;
    __syncthreads();
    Sums t = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) t = join(t, part[i], k2);
    __syncthreads();
    return t;
}

// The upper half of a key that at least k lanes of the wavefront reach: the k-th largest value's,
// cut to its sign, exponent and 7 bits.
__device__ __forceinline__ uint32_t kth_of_lanes(float v, int k) {
    const uint32_t u = static_cast<uint32_t>(key_of(v, 0) >> 32);
    uint32_t t = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t c = t | (1u << bit);
        if (__popcll(__ballot(u >= c)) >= k) t = c;
    }
    return t;
}

struct TopList {
    Key keys[kCandidates];
    uint32_t bound[kThreads / 64];
    Key best[kThreads / 64];
    int count;
};

// The `top` largest keys of columns [c0, c1), handed to put(rank, key); c1 - c0 >= top.  each:
// calls its argument for this thread's vectors, as each_vector does.  mx: the largest value among
// them.
template <int VE, typename Each, typename Put>
__device__ __forceinline__ void block_top(Each each, int c0, int c1, int top, float mx,
                                          TopList& list, Put put) {
    const int wave = threadIdx.x >> 6;
    constexpr int kWaves = kThreads / 64;
    // for a few the largest bound that all of them reach in one wavefront is as good, with fewer
    // kept
    const bool few = top <= kWaves;
    const uint32_t kth = kth_of_lanes(mx, few ? top : (top + kWaves - 1) / kWaves);
    if (lane_id() == 0) list.bound[wave] = kth;
    if (threadIdx.x == 0) list.count = 0;
    __syncthreads();
    uint32_t key = list.bound[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) key = few ? max(key, list.bound[i]) : min(key, list.bound[i]);
    // below -inf, where that is the k-th largest, it is a NaN, which every value passes
    const float bound = __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
    each([&](const auto& v, int c, int round, auto) {
        constexpr int n = sizeof(v) / sizeof(v[0]);
        bool any = false;
#pragma unroll
        for (int k = 0; k < n; ++k) any = any || !(v[k] < bound);
        if (!any) return;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const int col = c + (k / VE) * round + k % VE;
            if (v[k] < bound || col < c0 || col >= c1) continue;
            const int at = atomicAdd(&list.count, 1);
            if (at < kCandidates) list.keys[MSEL_IDX(at, kCandidates)] = key_of(v[k], col);
        }
    });
    __syncthreads();
    const int n = list.count;
    if (n <= kCandidates) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const Key mine = list.keys[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) rank += list.keys[j] > mine;
            if (rank < top) put(rank, mine);
        }
        return;
    }
    Key below = ~Key(0);
    for (int k = 0; k < top; ++k) {
        Key best = 0;
        each([&](const auto& v, int c, int round, auto) {
            constexpr int m = sizeof(v) / sizeof(v[0]);
#pragma unroll
            for (int j = 0; j < m; ++j) {
                const int col = c + (j / VE) * round + j % VE;
                const Key q = key_of(v[j], col);
                if (col >= c0 && col < c1 && q < below && q > best) best = q;
            }
        });
        best = team_max_key<64>(best);
        if (lane_id() == 0) list.best[wave] = best;
        __syncthreads();
        below = list.best[0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) below = max(below, list.best[i]);
        if (threadIdx.x == 0) put(k, below);
        __syncthreads();
    }
}

// The workspace of sliced rows: per (row, slice) its sums, then per (row, slice) its top keys.
__host__ __device__ inline size_t sums_bytes(int64_t rows, int slices) {
    return (static_cast<size_t>(rows) * slices * sizeof(Sums) + 255) / 256 * 256;
}

// What a block has of a (row, slice): to the outputs, or to the slice's part of the workspace.
template <typename T, bool TOP, typename Each>
__device__ __forceinline__ void finish(const LogprobParams& p, const T* row, int64_t u, int64_t r,
                                       int c0, int c1, float mx, const Sums& all, TopList* list,
                                       Each each) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    [[maybe_unused]] const int64_t units = p.rows * p.slices;
    if (p.slices > 1) {
        if (threadIdx.x == 0) static_cast<Sums*>(p.ws)[MSEL_IDX(u, units)] = all;
        if constexpr (TOP) {
            Key* keys = reinterpret_cast<Key*>(static_cast<char*>(p.ws) +
                                               sums_bytes(p.rows, p.slices));
            block_top<VE>(each, c0, c1, p.top, mx, *list, [&](int rank, Key k) {
                keys[MSEL_IDX(u * p.top + rank, units * p.top)] = k;
            });
        }
    } else {
        const RowOut o(all, p.scale);
        if (threadIdx.x == 0) write_row<T>(p, row, r, o);
        if constexpr (TOP)
            block_top<VE>(each, c0, c1, p.top, mx, *list,
                          [&](int rank, Key k) { write_top(p, r, rank, k, o); });
    }
}

template <typename T, bool ENTROPY, bool TOP>
__global__ __launch_bounds__(kThreads) void wide_fwd_kernel(LogprobParams p) {
    __shared__ Sums part[kThreads / 64];
    __shared__ typename std::conditional<TOP, TopList, char>::type list;
    const float k2 = base2(p.scale);
    const int64_t units = p.rows * p.slices;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t r = p.slices == 1 ? u : u / p.slices;
        const int q = static_cast<int>(u - r * p.slices);
        const T* row = static_cast<const T*>(p.logits) + MSEL_IDX(r, p.rows) * p.stride;
        const int c0 = q * p.slice, c1 = min(p.V, c0 + p.slice);
        const Sums mine = thread_sums<T, ENTROPY>(row, c0, c1, k2);
        const Sums all = block_join(mine, k2, part);
        finish<T, TOP>(p, row, u, r, c0, c1, mine.max, all, reinterpret_cast<TopList*>(&list),
                       [&](auto fn) { each_vector<T>(row, c0, c1, fn); });
        __syncthreads();  // the list is the next row's too
    }
}

// Slices of up to kHeld columns stay in registers: loaded at once, and read once (64 rows of 50257
// in fp32 with 20 likeliest tokens: 17 us in two readings).
constexpr int kHeldCols = 8192, kHeld = kHeldCols - 64;  // 64: what may lie before a line

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void held_fwd_kernel(LogprobParams p) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    constexpr int kRound = kThreads * VE, N = kHeldCols / kRound;
    __shared__ Sums part[kThreads / 64];
    __shared__ typename std::conditional<TOP, TopList, char>::type list;
    const float k2 = base2(p.scale);
    const int64_t units = p.rows * p.slices;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t r = p.slices == 1 ? u : u / p.slices;
        const int q = static_cast<int>(u - r * p.slices);
        const T* row = static_cast<const T*>(p.logits) + MSEL_IDX(r, p.rows) * p.stride;
        const int c0 = q * p.slice, c1 = min(p.V, c0 + p.slice);
        const int c = c0 - before_line(row, c0) + static_cast<int>(threadIdx.x) * VE;
        RawVec<T, VE> raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = ld_between<T, VE>(row, c + i * kRound, c0, c1);
        const auto each = [&](auto fn) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float v[VE];
                to_f32<T, VE>(raw[i], v);
                const int col = c + i * kRound;
                if (col < c1) fn(v, col, kRound, std::integral_constant<int, 1>());
            }
        };
        Sums mine{-INFINITY, 0.0f, 0.0f};
        each([&](const auto& v, int, int, auto) {
#pragma unroll
            for (int k = 0; k < VE; ++k) mine.max = fmaxf(mine.max, v[k]);
        });
        const float at = mine.m();
        each([&](const auto& v, int, int, auto) {
#pragma unroll
            for (int k = 0; k < VE; ++k) add_term(v[k], at, k2, mine.s, mine.w);
        });
        const Sums all = block_join(mine, k2, part);
        finish<T, TOP>(p, row, u, r, c0, c1, mine.max, all, reinterpret_cast<TopList*>(&list),
                       each);
        __syncthreads();
    }
}

// The slices of a row joined, a block per row.  Up to kCandidates keys, of which those count that
// reach the least of the slices' (top / slices)-th keys, as top of them do (64 likeliest of 8 rows
// of 50257 in fp32: 58 us with all of them ranked).
template <typename T>
__global__ __launch_bounds__(kThreads) void join_kernel(LogprobParams p) {
    const float k2 = base2(p.scale);
    const Sums* parts = static_cast<const Sums*>(p.ws);
    const Key* keys = reinterpret_cast<const Key*>(static_cast<const char*>(p.ws) +
                                                   sums_bytes(p.rows, p.slices));
    __shared__ Key held[kCandidates];
    __shared__ int count;
    const int n = p.slices * p.top, each = (p.top + p.slices - 1) / p.slices;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        Sums t{-INFINITY, 0.0f, 0.0f};
        Key bound = ~Key(0);
        if (lane_id() < p.slices) {
            t = parts[MSEL_IDX(r * p.slices + lane_id(), p.rows * p.slices)];
            if (n > 0) bound = keys[MSEL_IDX(r * n + lane_id() * p.top + each - 1, p.rows * n)];
        }
        Key mine[kCandidates / kThreads];
#pragma unroll
        for (int i = 0; i < kCandidates / kThreads; ++i) {
            const int at = i * kThreads + static_cast<int>(threadIdx.x);
            mine[i] = at < n ? keys[MSEL_IDX(r * n + at, p.rows * n)] : Key(0);
        }
        bound = ~team_max_key<64>(~bound);  // the least
        if (threadIdx.x == 0) count = 0;
        const RowOut o(wave_join(t, k2), p.scale);
        if (threadIdx.x == kThreads - 1)
            write_row<T>(p, static_cast<const T*>(p.logits) + MSEL_IDX(r, p.rows) * p.stride, r, o);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kCandidates / kThreads; ++i)
            if (i * kThreads + static_cast<int>(threadIdx.x) < n && mine[i] >= bound)
                held[MSEL_IDX(atomicAdd(&count, 1), kCandidates)] = mine[i];
        __syncthreads();
        const int kept = count;
        for (int i = threadIdx.x; i < kept; i += kThreads) {
            const Key key = held[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < kept; ++j) rank += held[j] > key;
            if (rank < p.top) write_top(p, r, rank, key, o);
        }
        __syncthreads();
    }
}

// A block per (row, slice); slices > 1 only where the gradient goes to memory of its own, since a
// row that is summed again is read whole before it is written (64 x 50257 fp32: 7.8 us, in place
// 17; 512 x 50257 bf16: 21 and 22).
template <typename T, bool PAST>
__global__ __launch_bounds__(kThreads) void wide_bwd_kernel(LogprobParams p) {
    constexpr int VE = 16 / static_cast<int>(sizeof(T));
    __shared__ Sums part[kThreads / 64];
    const int64_t units = p.rows * p.slices;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t r = p.slices == 1 ? u : u / p.slices;
        const int q = static_cast<int>(u - r * p.slices);
        const T* row = static_cast<const T*>(p.logits) + MSEL_IDX(r, p.rows) * p.stride;
        T* out = static_cast<T*>(p.dlogits) + MSEL_IDX(r, p.rows) * p.dstride;
        const int c0 = q * p.slice, c1 = min(p.V, c0 + p.slice);
        RowGrad g(p, r);
        if (g.again())  // the same in every thread of the block
            g.stand_at(block_join(thread_sums<T, false>(row, 0, p.V, g.k2), g.k2, part));
        each_vector<T>(row, c0, c1, [&](const auto& v, int c, int round, auto count) {
            constexpr int vecs = decltype(count)::value;
#pragma unroll
            for (int j = 0; j < vecs; ++j) {
                const int col = c + j * round;
                float d[VE];
#pragma unroll
                for (int k = 0; k < VE; ++k) d[k] = g.at(v[j * VE + k], p.scale);
                if (static_cast<unsigned>(g.t - col) < static_cast<unsigned>(VE)) {
#pragma unroll
                    for (int k = 0; k < VE; ++k)
                        if (col + k == g.t) d[k] = fmaf(g.dt, p.scale, d[k]);
                }
                if (g.dead) {
#pragma unroll
                    for (int k = 0; k < VE; ++k) d[k] = 0.0f;
                }
                if (col >= c0 && col + VE <= c1) {
                    st_raw<T, VE, PAST>(out + MSEL_SPAN(col, VE, c1), from_f32<T, VE>(d));
                } else {
#pragma unroll
                    for (int k = 0; k < VE; ++k)
                        if (col + k >= c0 && col + k < c1) Elem<T>::store1(out + col + k, d[k]);
                }
            }
        });
    }
}

// ---- plans -------------------------------------------------------------------------------------

// Lanes and vectors per lane of a narrow row (0 lanes: a wide one).
struct Narrow {
    int team, vecs;
};
Narrow narrow_of(int V, bool bf16) {
    const int ve = bf16 ? 8 : 4;
    for (const Narrow n : {Narrow{4, 1}, Narrow{4, 2}, Narrow{4, 4}, Narrow{16, 2}, Narrow{16, 4},
                           Narrow{64, 2}, Narrow{64, 4}})
        if (V <= n.team * n.vecs * ve) return n;
    return {0, 0};
}

// Whether a narrow row's many likeliest tokens are found by a block all the same: teams take a pass
// over their registers per token, a block ranks what reaches its bound, or the whole of a short
// row.  A bound needs lanes with columns in all 4 wavefronts.  256 rows, 64 tokens: of 250 columns
// 12 us, teams 46; of 2000 in bf16 12, 78; but of 500, with two wavefronts empty, 21, 37 for 64 and
// 12 for 17 tokens in fp32, and of 1000 in bf16 60, 51.  Many rows fill the chip with teams: 1024
// of 250 take 20 us by blocks whatever is asked for, by teams 15, 25 and 46 for 17, 32 and 64
// tokens; 4096 of 250 60, 15, 25 and 47.  (Wide ones would gain beyond: 4096 of 2000 in bf16 41 us,
// teams 154, for 64 tokens.)
bool top_by_block(int64_t rows, int V, int top, bool bf16) {
    return top > 16 && rows <= 1024 && (V <= 256 || V >= 224 * (bf16 ? 8 : 4));
}

// Slices of a row: enough blocks for the chip, of about 4096 columns at least, no more than a
// wavefront joins and than the joined keys' list holds.  The last slice has V / n - 64 (n - 1)
// columns or more, which for up to n = 48 is above 1000, so more than kMaxTop.
void slice_rows(int64_t rows, int V, int top, int64_t blocks, int& slices, int& slice) {
    int64_t n = std::min<int64_t>((blocks + rows - 1) / rows, (V + 4095) / 4096);
    n = std::min<int64_t>(n, top > 0 ? std::min(48, kCandidates / top) : 64);
    slice = static_cast<int>((V + n - 1) / n);
    slice = (slice + 63) / 64 * 64;
    slices = (V + slice - 1) / slice;
}
constexpr int64_t kFwdBlocks = 512, kBwdBlocks = 2048;

dim3 grid_for(int64_t units) {
    return dim3(static_cast<unsigned>(std::min<int64_t>(units, kMaxBlocks)));
}

template <typename T, int TEAM, int NV>
void launch_narrow(const LogprobParams& p, bool bwd, hipStream_t stream) {
    const dim3 grid = grid_for((p.rows + kThreads / TEAM - 1) / (kThreads / TEAM));
    if (bwd)
        hipLaunchKernelGGL((narrow_bwd_kernel<T, TEAM, NV>), grid, dim3(kThreads), 0, stream, p);
    else
        hipLaunchKernelGGL((narrow_fwd_kernel<T, TEAM, NV>), grid, dim3(kThreads), 0, stream, p);
}

template <typename T>
hipError_t launch_narrow(const LogprobParams& p, const Narrow& n, bool bwd, hipStream_t stream) {
    if (n.team == 4 && n.vecs == 1)
        launch_narrow<T, 4, 1>(p, bwd, stream);
    else if (n.team == 4 && n.vecs == 2)
        launch_narrow<T, 4, 2>(p, bwd, stream);
    else if (n.team == 4)
        launch_narrow<T, 4, 4>(p, bwd, stream);
    else if (n.team == 16 && n.vecs == 2)
        launch_narrow<T, 16, 2>(p, bwd, stream);
    else if (n.team == 16)
        launch_narrow<T, 16, 4>(p, bwd, stream);
    else if (n.vecs == 2)
        launch_narrow<T, 64, 2>(p, bwd, stream);
    else
        launch_narrow<T, 64, 4>(p, bwd, stream);
    return hipGetLastError();
}

template <typename T>
hipError_t forward(LogprobParams p, hipStream_t stream) {
    const dim3 block(kThreads);
    const Narrow narrow = narrow_of(p.V, sizeof(T) == 2);
    if (narrow.team != 0 && !top_by_block(p.rows, p.V, p.top, sizeof(T) == 2))
        return launch_narrow<T>(p, narrow, false, stream);
    slice_rows(p.rows, p.V, p.top, kFwdBlocks, p.slices, p.slice);
    const dim3 grid = grid_for(p.rows * p.slices);
    if (p.slice <= kHeld && p.top > 0)
        hipLaunchKernelGGL((held_fwd_kernel<T, true>), grid, block, 0, stream, p);
    else if (p.slice <= kHeld)
        hipLaunchKernelGGL((held_fwd_kernel<T, false>), grid, block, 0, stream, p);
    else if (p.top > 0)
        hipLaunchKernelGGL((wide_fwd_kernel<T, true, true>), grid, block, 0, stream, p);
    else if (p.entropy != nullptr)
        hipLaunchKernelGGL((wide_fwd_kernel<T, true, false>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((wide_fwd_kernel<T, false, false>), grid, block, 0, stream, p);
    if (p.slices > 1)
        hipLaunchKernelGGL(join_kernel<T>, grid_for(p.rows), block, 0, stream, p);
    return hipGetLastError();
}

template <typename T>
hipError_t backward(LogprobParams p, hipStream_t stream) {
    const dim3 block(kThreads);
    const Narrow narrow = narrow_of(p.V, sizeof(T) == 2);
    if (narrow.team != 0) return launch_narrow<T>(p, narrow, true, stream);
    p.slices = 1;
    p.slice = p.V;
    if (p.dlogits != p.logits) slice_rows(p.rows, p.V, 0, kBwdBlocks, p.slices, p.slice);
    const dim3 grid = grid_for(p.rows * p.slices);
    if (past_cache(p.rows * p.V * static_cast<int64_t>(sizeof(T))))
        hipLaunchKernelGGL((wide_bwd_kernel<T, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((wide_bwd_kernel<T, false>), grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace

size_t logprob_workspace_bytes(int64_t rows, int V, int top, bool bf16) {
    if (narrow_of(V, bf16).team != 0) return 0;
    int slices = 1, slice = 0;
    slice_rows(rows, V, top, kFwdBlocks, slices, slice);
    if (slices == 1) return 0;
    return sums_bytes(rows, slices) + static_cast<size_t>(rows) * slices * top * sizeof(Key);
}

hipError_t launch_logprob_fwd(const LogprobParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? forward<bf16_t>(p, stream) : forward<float>(p, stream);
}

hipError_t launch_logprob_bwd(const LogprobParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? backward<bf16_t>(p, stream) : backward<float>(p, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_logprob)

}  // namespace msel
