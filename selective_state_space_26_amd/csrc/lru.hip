// lru.hip -- the gated linear recurrence, one state per channel, over rows of [batch, dim, seqlen]:
//   r = sigmoid(gate_a), i = sigmoid(gate_x), a = exp(lam r), m = sqrt(1 - a^2)
//   h_t = a_t h_{t-1} + m_t i_t x_t,   out = h
// and its backward.  With g_t the gradient that reaches h_t and e_t = a_t g_t what it hands on to
// the step before:
//   e_t = a_t (dout_t + e_{t+1}),   g_t = dout_t + e_{t+1}
//   dx = g m i,   dgate_x = g m x i (1 - i),   dgate_a = q lam r (1 - r),   dlam = sum q r
//   with q = g (a h_{t-1} - i x a^2 / m), the gradient of log a
// Both recurrences are affine, so steps compose: a lane composes kStep consecutive steps, the lanes
// of a team scan their pairs with DPP, and a team walks the tiles of its row with the state in a
// register.  The backward rebuilds h from the states at the chunk boundaries and walks the tiles
// from the last to the first.
//
// HBM bounds it: 4 tensors forward, 7 backward, against about 45 and 75 VALU instructions per
// element, 6 and 7 of them transcendental (quarter rate).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "block_kernels.hpp"
#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

constexpr int kStep = 8;  // steps per lane: 16 bytes of bf16
constexpr int kTile = 64 * kStep;
static_assert(kTile == kChunk, "a wavefront's tile starts at a chunk boundary");
constexpr unsigned kMaxBlocks = 1u << 21;  // of up to 1024: a grid has fewer than 2^32 threads
constexpr int kMaxSegments = 63;           // a wavefront composes them and h0

// One step's factors.
struct Gates {
    float r, i, a;
    float m2;  // 1 - a^2
};

// lam2: lam log2 e, so that a = 2^l, l = lam2 r.  1 - a^2 = 1 - e^-q, q = -2 ln 2 l: near q = 0 the
// difference would cancel, so up to q = 0.3 it is the series q - q^2 / 2! + ... - q^6 / 6! in
// powers of l, whose first missing term is q^6 / 7! < 1.5e-7 of it; from there on the difference
// loses at most 2 bits.
__device__ __forceinline__ Gates gates_of(float ga, float gx, float lam2) {
    Gates s;
    s.r = sigmoid_f(ga);
    s.i = sigmoid_f(gx);
    const float l = lam2 * s.r;
    s.a = exp2_hw(l);
    constexpr float c = -2.0f * kLn2;  // q = c l
    float p = -c * c * c * c * c * c / 720.0f;
    p = fmaf(p, l, c * c * c * c * c / 120.0f);
    p = fmaf(p, l, -c * c * c * c / 24.0f);
    p = fmaf(p, l, c * c * c / 6.0f);
    p = fmaf(p, l, -c * c / 2.0f);
    p = fmaf(p, l, c);
    s.m2 = l > 0.3f / c ? p * l : fmaf(-s.a, s.a, 1.0f);
    return s;
}

template <typename T>
__device__ __forceinline__ RawVec<T, kStep> ld_row(const T* row, int t0, int L) {
    if (t0 + kStep <= L) return ld_raw<T, kStep>(row + MSEL_SPAN(t0, kStep, L));
    return ld_part<T, kStep>(row + t0, L - t0);
}

template <typename T, bool PAST>
__device__ __forceinline__ void st_row(T* row, int t0, int L, const float (&v)[kStep]) {
    const RawVec<T, kStep> r = from_f32<T, kStep>(v);
    if (t0 + kStep <= L)
        st_raw<T, kStep, PAST>(row + MSEL_SPAN(t0, kStep, L), r);
    else if (t0 < L)
        st_part<T, kStep>(row + t0, r, L - t0);
}

// Inclusive scan over 16 lanes, and the suffix one (each lane with the lanes after it).
__device__ __forceinline__ void scan16(float& P, float& S) {
    asm volatile("s_nop 1\n" MSEL_FWD_LEVEL("row_shr:1", "0xf") MSEL_FWD_LEVEL("row_shr:2", "0xf")
                     MSEL_FWD_LEVEL("row_shr:4", "0xf") MSEL_FWD_LEVEL("row_shr:8", "0xf")
                 : [P] "+v"(P), [S] "+v"(S));
}
__device__ __forceinline__ void suffix16(float& P, float& S) {
    asm volatile("s_nop 1\n" MSEL_FWD_LEVEL("row_shl:1", "0xf") MSEL_FWD_LEVEL("row_shl:2", "0xf")
                     MSEL_FWD_LEVEL("row_shl:4", "0xf") MSEL_FWD_LEVEL("row_shl:8", "0xf")
                 : [P] "+v"(P), [S] "+v"(S));
}

// The same over 4 or 8 lanes of 16: a pair is composed with the one that lies a shift away, where
// the team has a lane there.
template <int SHIFT>
__device__ __forceinline__ void compose_from(float& P, float& S, bool has) {
    const float p = dpp<SHIFT, 0xf>(P, P), s = dpp<SHIFT, 0xf>(S, S);
    S = has ? fmaf(P, s, S) : S;
    P = has ? P * p : P;
}
template <int TEAM>
__device__ __forceinline__ void scan_part(float& P, float& S) {
    const int l = lane_id() % TEAM;
    compose_from<kRowShr1>(P, S, l >= 1);
    compose_from<kRowShr2>(P, S, l >= 2);
    if constexpr (TEAM == 8) compose_from<kRowShr4>(P, S, l >= 4);
}
template <int TEAM>
__device__ __forceinline__ void suffix_part(float& P, float& S) {
    const int l = TEAM - 1 - lane_id() % TEAM;
    compose_from<kRowShl1>(P, S, l >= 1);
    compose_from<kRowShl2>(P, S, l >= 2);
    if constexpr (TEAM == 8) compose_from<kRowShl4>(P, S, l >= 4);
}

// The state that enters each lane, from the lanes' own pairs (P, S) and the state h that enters
// the team (1, 4, 8, 16 or 64 lanes); h becomes the one that leaves it (in every lane).
template <int TEAM>
__device__ __forceinline__ float enter_forward(float P, float S, float& h) {
    if constexpr (TEAM == 1) {
        const float in = h;
        h = fmaf(P, h, S);
        return in;
    } else if constexpr (TEAM < 16) {
        scan_part<TEAM>(P, S);
        const float before = fmaf(dpp<kRowShr1, 0xf>(P, P), h, dpp<kRowShr1, 0xf>(S, S));
        const float in = lane_id() % TEAM == 0 ? h : before;
        const float out = fmaf(P, h, S);
        h = __shfl(out, lane_id() | (TEAM - 1));
        return in;
    } else if constexpr (TEAM == 16) {
        scan16(P, S);
        const float in = fmaf(dpp<kRowShr1, 0xf>(1.0f, P), h, dpp<kRowShr1, 0xf>(0.0f, S));
        const float out = fmaf(P, h, S);
        h = __shfl(out, (lane_id() & 48) | 15);
        return in;
    } else {
        scan_fwd_fused(P, S);
        const float in = fmaf(shift_up(P, 1.0f), h, shift_up(S, 0.0f));
        h = fmaf(readlane(P, 63), h, readlane(S, 63));
        return in;
    }
}

// The suffix composition over a wavefront: per lane the pair of the lanes after it in its row of
// 16, per row its pair, and the whole wavefront's.
struct Suffix {
    float P, S;             // of the lanes after this one in its row
    float rp[4], rs[4];     // of whole rows
    __device__ __forceinline__ Suffix(float p, float s) {
        suffix16(p, s);
        P = dpp<kRowShl1, 0xf>(1.0f, p);
        S = dpp<kRowShl1, 0xf>(0.0f, s);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            rp[k] = readlane(p, 16 * k);
            rs[k] = readlane(s, 16 * k);
        }
    }
    __device__ __forceinline__ float whole_p() const { return rp[0] * rp[1] * rp[2] * rp[3]; }
    __device__ __forceinline__ float through(float e) const {
#pragma unroll
        for (int k = 3; k >= 0; --k) e = fmaf(rp[k], e, rs[k]);
        return e;
    }
    // what enters each lane when e enters the wavefront behind its last lane
    __device__ __forceinline__ float enter(float e) const {
        const int row = lane_id() >> 4;
        float in = e;
#pragma unroll
        for (int k = 3; k >= 1; --k) {
            e = fmaf(rp[k], e, rs[k]);
            in = row < k ? e : in;
        }
        return fmaf(P, in, S);
    }
};

// What enters each lane from behind, as enter_forward.
template <int TEAM>
__device__ __forceinline__ float enter_backward(float P, float S, float& e) {
    if constexpr (TEAM == 1) {
        const float in = e;
        e = fmaf(P, e, S);
        return in;
    } else if constexpr (TEAM < 16) {
        suffix_part<TEAM>(P, S);
        const float behind = fmaf(dpp<kRowShl1, 0xf>(P, P), e, dpp<kRowShl1, 0xf>(S, S));
        const float in = lane_id() % TEAM == TEAM - 1 ? e : behind;
        const float out = fmaf(P, e, S);
        e = __shfl(out, lane_id() & -TEAM);
        return in;
    } else if constexpr (TEAM == 16) {
        suffix16(P, S);
        const float in = fmaf(dpp<kRowShl1, 0xf>(1.0f, P), e, dpp<kRowShl1, 0xf>(0.0f, S));
        const float out = fmaf(P, e, S);
        e = __shfl(out, lane_id() & 48);
        return in;
    } else {
        const Suffix s(P, S);
        const float in = s.enter(e);
        e = s.through(e);
        return in;
    }
}

// a_t and the input's share b_t of kStep steps, the first `valid` of them real and the others the
// identity; whole: all of them are (uniform).
template <typename T>
__device__ __forceinline__ void steps_of(const RawVec<T, kStep>& rx, const RawVec<T, kStep>& ra,
                                         const RawVec<T, kStep>& ri, float lam2, bool whole,
                                         int valid, float (&a)[kStep], float (&b)[kStep]) {
    float x[kStep], ga[kStep], gx[kStep];
    to_f32<T, kStep>(rx, x);
    to_f32<T, kStep>(ra, ga);
    to_f32<T, kStep>(ri, gx);
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
        const Gates s = gates_of(ga[k], gx[k], lam2);
        a[k] = s.a;
        b[k] = __builtin_amdgcn_sqrtf(s.m2) * s.i * x[k];
    }
    if (!whole) {
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            a[k] = k < valid ? a[k] : 1.0f;
            b[k] = k < valid ? b[k] : 0.0f;
        }
    }
}

__device__ __forceinline__ void compose(const float (&a)[kStep], const float (&b)[kStep], float& P,
                                        float& S) {
    P = a[0];
    S = b[0];
#pragma unroll
    for (int k = 1; k < kStep; ++k) {
        P *= a[k];
        S = fmaf(a[k], S, b[k]);
    }
}

// One step per row (decoding).
template <typename T>
__global__ __launch_bounds__(256) void lru_step_kernel(LruParams p) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.D;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; row < rows;
         row += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t at = MSEL_IDX(row, rows);
        const Gates s = gates_of(Elem<T>::load1(static_cast<const T*>(p.ga) + at),
                                 Elem<T>::load1(static_cast<const T*>(p.gx) + at),
                                 p.lam[MSEL_IDX(static_cast<int>(row % p.D), p.D)] * kLog2e);
        const float h0 = p.h0 != nullptr ? p.h0[at] : 0.0f;
        const float x = Elem<T>::load1(static_cast<const T*>(p.x) + at);
        const float h = fmaf(s.a, h0, __builtin_amdgcn_sqrtf(s.m2) * s.i * x);
        if (p.chunks != nullptr) p.chunks[at] = h0;
        if (p.out != nullptr) Elem<T>::store1(static_cast<T*>(p.out) + at, h);
        if (p.final_state != nullptr) p.final_state[at] = h;
    }
}

// Pairs of a row's segments before (DIR = 1) or behind (DIR = -1) segment `seg`, composed onto v.
// Forward, segment s is entry s + 1 and entry 0 is (0, h0): the state is read from there, since
// the row's last segment may write final_state over h0 meanwhile.
template <int DIR>
__device__ __forceinline__ float through_segments(const float2* pairs, int64_t row, int64_t rows,
                                                  int seg, int nseg, float v) {
    const int l = lane_id();
    const int s = DIR > 0 ? l : nseg - 1 - l;  // in the order of composition
    float P = 1.0f, S = 0.0f;
    if (DIR > 0 ? s <= seg : s > seg) {
        const float2 q = pairs[MSEL_IDX(row * (nseg + 1) + s, rows * (nseg + 1))];
        P = q.x;
        S = q.y;
    }
    scan_fwd_fused(P, S);
    return fmaf(readlane(P, 63), v, readlane(S, 63));
}

// The pair of every segment of a row: of the states (DIR = 1), or of the adjoint, from the gates
// and dout (DIR = -1).  A wavefront per (row, segment).
template <typename T, int DIR>
__global__ __launch_bounds__(256) void lru_summary_kernel(LruParams p) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.D, units = rows * p.nseg;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); u < units;
         u += static_cast<int64_t>(gridDim.x) * 4) {
        const int64_t row = u / p.nseg;
        const int seg = static_cast<int>(u - row * p.nseg);
        const float lam2 = p.lam[MSEL_IDX(static_cast<int>(row % p.D), p.D)] * kLog2e;
        const int64_t base = MSEL_IDX(row, rows) * p.L;
        const T* ga = static_cast<const T*>(p.ga) + base;
        const T* gx = static_cast<const T*>(p.gx) + base;
        const T* x = static_cast<const T*>(DIR > 0 ? p.x : p.dout) + base;
        const int t_lo = seg * p.seg_tiles * kTile;
        const int t_hi = min(p.L, t_lo + p.seg_tiles * kTile);
        const int n = (t_hi - t_lo + kTile - 1) / kTile;
        const int l8 = lane_id() * kStep;
        float WP = 1.0f, WS = 0.0f;
        RawVec<T, kStep> nx, na, ni;
        const auto fetch = [&](int k) {
            const int t = t_lo + (DIR > 0 ? k : n - 1 - k) * kTile + l8;
            nx = ld_row(x, t, p.L);
            na = ld_row(ga, t, p.L);
            if constexpr (DIR > 0) ni = ld_row(gx, t, p.L);
        };
        fetch(0);
        for (int k = 0; k < n; ++k) {
            const RawVec<T, kStep> rx = nx, ra = na, ri = ni;
            const int t = t_lo + (DIR > 0 ? k : n - 1 - k) * kTile + l8;
            if (k + 1 < n) fetch(k + 1);
            float P, S;
            if constexpr (DIR > 0) {
                float a[kStep], b[kStep];
                steps_of<T>(rx, ra, ri, lam2, t - l8 + kTile <= p.L, p.L - t, a, b);
                compose(a, b, P, S);
                scan_fwd_fused(P, S);
                P = readlane(P, 63);
                S = readlane(S, 63);
            } else {
                float d[kStep], g[kStep];
                to_f32<T, kStep>(rx, d);
                to_f32<T, kStep>(ra, g);
                P = 1.0f;
                S = 0.0f;
#pragma unroll
                for (int j = kStep - 1; j >= 0; --j) {
                    const float a = j < p.L - t ? exp2_hw(lam2 * sigmoid_f(g[j])) : 1.0f;
                    P *= a;
                    S = a * (d[j] + S);
                }
                const Suffix s(P, S);
                P = s.whole_p();
                S = s.through(0.0f);
            }
            WS = fmaf(P, WS, S);
            WP *= P;
        }
        if (lane_id() == 0) {
            const int64_t at = row * (p.nseg + 1);
            [[maybe_unused]] const int64_t n = rows * (p.nseg + 1);
            p.pairs[MSEL_IDX(at + seg + (DIR > 0 ? 1 : 0), n)] = float2{WP, WS};
            if (DIR > 0 && seg == 0)
                p.pairs[MSEL_IDX(at, n)] =
                    float2{0.0f, p.h0 != nullptr ? p.h0[MSEL_IDX(row, rows)] : 0.0f};
        }
    }
}

// The forward.  A team of 1 to 64 lanes, or of several wavefronts, per row, or a wavefront per
// segment of a row when there are several (their pairs known).  out may be null (states only).
// PAST: out is stored past the caches.
template <typename T, int TEAM, bool PAST>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void lru_fwd_kernel(LruParams p) {
    constexpr bool kBlock = TEAM > 64;
    constexpr int kLanes = kBlock ? 64 : TEAM;  // of one scan
    constexpr int kTeams = kBlock ? 1 : 256 / TEAM, kWaves = kBlock ? TEAM / 64 : 1;
    __shared__ float2 total[2][kWaves];
    const int64_t rows = static_cast<int64_t>(p.B) * p.D;
    const int nseg = TEAM == 64 ? p.nseg : 1;
    const int64_t units = rows * nseg;
    const int wave = threadIdx.x >> 6;
    const int l8 = static_cast<int>(threadIdx.x % TEAM) * kStep;
    const int tile = TEAM * kStep;
    // the loop is uniform over a block where the teams need its barrier, and over a wavefront where
    // they need its lanes
    const int64_t bid = xcd_order(blockIdx.x, gridDim.x);
    for (int64_t u0 = bid * kTeams; u0 < units; u0 += static_cast<int64_t>(gridDim.x) * kTeams) {
        const int64_t mine = u0 + threadIdx.x / TEAM;
        if (TEAM == 64 && mine >= units) break;  // whole wavefronts
        const bool live = mine < units;
        const int64_t u = live ? mine : units - 1;  // lanes without a row repeat the last one
        const int64_t row = nseg == 1 ? u : u / nseg;
        const int seg = static_cast<int>(u - row * nseg);
        const float lam2 = p.lam[MSEL_IDX(static_cast<int>(row % p.D), p.D)] * kLog2e;
        const int64_t base = MSEL_IDX(row, rows) * p.L;
        const T* x = static_cast<const T*>(p.x) + base;
        const T* ga = static_cast<const T*>(p.ga) + base;
        const T* gx = static_cast<const T*>(p.gx) + base;
        T* out = p.out != nullptr ? static_cast<T*>(p.out) + base : nullptr;
        const int t_lo = seg * p.seg_tiles * kTile;
        const int t_hi = nseg == 1 ? p.L : min(p.L, t_lo + p.seg_tiles * kTile);
        float h = 0.0f;
        if (nseg > 1)
            h = through_segments<1>(p.pairs, row, rows, seg, nseg, h);
        else if (p.h0 != nullptr)
            h = p.h0[MSEL_IDX(row, rows)];
        RawVec<T, kStep> nx = ld_row(x, t_lo + l8, p.L), na = ld_row(ga, t_lo + l8, p.L),
                         ni = ld_row(gx, t_lo + l8, p.L);
        int turn = 0;
        for (int t0 = t_lo; t0 < t_hi; t0 += tile, turn ^= 1) {
            const RawVec<T, kStep> rx = nx, ra = na, ri = ni;
            const int t = t0 + l8;
            if (t0 + tile < t_hi) {
                nx = ld_row(x, t + tile, p.L);
                na = ld_row(ga, t + tile, p.L);
                ni = ld_row(gx, t + tile, p.L);
            }
            float a[kStep], b[kStep], P, S;
            steps_of<T>(rx, ra, ri, lam2, t0 + tile <= p.L, p.L - t, a, b);
            compose(a, b, P, S);
            float in, entered = h;  // what enters the wavefront
            if constexpr (kBlock) {
                scan_fwd_fused(P, S);
                if (lane_id() == 63) total[turn][wave] = float2{P, S};
                __syncthreads();  // the other buffer is written before the next one
                float before = h;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    if (w == wave) before = h;
                    h = fmaf(total[turn][w].x, h, total[turn][w].y);
                }
                entered = before;
                in = fmaf(shift_up(P, 1.0f), before, shift_up(S, 0.0f));
            } else {
                in = enter_forward<kLanes>(P, S, h);
            }
            if (p.chunks != nullptr && live && threadIdx.x % kLanes == 0) {
                const int c = t / kTile;
                if (t < p.L) p.chunks[MSEL_IDX(row * p.nchunks + c, rows * p.nchunks)] = entered;
            }
            if (out != nullptr) {
                float v[kStep];
#pragma unroll
                for (int k = 0; k < kStep; ++k) v[k] = in = fmaf(a[k], in, b[k]);
                if (live) st_row<T, PAST>(out, t, p.L, v);
            }
        }
        if (p.final_state != nullptr && t_hi == p.L && live && threadIdx.x % TEAM == 0)
            p.final_state[MSEL_IDX(row, rows)] = h;
        if (kBlock) __syncthreads();  // the next row's first buffer may be the last one read
    }
}

// The backward, teams as in the forward.  dlam's parts: one per row (and segment).
template <typename T, int TEAM, bool PAST>
__global__ __launch_bounds__(TEAM > 256 ? TEAM : 256) void lru_bwd_kernel(LruParams p) {
    constexpr bool kBlock = TEAM > 64;
    constexpr int kLanes = kBlock ? 64 : TEAM;
    constexpr int kTeams = kBlock ? 1 : 256 / TEAM, kWaves = kBlock ? TEAM / 64 : 1;
    __shared__ float2 total[2][kWaves];
    __shared__ float sums[kWaves];
    const int64_t rows = static_cast<int64_t>(p.B) * p.D;
    const int nseg = TEAM == 64 ? p.nseg : 1;
    const int64_t units = rows * nseg;
    const int wave = threadIdx.x >> 6;
    const int l8 = static_cast<int>(threadIdx.x % TEAM) * kStep;
    const int tile = TEAM * kStep;
    const int64_t bid = xcd_order(blockIdx.x, gridDim.x);
    for (int64_t u0 = bid * kTeams; u0 < units; u0 += static_cast<int64_t>(gridDim.x) * kTeams) {
        const int64_t mine = u0 + threadIdx.x / TEAM;
        if (TEAM == 64 && mine >= units) break;
        const bool live = mine < units;
        const int64_t u = live ? mine : units - 1;
        const int64_t row = nseg == 1 ? u : u / nseg;
        const int seg = static_cast<int>(u - row * nseg);
        const int d = static_cast<int>(row % p.D);
        const float lam = p.lam[MSEL_IDX(d, p.D)], lam2 = lam * kLog2e;
        const int64_t base = MSEL_IDX(row, rows) * p.L;
        const T* x = static_cast<const T*>(p.x) + base;
        const T* ga = static_cast<const T*>(p.ga) + base;
        const T* gx = static_cast<const T*>(p.gx) + base;
        const T* dout = static_cast<const T*>(p.dout) + base;
        const int t_lo = seg * p.seg_tiles * kTile;
        const int t_hi = nseg == 1 ? p.L : min(p.L, t_lo + p.seg_tiles * kTile);
        float e = p.dfinal != nullptr ? p.dfinal[MSEL_IDX(row, rows)] : 0.0f;
        if (nseg > 1) e = through_segments<-1>(p.pairs, row, rows, seg, nseg, e);
        float dlam = 0.0f;
        const int last = t_lo + (t_hi - t_lo - 1) / tile * tile;
        RawVec<T, kStep> nx = ld_row(x, last + l8, p.L), na = ld_row(ga, last + l8, p.L),
                         ni = ld_row(gx, last + l8, p.L), nd = ld_row(dout, last + l8, p.L);
        int turn = 0;
        for (int t0 = last; t0 >= t_lo; t0 -= tile, turn ^= 1) {
            const RawVec<T, kStep> rx = nx, ra = na, ri = ni, rd = nd;
            const int t = t0 + l8;
            // the state that enters the wavefront, from the chunk that starts there
            float h;
            if constexpr (TEAM >= 64) {
                const int c = min(__builtin_amdgcn_readfirstlane(t / kTile), p.nchunks - 1);
                h = p.chunks[MSEL_IDX(row * p.nchunks + c, rows * p.nchunks)];
            } else {  // a row is one chunk: its state, or without chunk states the row's own
                const float* const from = p.chunks != nullptr ? p.chunks : p.h0;
                h = from != nullptr ? from[MSEL_IDX(row, rows)] : 0.0f;
            }
            if (t0 - tile >= t_lo) {
                nx = ld_row(x, t - tile, p.L);
                na = ld_row(ga, t - tile, p.L);
                ni = ld_row(gx, t - tile, p.L);
                nd = ld_row(dout, t - tile, p.L);
            }
            float xs[kStep], va[kStep], vi[kStep], ds[kStep];
            to_f32<T, kStep>(rx, xs);
            to_f32<T, kStep>(ra, va);
            to_f32<T, kStep>(ri, vi);
            to_f32<T, kStep>(rd, ds);
            float a[kStep], rr[kStep], ii[kStep], ms[kStep], b[kStep];
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
                const Gates s = gates_of(va[k], vi[k], lam2);
                a[k] = s.a;
                rr[k] = s.r;
                ii[k] = s.i;
                ms[k] = __builtin_amdgcn_sqrtf(s.m2);
                b[k] = ms[k] * s.i * xs[k];
            }
            if (t0 + tile > p.L) {  // steps past the end: the identity, and nothing to dlam
#pragma unroll
                for (int k = 0; k < kStep; ++k) {
                    const bool valid = k < p.L - t;
                    a[k] = valid ? a[k] : 1.0f;
                    b[k] = valid ? b[k] : 0.0f;
                    ds[k] = valid ? ds[k] : 0.0f;
                    rr[k] = valid ? rr[k] : 0.0f;
                }
            }
            float P, S;
            compose(a, b, P, S);
            float hin = enter_forward<kLanes>(P, S, h);
            // the adjoint's pairs, from the last step to the first
            float Q = 1.0f, R = 0.0f;
#pragma unroll
            for (int k = kStep - 1; k >= 0; --k) {
                Q *= a[k];
                R = a[k] * (ds[k] + R);
            }
            float ein;
            if constexpr (kBlock) {
                const Suffix s(Q, R);
                if (lane_id() == 0) total[turn][wave] = float2{s.whole_p(), s.through(0.0f)};
                __syncthreads();
                float behind = e;
#pragma unroll
                for (int w = kWaves - 1; w >= 0; --w) {
                    if (w == wave) behind = e;
                    e = fmaf(total[turn][w].x, e, total[turn][w].y);
                }
                ein = s.enter(behind);
            } else {
                ein = enter_backward<kLanes>(Q, R, e);
            }
            float g[kStep];
#pragma unroll
            for (int k = kStep - 1; k >= 0; --k) {
                g[k] = ds[k] + ein;
                ein = a[k] * g[k];
            }
            float dx[kStep], dga[kStep], dgx[kStep];
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
                const float m = ms[k];
                const float ix = ii[k] * xs[k];
                // where m = 0 the square root has no slope: its part is 0
                const float by_m = m > 0.0f ? ix * a[k] * a[k] * rcp_hw(m) : m;
                const float q = g[k] * fmaf(a[k], hin, -by_m);
                hin = fmaf(a[k], hin, b[k]);
                const float gm = g[k] * m;
                dx[k] = gm * ii[k];
                dgx[k] = gm * ix * (1.0f - ii[k]);
                const float qr = q * rr[k];
                dga[k] = qr * lam * (1.0f - rr[k]);
                dlam += t0 + tile <= p.L || k < p.L - t ? qr : 0.0f;
            }
            if (live) {
                st_row<T, PAST>(static_cast<T*>(p.dx) + base, t, p.L, dx);
                st_row<T, PAST>(static_cast<T*>(p.dga) + base, t, p.L, dga);
                st_row<T, PAST>(static_cast<T*>(p.dgx) + base, t, p.L, dgx);
            }
        }
        if (p.dh0 != nullptr && t_lo == 0 && live && threadIdx.x % TEAM == 0)
            p.dh0[MSEL_IDX(row, rows)] = e;
        if (p.dlam_part != nullptr) {
            if constexpr (TEAM >= 64) {
                dlam = wave_sum_fused(dlam);
            } else {
#pragma unroll
                for (int k = TEAM / 2; k > 0; k /= 2) dlam += __shfl_xor(dlam, k);
            }
            if constexpr (kBlock) {
                if (lane_id() == 0) sums[wave] = dlam;
                __syncthreads();
                dlam = sums[0];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) dlam += sums[w];
            }
            if (live && threadIdx.x % TEAM == 0) {
                const int64_t part = (row / p.D * nseg + seg) * p.D + d;
                p.dlam_part[MSEL_IDX(part, units)] = dlam;
            }
        }
        if (kBlock) __syncthreads();
    }
}

}  // namespace

// Teams: as few of 1, 4, 8, 16 and 64 lanes as hold a row, 8 steps each (41 x 3992 rows of 14 in
// bf16, forward and backward: 14 and 24 us, 39 and 76 with 16 lanes).  Above 512 steps a wavefront
// a row where there are rows enough; four, whose loads are one stretch of 4 KB, where many rows
// fill their tiles of 2048 steps (8192 x 4096, forward and backward: bf16 54 and 88 us, 61 and 107
// with one, fp32 106 and 190, 119 and 222; 12288 x 2048 bf16: 107 us together, 110) or where fewer
// rows than that leave wavefronts wanting (1536 x 16384 bf16: 41 and 75, 52 and 78); sixteen
// (eight in the backward, for its registers) for very long rows (5120 x 65536 forward: 481, 541
// with one or four) and for up to a row per CU (200 x 30011 bf16: 17 and 25 us, 22 and 31 with
// four, fp32 22 and 36, 24 and 39; but of 511 x 12000, whose blocks take two turns, fp32 27 and 38,
// 20 and 34 with four).  Below 128 rows those are cut into segments that are composed first (64 x
// 65536: 44 us, 63 with sixteen).
LruPlan lru_plan(int64_t rows, int L, bool bwd) {
    LruPlan q{};
    q.tiles = (L + kTile - 1) / kTile;
    q.seg_tiles = q.tiles;
    q.nseg = 1;
    const int most = bwd ? 512 : 1024;
    if (L <= kStep) {
        q.team = 1;
    } else if (L <= 8 * kStep) {
        q.team = L <= 4 * kStep ? 4 : 8;
    } else if (L <= 16 * kStep) {
        q.team = 16;
    } else if (q.tiles == 1) {
        q.team = 64;
    } else if (rows >= 2048) {
        const bool full = (L + 4 * kTile - 1) / (4 * kTile) * static_cast<int64_t>(4 * kTile) <=
                          L + L / 20;
        q.team = L >= 64 * kTile && (!bwd || rows >= 4096) ? most
                 : rows >= 8192 && full                      ? 256
                                                             : 64;
    } else if (rows >= 128) {
        q.team = L >= 64 * kTile || (rows <= 256 && L > 8 * kTile) ? most : 256;
    } else {
        q.team = 64;
        const int64_t want = std::min<int64_t>(kMaxSegments, (4096 + rows - 1) / rows);
        const int nseg = static_cast<int>(std::min<int64_t>(want, q.tiles));
        q.seg_tiles = (q.tiles + nseg - 1) / nseg;
        q.nseg = (q.tiles + q.seg_tiles - 1) / q.seg_tiles;
    }
    return q;
}

namespace {

dim3 grid_for(int64_t units, int per_block) {
    const int64_t blocks = (units + per_block - 1) / per_block;
    return dim3(static_cast<unsigned>(std::min<int64_t>(blocks, kMaxBlocks)));
}

template <typename T, int TEAM>
void launch_fwd(const LruParams& p, bool past, int64_t units, hipStream_t stream) {
    constexpr int threads = TEAM > 256 ? TEAM : 256;
    const dim3 grid = grid_for(units, threads / TEAM), block(threads);
    if (past)
        hipLaunchKernelGGL((lru_fwd_kernel<T, TEAM, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((lru_fwd_kernel<T, TEAM, false>), grid, block, 0, stream, p);
}

template <typename T, int TEAM>
void launch_bwd(const LruParams& p, bool past, int64_t units, hipStream_t stream) {
    constexpr int threads = TEAM > 256 ? TEAM : 256;
    const dim3 grid = grid_for(units, threads / TEAM), block(threads);
    if (past)
        hipLaunchKernelGGL((lru_bwd_kernel<T, TEAM, true>), grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL((lru_bwd_kernel<T, TEAM, false>), grid, block, 0, stream, p);
}

template <typename T>
hipError_t forward(LruParams p, hipStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.D;
    if (p.L == 1) {
        hipLaunchKernelGGL(lru_step_kernel<T>, grid_for(rows, 256), dim3(256), 0, stream, p);
        return hipGetLastError();
    }
    const LruPlan q = lru_plan(rows, p.L, false);
    p.nseg = q.nseg;
    p.seg_tiles = q.seg_tiles;
    const int64_t units = rows * q.nseg;
    if (q.nseg > 1)
        hipLaunchKernelGGL((lru_summary_kernel<T, 1>), grid_for(units, 4), dim3(256), 0, stream, p);
    const bool past = past_cache(rows * p.L * static_cast<int64_t>(sizeof(T)));
    switch (q.team) {
        case 1: launch_fwd<T, 1>(p, past, units, stream); break;
        case 4: launch_fwd<T, 4>(p, past, units, stream); break;
        case 8: launch_fwd<T, 8>(p, past, units, stream); break;
        case 16: launch_fwd<T, 16>(p, past, units, stream); break;
        case 64: launch_fwd<T, 64>(p, past, units, stream); break;
        case 256: launch_fwd<T, 256>(p, past, units, stream); break;
        default: launch_fwd<T, 1024>(p, past, units, stream); break;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t backward(LruParams p, hipStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.B) * p.D;
    const LruPlan q = lru_plan(rows, p.L, true);
    p.nseg = q.nseg;
    p.seg_tiles = q.seg_tiles;
    const int64_t units = rows * q.nseg;
    const int64_t parts = static_cast<int64_t>(p.B) * q.nseg;
    if (parts == 1) p.dlam_part = p.dlam;  // the one part is the sum
    if (q.nseg > 1)
        hipLaunchKernelGGL((lru_summary_kernel<T, -1>), grid_for(units, 4), dim3(256), 0, stream,
                           p);
    const bool past = past_cache(3 * rows * p.L * static_cast<int64_t>(sizeof(T)));
    switch (q.team) {
        case 1: launch_bwd<T, 1>(p, past, units, stream); break;
        case 4: launch_bwd<T, 4>(p, past, units, stream); break;
        case 8: launch_bwd<T, 8>(p, past, units, stream); break;
        case 16: launch_bwd<T, 16>(p, past, units, stream); break;
        case 64: launch_bwd<T, 64>(p, past, units, stream); break;
        case 256: launch_bwd<T, 256>(p, past, units, stream); break;
        default: launch_bwd<T, 512>(p, past, units, stream); break;
    }
    const hipError_t s = hipGetLastError();
    if (s != hipSuccess || p.dlam == nullptr || parts == 1) return s;
    return launch_column_sums(p.dlam_part, parts, p.D, p.dlam, stream);
}

}  // namespace

hipError_t launch_lru_fwd(const LruParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? forward<bf16_t>(p, stream) : forward<float>(p, stream);
}

hipError_t launch_lru_bwd(const LruParams& p, bool bf16, hipStream_t stream) {
    return bf16 ? backward<bf16_t>(p, stream) : backward<float>(p, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_lru)

}  // namespace msel
