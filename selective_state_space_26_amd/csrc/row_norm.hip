// row_norm.hip -- the RMS norms over contiguous rows, forward and backward: the norm before a
// block with its residual sum and scale, and the gated norm over [batch, seqlen, dim].
//
// Per row of n values v (v = residual + scale x, or x silu(z), or x):
//   rstd = (sum v^2 / n + eps)^(-1/2),  out = v rstd w  (times silu(z) when the gate is last).
// Backward, with g = dout w (times silu(z) when the gate is last):
//   dv = rstd (g - v rstd^2 (sum g v) / n),  dw += dout v rstd (times silu(z), gate last),
// then dx and dz or the residual's gradient from dv.  rstd is recomputed: sum v^2 and sum g v
// come from the same registers in one pass.
//
// Each value is read once and written once, with a few operations in between, so HBM bounds
// both kernels.  A row stays in registers between its sum and its output: a team of W
// wavefronts holds it as kVecs vectors of VE elements per lane, W = 1, 4 or 16 by the row's
// width (one wavefront needs no barrier, wider rows need the lanes).  Teams walk rows with the
// grid's stride, so that the weights, and the backward's dweight sums, stay in registers too;
// a block adds its dweight sums over its teams in LDS and writes one row of partial sums, and a
// second kernel adds those in a fixed order (no atomics: deterministic).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

constexpr int kVecs = 4;  // vectors per lane
// elements per vector: 16 bytes of the wider type; 16 wavefronts (128 VGPRs each) hold 4
template <typename TA, typename TB>
constexpr int row_ve(int W) { return sizeof(TA) == 2 && sizeof(TB) == 2 && W < 16 ? 8 : 4; }

constexpr int team_threads(int W) { return 64 * W; }
constexpr int block_threads(int W) { return W == 1 ? 256 : 64 * W; }
constexpr int block_teams(int W) { return block_threads(W) / team_threads(W); }

// Blocks a launch aims for, over all groups: the threads that fit on 256 CUs at once.
constexpr int grid_target(int W) { return W == 1 ? 2048 : W == 4 ? 2048 : 512; }
// The backward writes a row of partial sums per block, so it takes fewer.
constexpr int bwd_grid_target(int W) { return W == 1 ? 1024 : W == 4 ? 1024 : 512; }

// Sum over a team; red: [2][16] floats of LDS per block (W > 1), alternating between calls so
// that one barrier per call suffices.
template <int W>
__device__ __forceinline__ float team_sum(float v, float (*red)[16], int& phase) {
    v = wave_sum_fused(v);
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6;
        if (lane_id() == 0) red[phase][wave] = v;
        __syncthreads();
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) t += red[phase][i];
        v = t;
        phase ^= 1;
    }
    return v;
}

// A team's row: vectors i = lane + k * team for k < kVecs that lie wholly in the row, and the
// last n % VE elements, one per lane.
template <typename T, int VE>
struct RowRegs {
    RawVec<T, VE> v[kVecs];
    float tail;
};

template <typename T, int VE, int TEAM>
__device__ __forceinline__ void load_row(const T* row, int n, int lane, RowRegs<T, VE>& r) {
    const int full = n / VE;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const int i = lane + k * TEAM;
        r.v[k].w = 0;
        if (i < full) r.v[k] = ld_raw<T, VE>(row + MSEL_SPAN(i * VE, VE, n));
    }
    r.tail = lane < n - full * VE ? Elem<T>::load1(row + MSEL_IDX(full * VE + lane, n)) : 0.0f;
}

#define MSEL_FOR_ROW(k) _Pragma("unroll") for (int k = 0; k < kVecs; ++k)

template <typename TA, typename TB, NormMode MODE, int W>
__global__ __launch_bounds__(block_threads(W)) void row_norm_fwd_kernel(RowNormParams p) {
    constexpr int VE = row_ve<TA, TB>(W);
    constexpr int TEAM = team_threads(W);
    constexpr int TEAMS = block_teams(W);
    using TO = std::conditional_t<MODE == NormMode::kResidual, TB, TA>;
    __shared__ float red[2][16];
    int phase = 0;
    const int n = p.n;
    const int full = n / VE;
    const int lane = threadIdx.x % TEAM;
    const int g = blockIdx.y;
    const float inv_n = 1.0f / static_cast<float>(n);

    RowRegs<float, VE> w;
    if (p.w != nullptr) {
        load_row<float, VE, TEAM>(p.w + static_cast<int64_t>(g) * n, n, lane, w);
    } else {
        MSEL_FOR_ROW(k)
#pragma unroll
        for (int e = 0; e < VE; ++e) w.v[k].w[e] = __float_as_uint(1.0f);
        w.tail = 1.0f;
    }

    // the team index is wave-uniform; W > 1 has one team, so its barriers are block-uniform
    const int team = TEAMS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const int64_t base = MSEL_SPAN((r * p.groups + g) * n, n, p.rows * p.groups * n);
        RowRegs<TA, VE> a;
        RowRegs<TB, VE> b;
        load_row<TA, VE, TEAM>(static_cast<const TA*>(p.a) + base, n, lane, a);
        if (p.b != nullptr) load_row<TB, VE, TEAM>(static_cast<const TB*>(p.b) + base, n, lane, b);

        float v[kVecs][VE], tail;
        float gate[MODE == NormMode::kGateLast ? kVecs : 1][VE], tgate = 0.0f;
        float sum = 0.0f;
        MSEL_FOR_ROW(k) {
            float av[VE], bv[VE];
            to_f32<TA, VE>(a.v[k], av);
            if (MODE != NormMode::kResidual || p.b != nullptr) to_f32<TB, VE>(b.v[k], bv);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if constexpr (MODE == NormMode::kResidual)
                    v[k][e] = p.b != nullptr ? fmaf(p.scale, av[e], bv[e]) : p.scale * av[e];
                else if constexpr (MODE == NormMode::kGateFirst)
                    v[k][e] = av[e] * silu_f(bv[e]);
                else {
                    v[k][e] = av[e];
                    gate[k][e] = silu_f(bv[e]);
                }
                sum = fmaf(v[k][e], v[k][e], sum);
            }
        }
        if constexpr (MODE == NormMode::kResidual)
            tail = p.b != nullptr ? fmaf(p.scale, a.tail, b.tail) : p.scale * a.tail;
        else if constexpr (MODE == NormMode::kGateFirst)
            tail = a.tail * silu_f(b.tail);
        else {
            tail = a.tail;
            tgate = silu_f(b.tail);
        }
        sum = fmaf(tail, tail, sum);

        if (MODE == NormMode::kResidual && p.out2 != nullptr) {
            TO* so = static_cast<TO*>(p.out2) + base;
            MSEL_FOR_ROW(k) {
                const int i = lane + k * TEAM;
                if (i < full) st_vec<TO, VE>(so + MSEL_SPAN(i * VE, VE, n), v[k]);
            }
            if (lane < n - full * VE) Elem<TO>::store1(so + MSEL_IDX(full * VE + lane, n), tail);
        }

        const float rstd = rstd_of(team_sum<W>(sum, red, phase), inv_n, p.eps);
        TA* out = static_cast<TA*>(p.out) + base;
        MSEL_FOR_ROW(k) {
            const int i = lane + k * TEAM;
            float wv[VE], o[VE];
            to_f32<float, VE>(w.v[k], wv);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = v[k][e] * rstd * wv[e];
                if constexpr (MODE == NormMode::kGateLast) o[e] *= gate[k][e];
            }
            if (i < full) st_vec<TA, VE>(out + MSEL_SPAN(i * VE, VE, n), o);
        }
        if (lane < n - full * VE) {
            float o = tail * rstd * w.tail;
            if constexpr (MODE == NormMode::kGateLast) o *= tgate;
            Elem<TA>::store1(out + MSEL_IDX(full * VE + lane, n), o);
        }
    }
}

// One element of the backward, given rstd and c = rstd^2 (sum g v) / n.
template <NormMode MODE>
__device__ __forceinline__ void bwd_element(float a, float b, float dy, float w, float rstd,
                                            float c, float scale, float& o1, float& o2,
                                            float& dw) {
    if constexpr (MODE == NormMode::kResidual) {
        const float ds = fmaf(rstd, fmaf(-a, c, dy * w), b);
        o1 = scale * ds;
        o2 = ds;
        dw = fmaf(dy, a * rstd, dw);
    } else {
        float gate, slope;
        silu_grad_f(b, gate, slope);
        if constexpr (MODE == NormMode::kGateFirst) {
            const float v = a * gate;
            const float dv = rstd * fmaf(-v, c, dy * w);
            o1 = dv * gate;
            o2 = dv * a * slope;
            dw = fmaf(dy, v * rstd, dw);
        } else {
            const float xh = a * rstd;
            o1 = rstd * fmaf(-a, c, dy * w * gate);
            o2 = dy * w * xh * slope;
            dw = fmaf(dy * gate, xh, dw);
        }
    }
}

// v and g v of one element, for the two sums.
template <NormMode MODE>
__device__ __forceinline__ void bwd_sums(float a, float b, float dy, float w, float& sv,
                                         float& sg) {
    float v = a, g = dy * w;
    if constexpr (MODE == NormMode::kGateFirst) v = a * silu_f(b);
    if constexpr (MODE == NormMode::kGateLast) g *= silu_f(b);
    sv = fmaf(v, v, sv);
    sg = fmaf(g, v, sg);
}

// TA: a, TB: b; T: dout and dx
template <typename T, typename TA, typename TB, NormMode MODE, int W>
__global__ __launch_bounds__(block_threads(W)) void row_norm_bwd_kernel(RowNormParams p) {
    constexpr int VE = row_ve<TA, T>(W);
    constexpr int TEAM = team_threads(W);
    constexpr int TEAMS = block_teams(W);
    constexpr int ROW = kVecs * VE * TEAM;  // floats of a team's dweight vectors
    __shared__ float red[2][16];
    __shared__ float comb[TEAMS > 1 ? (TEAMS - 1) * (ROW + 64) : 1];
    int phase = 0;
    const int n = p.n;
    const int full = n / VE;
    const int ntail = n - full * VE;
    const int lane = threadIdx.x % TEAM;
    const int g = blockIdx.y;
    const float inv_n = 1.0f / static_cast<float>(n);

    RowRegs<float, VE> w;
    if (p.w != nullptr) {
        load_row<float, VE, TEAM>(p.w + static_cast<int64_t>(g) * n, n, lane, w);
    } else {
        MSEL_FOR_ROW(k)
#pragma unroll
        for (int e = 0; e < VE; ++e) w.v[k].w[e] = __float_as_uint(1.0f);
        w.tail = 1.0f;
    }
    float dw[kVecs][VE] = {}, dwt = 0.0f;

    const int team = TEAMS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / TEAM);
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const int64_t base = MSEL_SPAN((r * p.groups + g) * n, n, p.rows * p.groups * n);
        RowRegs<TA, VE> a;
        RowRegs<TB, VE> b;
        RowRegs<T, VE> dy;
        load_row<TA, VE, TEAM>(static_cast<const TA*>(p.a) + base, n, lane, a);
        load_row<T, VE, TEAM>(static_cast<const T*>(p.dout) + base, n, lane, dy);
        MSEL_FOR_ROW(k) b.v[k].w = 0;
        b.tail = 0.0f;
        if (p.b != nullptr) load_row<TB, VE, TEAM>(static_cast<const TB*>(p.b) + base, n, lane, b);

        float sv = 0.0f, sg = 0.0f;
        MSEL_FOR_ROW(k) {
            float av[VE], bv[VE], dv[VE], wv[VE];
            to_f32<TA, VE>(a.v[k], av);
            to_f32<TB, VE>(b.v[k], bv);
            to_f32<T, VE>(dy.v[k], dv);
            to_f32<float, VE>(w.v[k], wv);
#pragma unroll
            for (int e = 0; e < VE; ++e) bwd_sums<MODE>(av[e], bv[e], dv[e], wv[e], sv, sg);
        }
        bwd_sums<MODE>(a.tail, b.tail, dy.tail, w.tail, sv, sg);
        sv = team_sum<W>(sv, red, phase);
        sg = team_sum<W>(sg, red, phase);
        const float rstd = rstd_of(sv, inv_n, p.eps);
        const float c = rstd * rstd * (sg * inv_n);

        T* o1 = static_cast<T*>(p.out);
        TB* o2 = static_cast<TB*>(p.out2);
        MSEL_FOR_ROW(k) {
            const int i = lane + k * TEAM;
            float av[VE], bv[VE], dv[VE], wv[VE], r1[VE], r2[VE];
            to_f32<TA, VE>(a.v[k], av);
            to_f32<TB, VE>(b.v[k], bv);
            to_f32<T, VE>(dy.v[k], dv);
            to_f32<float, VE>(w.v[k], wv);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                bwd_element<MODE>(av[e], bv[e], dv[e], wv[e], rstd, c, p.scale, r1[e], r2[e],
                                  dw[k][e]);
            if (i < full) {
                const int64_t at = base + MSEL_SPAN(i * VE, VE, n);
                if (o1 != nullptr) st_vec<T, VE>(o1 + at, r1);
                if (o2 != nullptr) st_vec<TB, VE>(o2 + at, r2);
            }
        }
        float r1, r2;
        bwd_element<MODE>(a.tail, b.tail, dy.tail, w.tail, rstd, c, p.scale, r1, r2, dwt);
        if (lane < ntail) {
            const int64_t at = base + MSEL_IDX(full * VE + lane, n);
            if (o1 != nullptr) Elem<T>::store1(o1 + at, r1);
            if (o2 != nullptr) Elem<TB>::store1(o2 + at, r2);
        }
    }

    if (p.dw_part == nullptr) return;
    // the teams' sums, added in team order by team 0
    if constexpr (TEAMS > 1) {
        if (team > 0) {
            float* mine = comb + (team - 1) * (ROW + 64);
            MSEL_FOR_ROW(k)
#pragma unroll
            for (int e = 0; e < VE; ++e)
                mine[MSEL_IDX((k * VE + e) * TEAM + lane, ROW)] = dw[k][e];
            mine[ROW + lane] = dwt;
        }
        __syncthreads();
        if (team > 0) return;
#pragma unroll
        for (int t = 0; t < TEAMS - 1; ++t) {
            const float* other = comb + t * (ROW + 64);
            MSEL_FOR_ROW(k)
#pragma unroll
            for (int e = 0; e < VE; ++e) dw[k][e] += other[(k * VE + e) * TEAM + lane];
            dwt += other[ROW + lane];
        }
    }
    float* out = p.dw_part + (static_cast<int64_t>(blockIdx.x) * p.groups + g) * n;
    MSEL_FOR_ROW(k) {
        const int i = lane + k * TEAM;
        if (i < full) st_vec<float, VE>(out + MSEL_SPAN(i * VE, VE, n), dw[k]);
    }
    if (lane < ntail) out[MSEL_IDX(full * VE + lane, n)] = dwt;
}

// Wavefronts per row: the fewest that hold it in kVecs vectors per lane.
int waves_for(int n, int ve) {
    if (n <= kVecs * ve * 64) return 1;
    return n <= kVecs * ve * 256 ? 4 : 16;  // 16 hold kMaxNormDim values at any ve
}

unsigned grid_of(int64_t rows, int groups, int W, bool bwd) {
    const int64_t want = (rows + block_teams(W) - 1) / block_teams(W);
    const int64_t target = std::max(1, (bwd ? bwd_grid_target(W) : grid_target(W)) / groups);
    return static_cast<unsigned>(std::min(want, target));
}

template <typename TA, typename TB, NormMode MODE>
hipError_t fwd_go(const RowNormParams& p, hipStream_t stream) {
    const int W = waves_for(p.n, row_ve<TA, TB>(1));
    const dim3 grid(grid_of(p.rows, p.groups, W, false), static_cast<unsigned>(p.groups));
    const dim3 block(static_cast<unsigned>(block_threads(W)));
    switch (W) {
        case 1:
            hipLaunchKernelGGL((row_norm_fwd_kernel<TA, TB, MODE, 1>), grid, block, 0, stream, p);
            break;
        case 4:
            hipLaunchKernelGGL((row_norm_fwd_kernel<TA, TB, MODE, 4>), grid, block, 0, stream, p);
            break;
        default:
            hipLaunchKernelGGL((row_norm_fwd_kernel<TA, TB, MODE, 16>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

template <typename T, typename TA, typename TB, NormMode MODE>
hipError_t bwd_go(RowNormParams p, hipStream_t stream) {
    const int W = waves_for(p.n, row_ve<TA, T>(1));
    const dim3 grid(grid_of(p.rows, p.groups, W, true), static_cast<unsigned>(p.groups));
    const bool one = grid.x == 1 && p.dw_part != nullptr;
    if (one) p.dw_part = p.dw;  // one row of partial sums is the sum
    const dim3 block(static_cast<unsigned>(block_threads(W)));
    switch (W) {
        case 1:
            hipLaunchKernelGGL((row_norm_bwd_kernel<T, TA, TB, MODE, 1>), grid, block, 0, stream,
                               p);
            break;
        case 4:
            hipLaunchKernelGGL((row_norm_bwd_kernel<T, TA, TB, MODE, 4>), grid, block, 0, stream,
                               p);
            break;
        default:
            hipLaunchKernelGGL((row_norm_bwd_kernel<T, TA, TB, MODE, 16>), grid, block, 0, stream,
                               p);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.dw_part == nullptr || one) return e;
    return launch_column_sums(p.dw_part, static_cast<int>(grid.x),
                              static_cast<int64_t>(p.groups) * p.n, p.dw, stream);
}

// dw[c] = sum_r part[r][c]: a block takes 64 columns, its 16 wavefronts every 16th row each,
// and their sums are added in wavefront order.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* part, int rows,
                                                           int64_t cols, float* dw) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int r = wave; r < rows; r += 16)
            s += part[MSEL_IDX(r * cols + c, static_cast<int64_t>(rows) * cols)];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += red[i][lane];
        dw[MSEL_IDX(c, cols)] = s;
    }
}

}  // namespace

hipError_t launch_column_sums(const float* part, int rows, int64_t cols, float* dw,
                              hipStream_t stream) {
    hipLaunchKernelGGL(column_sums_kernel, dim3(static_cast<unsigned>((cols + 63) / 64)),
                       dim3(1024), 0, stream, part, rows, cols, dw);
    return hipGetLastError();
}

int row_norm_partials(int64_t rows, int groups, int n, NormMode mode, bool bf16, bool rbf16) {
    const bool narrow = bf16 && (mode != NormMode::kResidual || rbf16);
    return static_cast<int>(grid_of(rows, groups, waves_for(n, narrow ? 8 : 4), true));
}

hipError_t launch_row_norm_fwd(const RowNormParams& p, NormMode mode, bool bf16, bool rbf16,
                               hipStream_t stream) {
    using M = NormMode;
    switch (mode) {
        case M::kResidual:
            if (!bf16) return fwd_go<float, float, M::kResidual>(p, stream);
            return rbf16 ? fwd_go<bf16_t, bf16_t, M::kResidual>(p, stream)
                         : fwd_go<bf16_t, float, M::kResidual>(p, stream);
        case M::kGateFirst:
            return bf16 ? fwd_go<bf16_t, bf16_t, M::kGateFirst>(p, stream)
                        : fwd_go<float, float, M::kGateFirst>(p, stream);
        case M::kGateLast:
            return bf16 ? fwd_go<bf16_t, bf16_t, M::kGateLast>(p, stream)
                        : fwd_go<float, float, M::kGateLast>(p, stream);
    }
    return hipErrorInvalidValue;
}

hipError_t launch_row_norm_bwd(const RowNormParams& p, NormMode mode, bool bf16, bool rbf16,
                               hipStream_t stream) {
    using M = NormMode;
    switch (mode) {
        case M::kResidual:
            if (!bf16) return bwd_go<float, float, float, M::kResidual>(p, stream);
            return rbf16 ? bwd_go<bf16_t, bf16_t, bf16_t, M::kResidual>(p, stream)
                         : bwd_go<bf16_t, float, float, M::kResidual>(p, stream);
        case M::kGateFirst:
            return bf16 ? bwd_go<bf16_t, bf16_t, bf16_t, M::kGateFirst>(p, stream)
                        : bwd_go<float, float, float, M::kGateFirst>(p, stream);
        case M::kGateLast:
            return bf16 ? bwd_go<bf16_t, bf16_t, bf16_t, M::kGateLast>(p, stream)
                        : bwd_go<float, float, float, M::kGateLast>(p, stream);
    }
    return hipErrorInvalidValue;
}

MSEL_BOUNDS_TAKER(take_bounds_row_norm)

}  // namespace msel
