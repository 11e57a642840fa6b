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
// both kernels.  A row stays in registers between its sum and its output: a team of 16, 64, 256 or
// 1024 lanes holds it as NV vectors of VE elements per lane, by the row's width (up to a wavefront
// needs no barrier, wider rows need the lanes; narrow rows in small teams leave no lane to work on
// nothing).  Teams walk rows with the grid's stride, so that the weights, and the backward's
// dweight sums, stay in registers too; a block adds its dweight sums over its teams in LDS and
// writes one row of partial sums, and a second kernel adds those in a fixed order (no atomics:
// deterministic).
// Measured: 16384 x 768 bf16 with an fp32 residual 25 us forward (151 MB) and 34 us backward, 5 more
// for the sum (201 MB), both at the rate of a copy or above it, as a part is still in the last-level
// cache; 4099 x 2561 fp32 forward 30 us (168 MB); 200000 x 64 bf16 backward 27 us (128 MB), 152 with
// a wavefront per row; one row of 768 2.3 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

// elements per vector: 16 bytes of the wider type; 16 wavefronts (128 VGPRs each) hold 4
template <typename TA, typename TB>
constexpr int row_ve(int team) { return sizeof(TA) == 2 && sizeof(TB) == 2 && team < 1024 ? 8 : 4; }

constexpr int block_threads(int team) { return team < 256 ? 256 : team; }
constexpr int block_teams(int team) { return block_threads(team) / team; }

// Partial rows that one block per 64 columns adds; more are first added in spans (1024 x 768: 5.0
// us in one launch, 8.6 in two; 4096 x 128: 38 and 9.5).
constexpr int64_t kSumRows = 2048, kSumSpan = 64;

// Blocks a launch aims for, over all groups: the threads that fit on 256 CUs at once.
constexpr int grid_target(int team) { return team <= 256 ? 2048 : 512; }
// The backward writes a row of partial sums per block, so it takes fewer of wide rows.
constexpr int bwd_grid_target(int team, int vecs) {
    return vecs == 1 ? 2048 : team <= 256 ? 1024 : 512;
}

// Sum over a team of 16, 64, 256 or 1024 lanes; red: [2][16] floats of LDS per block (several
// wavefronts), alternating between calls so that one barrier per call suffices.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float (*red)[16], int& phase) {
    if constexpr (TEAM == 16) {  // one row of lanes, rotated by 8, 4, 2 and 1
        const auto rot = [](float x, auto ctrl) {
            return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x),
                                                              decltype(ctrl)::value, 0xf, 0xf, true));
        };
        v += rot(v, std::integral_constant<int, 0x128>{});
        v += rot(v, std::integral_constant<int, 0x124>{});
        v += rot(v, std::integral_constant<int, 0x122>{});
        v += rot(v, std::integral_constant<int, 0x121>{});
        return v;
    }
    v = wave_sum_fused(v);
    if constexpr (TEAM > 64) {
        const int wave = threadIdx.x >> 6;
        if (lane_id() == 0) red[phase][wave] = v;
        __syncthreads();
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < TEAM / 64; ++i) t += red[phase][i];
        v = t;
        phase ^= 1;
    }
    return v;
}

// The team of this thread in its block; uniform over a wavefront where a team has one or more.
template <int TEAM>
__device__ __forceinline__ int team_index() {
    if constexpr (block_teams(TEAM) == 1) return 0;
    const int t = static_cast<int>(threadIdx.x) / TEAM;
    return TEAM < 64 ? t : __builtin_amdgcn_readfirstlane(t);
}

// A team's row: vectors i = lane + k * team for k < NV that lie wholly in the row, and the
// last n % VE elements, one per lane.
template <typename T, int VE, int NV>
struct RowRegs {
    RawVec<T, VE> v[NV];
    float tail;
};

template <int TEAM, typename T, int VE, int NV>
__device__ __forceinline__ void load_row(const T* row, int n, int lane, RowRegs<T, VE, NV>& r) {
    const int full = n / VE;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int i = lane + k * TEAM;
        r.v[k].w = 0;
        if (i < full) r.v[k] = ld_raw<T, VE>(row + MSEL_SPAN(i * VE, VE, n));
    }
    r.tail = lane < n - full * VE ? Elem<T>::load1(row + MSEL_IDX(full * VE + lane, n)) : 0.0f;
}

#define MSEL_FOR_ROW(k) _Pragma("unroll") for (int k = 0; k < NV; ++k)

template <typename TA, typename TB, NormMode MODE, int TEAM, int NV>
__global__ __launch_bounds__(block_threads(TEAM)) void row_norm_fwd_kernel(RowNormParams p) {
    constexpr int VE = row_ve<TA, TB>(TEAM);
    constexpr int TEAMS = block_teams(TEAM);
    using TO = std::conditional_t<MODE == NormMode::kResidual, TB, TA>;
    __shared__ float red[2][16];
    int phase = 0;
    const int n = p.n;
    const int full = n / VE;
    const int lane = threadIdx.x % TEAM;
    const int g = blockIdx.y;
    const float inv_n = 1.0f / static_cast<float>(n);

    RowRegs<float, VE, NV> w;
    if (p.w != nullptr) {
        load_row<TEAM>(p.w + static_cast<int64_t>(g) * n, n, lane, w);
    } else {
        MSEL_FOR_ROW(k)
#pragma unroll
        for (int e = 0; e < VE; ++e) w.v[k].w[e] = __float_as_uint(1.0f);
        w.tail = 1.0f;
    }

    // a team of several wavefronts is alone in its block, so its barriers are block-uniform
    const int team = team_index<TEAM>();
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const int64_t base = MSEL_SPAN((r * p.groups + g) * n, n, p.rows * p.groups * n);
        RowRegs<TA, VE, NV> a;
        RowRegs<TB, VE, NV> b;
        load_row<TEAM>(static_cast<const TA*>(p.a) + base, n, lane, a);
        if (p.b != nullptr) load_row<TEAM>(static_cast<const TB*>(p.b) + base, n, lane, b);

        float v[NV][VE], tail;
        float gate[MODE == NormMode::kGateLast ? NV : 1][VE], tgate = 0.0f;
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

        const float rstd = rstd_of(team_sum<TEAM>(sum, red, phase), inv_n, p.eps);
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
template <typename T, typename TA, typename TB, NormMode MODE, int TEAM, int NV>
__global__ __launch_bounds__(block_threads(TEAM)) void row_norm_bwd_kernel(RowNormParams p) {
    constexpr int VE = row_ve<TA, T>(TEAM);
    constexpr int TEAMS = block_teams(TEAM);
    constexpr int ROW = NV * VE * TEAM;  // floats of a team's dweight vectors
    __shared__ float red[2][16];
    __shared__ float comb[TEAMS > 1 ? (TEAMS - 1) * (ROW + TEAM) : 1];
    int phase = 0;
    const int n = p.n;
    const int full = n / VE;
    const int ntail = n - full * VE;
    const int lane = threadIdx.x % TEAM;
    const int g = blockIdx.y;
    const float inv_n = 1.0f / static_cast<float>(n);

    RowRegs<float, VE, NV> w;
    if (p.w != nullptr) {
        load_row<TEAM>(p.w + static_cast<int64_t>(g) * n, n, lane, w);
    } else {
        MSEL_FOR_ROW(k)
#pragma unroll
        for (int e = 0; e < VE; ++e) w.v[k].w[e] = __float_as_uint(1.0f);
        w.tail = 1.0f;
    }
    float dw[NV][VE] = {}, dwt = 0.0f;

    const int team = team_index<TEAM>();
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * TEAMS + team; r < p.rows;
         r += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const int64_t base = MSEL_SPAN((r * p.groups + g) * n, n, p.rows * p.groups * n);
        RowRegs<TA, VE, NV> a;
        RowRegs<TB, VE, NV> b;
        RowRegs<T, VE, NV> dy;
        load_row<TEAM>(static_cast<const TA*>(p.a) + base, n, lane, a);
        load_row<TEAM>(static_cast<const T*>(p.dout) + base, n, lane, dy);
        MSEL_FOR_ROW(k) b.v[k].w = 0;
        b.tail = 0.0f;
        if (p.b != nullptr) load_row<TEAM>(static_cast<const TB*>(p.b) + base, n, lane, b);

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
        sv = team_sum<TEAM>(sv, red, phase);
        sg = team_sum<TEAM>(sg, red, phase);
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
            float* mine = comb + (team - 1) * (ROW + TEAM);
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
            const float* other = comb + t * (ROW + TEAM);
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

// Lanes per row and vectors per lane: the fewest that hold it, so that no lane works on vectors
// beyond it.
struct RowTeam {
    int team, vecs;
};
RowTeam team_for(int n, int ve) {
    if (n <= 16 * ve) return {16, 1};
    if (n <= 64 * ve) return {64, 1};
    if (n <= 4 * 64 * ve) return {64, 4};
    return {n <= 4 * 256 * ve ? 256 : 1024, 4};  // 1024 hold kMaxNormDim values at any ve
}

unsigned grid_of(int64_t rows, int groups, RowTeam t, bool bwd) {
    const int64_t want = (rows + block_teams(t.team) - 1) / block_teams(t.team);
    const int all = bwd ? bwd_grid_target(t.team, t.vecs) : grid_target(t.team);
    return static_cast<unsigned>(std::min<int64_t>(want, std::max(1, all / groups)));
}

// Calls go with the team's lanes and vectors as constants.
template <typename F>
void with_team(RowTeam t, F&& go) {
    using std::integral_constant;
    if (t.team == 16) return go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    if (t.team == 64 && t.vecs == 1)
        return go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (t.team == 64) return go(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (t.team == 256) return go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    return go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <typename TA, typename TB, NormMode MODE>
hipError_t fwd_go(const RowNormParams& p, hipStream_t stream) {
    const RowTeam t = team_for(p.n, row_ve<TA, TB>(64));
    const dim3 grid(grid_of(p.rows, p.groups, t, false), static_cast<unsigned>(p.groups));
    with_team(t, [&](auto team, auto vecs) {
        constexpr int TEAM = decltype(team)::value, NV = decltype(vecs)::value;
        hipLaunchKernelGGL((row_norm_fwd_kernel<TA, TB, MODE, TEAM, NV>), grid,
                           dim3(block_threads(TEAM)), 0, stream, p);
    });
    return hipGetLastError();
}

template <typename T, typename TA, typename TB, NormMode MODE>
hipError_t bwd_go(RowNormParams p, hipStream_t stream) {
    const RowTeam t = team_for(p.n, row_ve<TA, T>(64));
    const dim3 grid(grid_of(p.rows, p.groups, t, true), static_cast<unsigned>(p.groups));
    const bool one = grid.x == 1 && p.dw_part != nullptr;
    if (one) p.dw_part = p.dw;  // one row of partial sums is the sum
    with_team(t, [&](auto team, auto vecs) {
        constexpr int TEAM = decltype(team)::value, NV = decltype(vecs)::value;
        hipLaunchKernelGGL((row_norm_bwd_kernel<T, TA, TB, MODE, TEAM, NV>), grid,
                           dim3(block_threads(TEAM)), 0, stream, p);
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.dw_part == nullptr || one) return e;
    return launch_column_sums(p.dw_part, grid.x, static_cast<int64_t>(p.groups) * p.n, p.dw, stream);
}

// Sums of `span` rows of part[rows][cols] each, into the first of them (blockIdx.y: which), or of
// all rows into dw: a block takes 64 columns, its 16 wavefronts every 16th row each, and their
// sums are added in wavefront order.  Rows are `step` rows of the buffer apart.
__global__ __launch_bounds__(1024) void column_sums_kernel(float* part, int64_t rows, int64_t step,
                                                           int64_t span, int64_t cols, float* dw) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    const int64_t r0 = blockIdx.y * span, r1 = min(rows, r0 + span);
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = r0 + wave; r < r1; r += 16)
            s += part[MSEL_IDX(r * step * cols + c, ((rows - 1) * step + 1) * cols)];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 16; ++i) s += red[i][lane];
        if (dw != nullptr)
            dw[MSEL_IDX(c, cols)] = s;
        else
            part[MSEL_IDX(r0 * cols + c, rows * cols)] = s;
    }
}

}  // namespace

hipError_t launch_column_sums(float* part, int64_t rows, int64_t cols, float* dw,
                              hipStream_t stream) {
    const unsigned slabs = static_cast<unsigned>((cols + 63) / 64);
    int64_t step = 1;
    if (rows > kSumRows) {
        // many rows under few columns: first over spans of rows, in place
        const int64_t span = std::max<int64_t>(kSumSpan, (rows + kSumRows - 1) / kSumRows);
        const int64_t spans = (rows + span - 1) / span;
        hipLaunchKernelGGL(column_sums_kernel, dim3(slabs, static_cast<unsigned>(spans)), dim3(1024),
                           0, stream, part, rows, int64_t(1), span, cols, nullptr);
        step = span;
        rows = spans;
    }
    hipLaunchKernelGGL(column_sums_kernel, dim3(slabs), dim3(1024), 0, stream, part, rows, step,
                       rows, cols, dw);
    return hipGetLastError();
}

int row_norm_partials(int64_t rows, int groups, int n, NormMode mode, bool bf16, bool rbf16) {
    const bool narrow = bf16 && (mode != NormMode::kResidual || rbf16);
    return static_cast<int>(grid_of(rows, groups, team_for(n, narrow ? 8 : 4), true));
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
