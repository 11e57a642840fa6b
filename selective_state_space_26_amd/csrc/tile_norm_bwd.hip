// tile_norm_bwd.hip -- backward of the gated norm over the channels of [batch, dim, seqlen],
// dout in the same layout or [batch, seqlen, dim].  With g = dout w (times silu(z) when the
// gate is last) and v = x silu(z) (x when it is last):
//   dv = rstd (g - v rstd^2 sum(g v) / n),  dw += dout v rstd (times silu(z), gate last),
//   gate first: dx = dv silu(z), dz = dv x silu'(z);
//   gate last:  dx = dv,         dz = dout w x rstd silu'(z).
// The gate and rstd are recomputed.  HBM bounds it: x, z and dout read, dx and dz written (the
// tiles are described in tile_norm.hpp).  Blocks walk tiles with the grid's stride and keep
// their channels' dweight sums in LDS (one lane adds to each, no atomics); a second kernel adds
// the blocks' sums in block order.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "tile_norm.hpp"

namespace msel {

namespace {

// Blocks of a launch over all groups: each writes a row of partial dweight sums.
constexpr int kBwdBlocks = 512;

template <typename T, bool FIRST, bool DOUT_BLD, int TT, int THREADS, int NIT>
__global__ __launch_bounds__(THREADS) void tile_norm_bwd_kernel(TileNormParams p) {
    using Sh = TileShape<T, TT, THREADS>;
    constexpr int VE = Sh::VE, VL = Sh::VL, CPB = Sh::CPB;
    __shared__ float red[2][Sh::WAVES * TT];
    __shared__ TurnTile<T, TT, THREADS> turn[DOUT_BLD ? 2 : 1];
    extern __shared__ float dwl[];  // [passes * CPB]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int vl = tid % VL, ch = tid / VL;
    const int c0 = blockIdx.y * p.n;
    [[maybe_unused]] const int64_t elems = static_cast<int64_t>(p.B) * p.D * p.L;
    const T* x = static_cast<const T*>(p.x);
    const T* z = static_cast<const T*>(p.z);
    const T* dout = static_cast<const T*>(p.dout);
    T* dx = static_cast<T*>(p.out);
    T* dz = static_cast<T*>(p.dz);
    const float inv_n = 1.0f / static_cast<float>(p.n);
    const int passes = (p.n + CPB - 1) / CPB;
    const int ntiles = p.B * p.tiles;  // < 2^31: checked on the host
    if (vl == 0)
        for (int i = 0; i < passes; ++i) dwl[i * CPB + ch] = 0.0f;  // this lane's alone

    for (int tile = static_cast<int>(xcd_order(blockIdx.x, gridDim.x)); tile < ntiles;
         tile += static_cast<int>(gridDim.x)) {
        const int b = tile / p.tiles;
        const int t0 = (tile - b * p.tiles) * TT;
        const int t = t0 + vl * VE;
        const int valid = p.L - t;
        const bool whole = t0 + TT <= p.L;
        const auto at = [&](int c) {
            return (static_cast<int64_t>(b) * p.D + c0 + c) * p.L + t;
        };
        const auto load = [&](const T* q, int c) {
            RawVec<T, VE> r;
            r.w = 0;
            if (whole) {
                if (c < p.n) r = ld_raw<T, VE>(q + MSEL_SPAN(at(c), VE, elems));
            } else if (c < p.n && valid > 0) {
                r = ld_part<T, VE>(q + MSEL_SPAN(at(c), valid < VE ? valid : VE, elems), valid);
            }
            return r;
        };
        // dout of pass i: this lane's tokens of its channel
        const auto load_dout = [&](int i) {
            if constexpr (!DOUT_BLD) {
                return load(dout, i * CPB + ch);
            } else {
                const int row = tid / Sh::RV, cv = (tid % Sh::RV) * VE;
                const int left = p.n - (i * CPB + cv);
                RawVec<T, VE> r;
                r.w = 0;
                if (t0 + row < p.L && left > 0) {
                    const int64_t o0 =
                        (static_cast<int64_t>(b) * p.L + t0 + row) * p.D + c0 + i * CPB + cv;
                    r = ld_part<T, VE>(dout + MSEL_SPAN(o0, left < VE ? left : VE, elems), left);
                }
                return r;
            }
        };
        // turned to tokens through LDS when it came as rows; one barrier per pass (a buffer is
        // written again two passes later)
        const auto turn_dout = [&](int i, const RawVec<T, VE>& r, float (&dy)[VE]) {
            if constexpr (!DOUT_BLD) {
                to_f32<T, VE>(r, dy);
            } else {
                auto& tl = turn[i & 1];
                tl.put_channels(tid / Sh::RV, (tid % Sh::RV) * VE, r);
                __syncthreads();
                tl.get_tokens(vl, ch, dy);
            }
        };
        const auto weight = [&](int c) {
            return c < p.n && p.w != nullptr ? p.w[MSEL_IDX(c0 + c, p.D)] : 1.0f;
        };

        float sv[VE] = {}, sg[VE] = {};
        for (int i = 0; i < passes; ++i) {
            const int c = i * CPB + ch;
            float xv[VE], zv[VE], dy[VE];
            to_f32<T, VE>(load(x, c), xv);
            to_f32<T, VE>(load(z, c), zv);
            turn_dout(i, load_dout(i), dy);
            const float w = weight(c);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                const float gate = silu_f(zv[k]);
                const float v = FIRST ? xv[k] * gate : xv[k];
                const float g = FIRST ? dy[k] * w : dy[k] * w * gate;
                sv[k] = fmaf(v, v, sv[k]);
                sg[k] = fmaf(g, v, sg[k]);
            }
        }
        if constexpr (DOUT_BLD) __syncthreads();
        tile_sum<VE, VL, Sh::WAVES, TT>(sv, red[0], lane, wave);
        tile_sum<VE, VL, Sh::WAVES, TT>(sg, red[1], lane, wave);
        float rstd[VE], cf[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            rstd[k] = rstd_of(sv[k], inv_n, p.eps);
            cf[k] = rstd[k] * rstd[k] * (sg[k] * inv_n);
        }
        for (int i = 0; i < passes; ++i) {
            const int c = i * CPB + ch;
            float xv[VE], zv[VE], dy[VE], gx[VE], gz[VE];
            to_f32<T, VE>(load(x, c), xv);
            to_f32<T, VE>(load(z, c), zv);
            turn_dout(i, load_dout(i), dy);
            const float w = weight(c);
            float dw = 0.0f;
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                float gate, slope;
                silu_grad_f(zv[k], gate, slope);
                if constexpr (FIRST) {
                    const float v = xv[k] * gate;
                    const float dv = rstd[k] * fmaf(-v, cf[k], dy[k] * w);
                    gx[k] = dv * gate;
                    gz[k] = dv * xv[k] * slope;
                    dw = fmaf(dy[k], v * rstd[k], dw);
                } else {
                    const float xh = xv[k] * rstd[k];
                    gx[k] = rstd[k] * fmaf(-xv[k], cf[k], dy[k] * w * gate);
                    gz[k] = dy[k] * w * xh * slope;
                    dw = fmaf(dy[k] * gate, xh, dw);
                }
            }
            if (c < p.n && valid > 0) {
                const int64_t o0 = MSEL_SPAN(at(c), valid < VE ? valid : VE, elems);
                st_part<T, VE>(dx + o0, from_f32<T, VE>(gx), valid);
                st_part<T, VE>(dz + o0, from_f32<T, VE>(gz), valid);
            }
#pragma unroll
            for (int m = 1; m < VL; m *= 2) dw += __shfl_xor(dw, m);
            if (vl == 0) dwl[MSEL_IDX(c, passes * CPB)] += dw;
        }
        __syncthreads();  // red and turn are free again
    }
    if (p.dw_part == nullptr) return;
    float* out = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.D + c0;
    if (vl == 0)
        for (int i = 0; i < passes; ++i)
            if (i * CPB + ch < p.n) out[MSEL_IDX(i * CPB + ch, p.n)] = dwl[i * CPB + ch];
}

int bwd_blocks(int B, int tiles, int groups) {
    return static_cast<int>(std::min<int64_t>(static_cast<int64_t>(B) * tiles,
                                              std::max(1, kBwdBlocks / groups)));
}

constexpr int kTT = 32, kThreads = 512;

template <typename T, bool FIRST, bool DOUT_BLD>
hipError_t tile_bwd_go(TileNormParams p, hipStream_t stream) {
    using Sh = TileShape<T, kTT, kThreads>;
    p.tiles = (p.L + kTT - 1) / kTT;
    const dim3 grid(static_cast<unsigned>(bwd_blocks(p.B, p.tiles, p.groups)),
                    static_cast<unsigned>(p.groups));
    const int lds = (p.n + Sh::CPB - 1) / Sh::CPB * Sh::CPB * static_cast<int>(sizeof(float));
    constexpr auto kern = tile_norm_bwd_kernel<T, FIRST, DOUT_BLD, kTT, kThreads, 0>;
    hipError_t e = allow_dynamic_lds<kern>(kMaxNormDim * static_cast<int>(sizeof(float)));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, grid, dim3(kThreads), static_cast<size_t>(lds), stream, p);
    e = hipGetLastError();
    if (e != hipSuccess || p.dw_part == nullptr) return e;
    return launch_column_sums(p.dw_part, static_cast<int>(grid.x), p.D, p.dw, stream);
}

template <typename T>
hipError_t tile_bwd(const TileNormParams& p, bool gate_first, hipStream_t stream) {
    if (gate_first)
        return p.out_bld ? tile_bwd_go<T, true, true>(p, stream)
                         : tile_bwd_go<T, true, false>(p, stream);
    return p.out_bld ? tile_bwd_go<T, false, true>(p, stream)
                     : tile_bwd_go<T, false, false>(p, stream);
}

}  // namespace

int tile_norm_partials(int B, int D, int L, int groups, bool, bool) {
    (void)D;
    return bwd_blocks(B, (L + kTT - 1) / kTT, groups);
}

hipError_t launch_tile_norm_bwd(const TileNormParams& p, bool gate_first, bool bf16,
                                hipStream_t stream) {
    return bf16 ? tile_bwd<bf16_t>(p, gate_first, stream) : tile_bwd<float>(p, gate_first, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_tile_norm_bwd)

}  // namespace msel
