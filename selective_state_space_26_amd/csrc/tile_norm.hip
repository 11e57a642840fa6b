// tile_norm.hip -- the gated norm after the scan, forward, over the channels of
// [batch, dim, seqlen], to the same layout or turned to [batch, seqlen, dim]:
//   gate first:  v = x silu(z),  out = v rstd(v) w;   gate last:  out = x rstd(x) w silu(z),
//   rstd(v) = (sum over the group's n channels of v^2 / n + eps)^(-1/2).
// HBM bounds it: x and z read, out written (the tiles are described in tile_norm.hpp).
#include <hip/hip_runtime.h>

#include "tile_norm.hpp"

namespace msel {

namespace {

// NIT: passes whose values stay in registers between the sum and the output; 0: any number of
// passes, read again for the output.
template <typename T, bool FIRST, bool OUT_BLD, int TT, int THREADS, int NIT>
__global__ __launch_bounds__(THREADS) void tile_norm_fwd_kernel(TileNormParams p) {
    using Sh = TileShape<T, TT, THREADS>;
    constexpr int VE = Sh::VE, VL = Sh::VL, CPB = Sh::CPB;
    __shared__ float red[Sh::WAVES * TT];
    __shared__ TurnTile<T, TT, THREADS> turn[OUT_BLD ? 2 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int vl = tid % VL, ch = tid / VL;
    const int tile = static_cast<int>(xcd_order(blockIdx.x, gridDim.x));
    const int b = tile / p.tiles;
    const int t0 = (tile - b * p.tiles) * TT;
    const int t = t0 + vl * VE;
    const int valid = p.L - t;  // of this lane's tokens, may be <= 0
    const int c0 = blockIdx.y * p.n;
    [[maybe_unused]] const int64_t elems = static_cast<int64_t>(p.B) * p.D * p.L;
    const T* x = static_cast<const T*>(p.x);
    const T* z = static_cast<const T*>(p.z);
    const bool whole = t0 + TT <= p.L;  // block-uniform

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

    constexpr int R = NIT > 0 ? NIT : 1;
    RawVec<T, VE> rx[R], rz[R];
    float acc[VE] = {};
    const auto add = [&](const RawVec<T, VE>& ax, const RawVec<T, VE>& az) {
        float xv[VE], zv[VE];
        to_f32<T, VE>(ax, xv);
        to_f32<T, VE>(az, zv);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const float v = FIRST ? xv[k] * silu_f(zv[k]) : xv[k];
            acc[k] = fmaf(v, v, acc[k]);
        }
    };
    const int passes = (p.n + CPB - 1) / CPB;
    if constexpr (NIT > 0) {
#pragma unroll
        for (int i = 0; i < NIT; ++i) {
            rx[i] = load(x, i * CPB + ch);
            rz[i] = load(z, i * CPB + ch);
        }
#pragma unroll
        for (int i = 0; i < NIT; ++i) add(rx[i], rz[i]);
    } else {
        for (int i = 0; i < passes; ++i) add(load(x, i * CPB + ch), load(z, i * CPB + ch));
    }
    tile_sum<VE, VL, Sh::WAVES, TT>(acc, red, lane, wave);
    float rstd[VE];
    const float inv_n = 1.0f / static_cast<float>(p.n);
#pragma unroll
    for (int k = 0; k < VE; ++k) rstd[k] = rstd_of(acc[k], inv_n, p.eps);

    T* out = static_cast<T*>(p.out);
    const auto emit = [&](int i, const RawVec<T, VE>& ax, const RawVec<T, VE>& az) {
        const int c = i * CPB + ch;
        const float w =
            c < p.n && p.w != nullptr ? p.w[MSEL_IDX(c0 + c, p.D)] : 1.0f;
        float xv[VE], zv[VE], o[VE];
        to_f32<T, VE>(ax, xv);
        to_f32<T, VE>(az, zv);
#pragma unroll
        for (int k = 0; k < VE; ++k) o[k] = xv[k] * silu_f(zv[k]) * rstd[k] * w;
        if constexpr (OUT_BLD) {
            auto& tl = turn[i & 1];
            tl.put_tokens(vl, ch, o);
            // one barrier per pass: the buffer of pass i is written again in pass i + 2, whose
            // writes come after the barrier of pass i + 1, hence after every read of pass i
            __syncthreads();
            const int row = tid / Sh::RV, cv = (tid % Sh::RV) * VE;
            const int left = p.n - (i * CPB + cv);
            if (t0 + row < p.L && left > 0) {
                const int64_t o0 =
                    (static_cast<int64_t>(b) * p.L + t0 + row) * p.D + c0 + i * CPB + cv;
                st_part<T, VE>(out + MSEL_SPAN(o0, left < VE ? left : VE, elems),
                               tl.get_channels(row, cv), left);
            }
        } else if (c < p.n && valid > 0) {
            st_part<T, VE>(out + MSEL_SPAN(at(c), valid < VE ? valid : VE, elems),
                           from_f32<T, VE>(o), valid);
        }
    };
    if constexpr (NIT > 0) {
#pragma unroll
        for (int i = 0; i < NIT; ++i)
            if (i < passes) emit(i, rx[i], rz[i]);
    } else {
        for (int i = 0; i < passes; ++i) emit(i, load(x, i * CPB + ch), load(z, i * CPB + ch));
    }
}

template <typename T, bool FIRST, bool OUT_BLD>
hipError_t tile_fwd_go(TileNormParams p, hipStream_t stream) {
    constexpr int TT = 32, THREADS = 512;
    p.tiles = (p.L + TT - 1) / TT;
    const dim3 grid(static_cast<unsigned>(p.B) * static_cast<unsigned>(p.tiles),
                    static_cast<unsigned>(p.groups));
    hipLaunchKernelGGL((tile_norm_fwd_kernel<T, FIRST, OUT_BLD, TT, THREADS, 0>), grid,
                       dim3(THREADS), 0, stream, p);
    return hipGetLastError();
}

template <typename T>
hipError_t tile_fwd(const TileNormParams& p, bool gate_first, hipStream_t stream) {
    if (gate_first)
        return p.out_bld ? tile_fwd_go<T, true, true>(p, stream)
                         : tile_fwd_go<T, true, false>(p, stream);
    return p.out_bld ? tile_fwd_go<T, false, true>(p, stream)
                     : tile_fwd_go<T, false, false>(p, stream);
}

}  // namespace

hipError_t launch_tile_norm_fwd(const TileNormParams& p, bool gate_first, bool bf16,
                                hipStream_t stream) {
    return bf16 ? tile_fwd<bf16_t>(p, gate_first, stream) : tile_fwd<float>(p, gate_first, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_tile_norm)

}  // namespace msel
