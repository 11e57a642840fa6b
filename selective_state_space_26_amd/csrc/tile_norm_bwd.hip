// tile_norm_bwd.hip -- backward of the gated norm over the channels of [batch, dim, seqlen],
// dout in the same layout or [batch, seqlen, dim].  With g = dout w (times silu(z) when the
// gate is last) and v = x silu(z) (x when it is last):
//   dv = rstd (g - v rstd^2 sum(g v) / n),  dw += dout v rstd (times silu(z), gate last),
//   gate first: dx = dv silu(z), dz = dv x silu'(z);
//   gate last:  dx = dv,         dz = dout w x rstd silu'(z).
// The gate and rstd are recomputed.  HBM bounds it: x, z and dout read, dx and dz written (the
// tiles are described in tile_norm.hpp).  A tile also writes its tokens' share of dweight, a row
// of partial sums, and a second kernel adds the rows in a fixed order (no atomics:
// deterministic).
// Measured: 8 x 1536 x 2048 bf16 from rows 70 us and 5 for the sum (252 MB, 3.6 TB/s; VALU busy 45%),
// 5120 x 16384 257 us (839 MB, 3.3 TB/s, two passes read twice).  As in the forward, a CU holds one
// tile, and its loads, arithmetic and stores follow one another.
#include <hip/hip_runtime.h>

#include "tile_norm.hpp"

namespace msel {

namespace {

// NIT: passes kept in registers, NL: passes after them kept in LDS (a thread's own words; no
// barrier), STREAM: there may be more, which are read twice.
template <typename T, bool FIRST, bool DOUT_BLD, int SB, int THREADS, int NIT, int NL,
          bool STREAM, bool PAST>
__global__ __launch_bounds__(THREADS) void tile_norm_bwd_kernel(TileNormParams p) {
    using Sh = TileShape<T, SB, THREADS>;
    using Rows = RowLane<T, SB, THREADS>;
    using Vec = RawVec<T, Sh::VE>;
    constexpr int VE = Sh::VE, TT = Sh::TT, CPB = Sh::CPB;
    __shared__ float red[2 * Sh::WAVES * TT];
    __shared__ float tok[2 * TT];  // rstd and c of the tile's tokens
    __shared__ std::conditional_t<DOUT_BLD, TurnTile<T, SB, THREADS>, NoTile> turn[2];
    constexpr int HELD = NIT + NL;
    __shared__ decltype(Vec::w) held[NL > 0 ? NL : 1][3][NL > 0 ? THREADS : 1];
    const int tid = threadIdx.x;
    const TileLane<T, SB, THREADS> me(p, tid);
    const int tile = tile_of_block();
    if (tile >= p.B * p.tiles) return;  // block-uniform
    const TilePlace<TT> at(p, tile);
    const int c0 = blockIdx.y * p.n;

    const auto load_dout = [&](int c) {
        if constexpr (DOUT_BLD) return Rows::load(p, p.dout, at, c0, c, tid);
        else return me.load(p, p.dout, at, c0, c);
    };
    // dout that came as rows, turned through LDS; one barrier per pass (a buffer is written again
    // two passes later, after the barrier of the pass between)
    const auto turned = [&](const Vec& d, int buf) {
        if constexpr (DOUT_BLD) {
            turn[buf].put_group(tid, d);
            __syncthreads();
            return turn[buf].get_tokens(me.vl, me.ch);
        } else {
            return d;
        }
    };
    const auto weight = [&](int c) {
        const int ch = c + me.ch;
        return ch < p.n && p.w != nullptr ? p.w[MSEL_IDX(c0 + ch, p.D)] : 1.0f;
    };

    Vec x[NIT > 0 ? NIT : 1], z[NIT > 0 ? NIT : 1], d[NIT > 0 ? NIT : 1];
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        x[i].w = 0;
        z[i].w = 0;
        d[i].w = 0;
        if (i * CPB < p.n) {  // block-uniform, here and below
            x[i] = me.load(p, p.x, at, c0, i * CPB);
            z[i] = me.load(p, p.z, at, c0, i * CPB);
            d[i] = load_dout(i * CPB);
        }
    }
    float acc[2][VE] = {};  // sums of v^2 and of g v
    const auto add = [&](int c, const Vec& ax, const Vec& az, const Vec& ad) {
        const float w = weight(c);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            // g v is dout w x silu(z) in either order
            const float xk = elem_of(ax, k), xg = xk * silu_f(elem_of(az, k));
            const float v = FIRST ? xg : xk;
            acc[0][k] = fmaf(v, v, acc[0][k]);
            acc[1][k] = fmaf(elem_of(ad, k) * w, xg, acc[1][k]);
            if (k & 1) one_at_a_time();
        }
    };
#pragma unroll
    for (int i = 0; i < NIT; ++i)
        if (i * CPB < p.n) {
            d[i] = turned(d[i], i & 1);
            add(i * CPB, x[i], z[i], d[i]);
            // the loaded words alone stay, not their fp32 values beside them
            asm volatile("" : "+v"(x[i].w), "+v"(z[i].w), "+v"(d[i].w));
        }
    const auto stream = [&](int first, auto&& f) {
        Vec sx = me.load(p, p.x, at, c0, first * CPB), sz = me.load(p, p.z, at, c0, first * CPB);
        Vec sd = load_dout(first * CPB);
        for (int i = first; i * CPB < p.n; ++i) {  // one pass ahead
            const Vec nx = me.load(p, p.x, at, c0, (i + 1) * CPB);
            const Vec nz = me.load(p, p.z, at, c0, (i + 1) * CPB);
            const Vec nd = load_dout((i + 1) * CPB);
            f(i, sx, sz, turned(sd, i & 1));
            sx = nx;
            sz = nz;
            sd = nd;
        }
    };
    if constexpr (STREAM)
        stream(NIT, [&](int i, const Vec& ax, const Vec& az, const Vec& ad) {
            add(i * CPB, ax, az, ad);
            if (NL > 0 && i < HELD) {
                held[i - NIT][0][tid] = ax.w;
                held[i - NIT][1][tid] = az.w;
                held[i - NIT][2][tid] = ad.w;
            }
        });
    const float s = tile_sum<2, VE, Sh::VL, Sh::WAVES, TT>(acc, red, tid);
    const float inv_n = 1.0f / static_cast<float>(p.n);
    if (tid < TT) tok[tid] = rstd_of(s, inv_n, p.eps);
    __syncthreads();
    if (tid >= TT && tid < 2 * TT) tok[tid] = tok[tid - TT] * tok[tid - TT] * (s * inv_n);
    __syncthreads();

    // tokens that another tile or vector counts in dweight: those below this place in the tile
    const int skip = max(at.skip, me.early > 0 ? me.vl * VE + me.early : 0);
    float* part = p.dw_part == nullptr ? nullptr : p.dw_part + static_cast<int64_t>(tile) * p.D + c0;
    const auto emit = [&](int c, const Vec& ax, const Vec& az, const Vec& ad) {
        const float w = weight(c);
        float dw = 0.0f;
        Vec ox, oz;
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
            float gx[2], gz[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = me.vl * VE + k + e;
                const float xk = elem_of(ax, k + e), dy = elem_of(ad, k + e);
                const float r = tok[t], cf = tok[TT + t];
                float gate, slope, part_t;
                silu_grad_f(elem_of(az, k + e), gate, slope);
                if constexpr (FIRST) {
                    const float v = xk * gate;
                    const float dv = r * fmaf(-v, cf, dy * w);
                    gx[e] = dv * gate;
                    gz[e] = dv * xk * slope;
                    part_t = dy * (v * r);
                } else {
                    const float xh = xk * r;
                    gx[e] = r * fmaf(-xk, cf, dy * w * gate);
                    gz[e] = dy * w * xh * slope;
                    part_t = dy * gate * xh;
                }
                dw += t >= skip ? part_t : 0.0f;
            }
            set_pair(ox, k, gx[0], gx[1]);
            set_pair(oz, k, gz[0], gz[1]);
            one_at_a_time();
        }
        me.template store<PAST>(p, p.out, at, c0, c, ox);
        me.template store<PAST>(p, p.dz, at, c0, c, oz);
        if (part != nullptr) {
#pragma unroll
            for (int m = 1; m < Sh::VL; m *= 2) dw += __shfl_xor(dw, m);
            if (me.vl == 0 && c + me.ch < p.n) part[MSEL_IDX(c + me.ch, p.n)] = dw;
        }
    };
#pragma unroll
    for (int i = 0; i < NIT; ++i)
        if (i * CPB < p.n) emit(i * CPB, x[i], z[i], d[i]);
    if constexpr (NL > 0)
        for (int i = NIT; i < HELD && i * CPB < p.n; ++i) {
            Vec ax, az, ad;
            ax.w = held[i - NIT][0][tid];
            az.w = held[i - NIT][1][tid];
            ad.w = held[i - NIT][2][tid];
            emit(i * CPB, ax, az, ad);
        }
    if constexpr (STREAM)
        stream(HELD, [&](int i, const Vec& ax, const Vec& az, const Vec& ad) {
            emit(i * CPB, ax, az, ad);
        });
}

template <typename T, bool FIRST, bool DOUT_BLD, int SB, int THREADS, int NIT, int NL,
          bool STREAM, bool PAST>
hipError_t tile_bwd_launch(TileNormParams p, hipStream_t stream) {
    using Sh = TileShape<T, SB, THREADS>;
    p.tiles = (p.L + Sh::TT - 1) / Sh::TT;
    const unsigned tiles = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.tiles);
    const bool one = tiles == 1 && p.dw_part != nullptr;
    // the workspace has a row of partial sums for every tile
    if (p.dw_part != nullptr &&
        tiles > tile_norm_partials(p.B, p.groups, p.n, p.L, sizeof(T) == 2))
        return hipErrorInvalidValue;
    if (one) p.dw_part = p.dw;  // one row of partial sums is the sum
    hipLaunchKernelGGL(
        (tile_norm_bwd_kernel<T, FIRST, DOUT_BLD, SB, THREADS, NIT, NL, STREAM, PAST>),
        tile_grid(tiles, static_cast<unsigned>(p.groups)), dim3(THREADS), 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.dw_part == nullptr || one) return e;
    return launch_column_sums(p.dw_part, tiles, p.D, p.dw, stream);
}

template <typename T, bool FIRST, bool DOUT_BLD, int SB, int THREADS, int NIT, int NL,
          bool STREAM>
hipError_t tile_bwd_go(const TileNormParams& p, hipStream_t stream) {
    // Past the caches in wide tiles with a CU to themselves: 5120 x 16384 bf16 260 us with it, 277
    // without; 8 x 512 x 16384, in two blocks per CU, 195 and 189, and 8 x 1536 x 8192 in narrow
    // tiles, whose stores are half lines, 305 and 293.
    const int64_t bytes = static_cast<int64_t>(p.B) * p.D * p.L * static_cast<int64_t>(sizeof(T));
    if constexpr (THREADS == 1024 && SB == 128)
        if (past_cache(2 * bytes))
            return tile_bwd_launch<T, FIRST, DOUT_BLD, SB, THREADS, NIT, NL, STREAM, true>(p, stream);
    return tile_bwd_launch<T, FIRST, DOUT_BLD, SB, THREADS, NIT, NL, STREAM, false>(p, stream);
}

template <typename T, bool FIRST, bool DOUT_BLD>
hipError_t tile_bwd_width(const TileNormParams& p, hipStream_t stream) {
    // Wide tiles where the group stays on the CU (n <= 768 there) or does not in narrow ones
    // either (5120 x 16384 bf16: 273 us against 337); between the two narrow tiles hold it
    // (8 x 1536 x 2048 from [batch, seqlen, dim]: 72 us against 78).  Narrow groups take smaller
    // blocks, several on a CU (64 x 128 x 4096 fp32: 186 us against 208; in narrow tiles 2000 x 64
    // x 17 bf16: 21 us against 41, 600 x 512 x 17 fp32: 31 against 38).
    constexpr int kBytes = static_cast<int>(sizeof(T));
    const bool wide = p.L >= 128 / kBytes && tile_blocks<T, 128>(p) >= kWideBlocks;
    if (wide && p.n <= 64) return tile_bwd_go<T, FIRST, DOUT_BLD, 128, 128, 4, 0, false>(p, stream);
    if (wide && p.n <= 256) return tile_bwd_go<T, FIRST, DOUT_BLD, 128, 512, 4, 0, false>(p, stream);
    if (wide && (p.n <= 768 || p.n > 1536))
        return tile_bwd_go<T, FIRST, DOUT_BLD, 128, 1024, 4, 2, true>(p, stream);
    if (narrow_bytes(p.B, p.groups, p.n, p.L, kBytes == 2) == 32)
        return tile_bwd_go<T, FIRST, DOUT_BLD, 32, 1024, 4, 2, true>(p, stream);
    if (p.n <= 256) return tile_bwd_go<T, FIRST, DOUT_BLD, 64, 256, 4, 0, false>(p, stream);
    if (p.n <= 512) return tile_bwd_go<T, FIRST, DOUT_BLD, 64, 512, 4, 0, false>(p, stream);
    return tile_bwd_go<T, FIRST, DOUT_BLD, 64, 1024, 4, 2, true>(p, stream);
}

template <typename T>
hipError_t tile_bwd(const TileNormParams& p, bool gate_first, hipStream_t stream) {
    if (gate_first)
        return p.out_bld ? tile_bwd_width<T, true, true>(p, stream)
                         : tile_bwd_width<T, true, false>(p, stream);
    return p.out_bld ? tile_bwd_width<T, false, true>(p, stream)
                     : tile_bwd_width<T, false, false>(p, stream);
}

}  // namespace

int64_t tile_norm_partials(int B, int groups, int n, int L, bool bf16) {
    if (tile_is_short(B, groups, L, bf16)) return tile_short_partials(B, groups, L);
    const int tt = narrow_bytes(B, groups, n, L, bf16) / (bf16 ? 2 : 4);
    return static_cast<int64_t>(B) * ((L + tt - 1) / tt);
}

hipError_t launch_tile_norm_bwd(const TileNormParams& p, bool gate_first, bool bf16,
                                hipStream_t stream) {
    if (tile_is_short(p.B, p.groups, p.L, bf16))
        return launch_tile_short(p, gate_first, bf16, true, stream);
    return bf16 ? tile_bwd<bf16_t>(p, gate_first, stream) : tile_bwd<float>(p, gate_first, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_tile_norm_bwd)

}  // namespace msel
