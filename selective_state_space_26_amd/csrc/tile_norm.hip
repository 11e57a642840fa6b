// tile_norm.hip -- the gated norm after the scan, forward, over the channels of
// [batch, dim, seqlen], to the same layout or turned to [batch, seqlen, dim]:
//   gate first:  v = x silu(z),  out = v rstd(v) w;   gate last:  out = x rstd(x) w silu(z),
//   rstd(v) = (sum over the group's n channels of v^2 / n + eps)^(-1/2).
// HBM bounds it: x and z read, out written (the tiles are described in tile_norm.hpp).  The
// gate's exp and reciprocal are computed once for a pass in registers: gate first keeps v, in the
// registers of x and z (as many in bf16); gate last keeps x and z, and needs the gate for the
// output alone.
// Measured: 5120 x 65536 bf16 to rows 513 us (2.01 GB, 3.9 TB/s; a copy moves 5.1), 8 x 1536 x 2048
// 34 us (151 MB, 4.4 TB/s).  What is missing is overlap: at these widths a CU holds one tile, whose
// loads, arithmetic (VALU busy 40% of the time) and stores follow one another.
#include <hip/hip_runtime.h>

#include "tile_norm.hpp"

namespace msel {

namespace {

// fp32 values in the words of two vectors as loaded: neighbours k, k + 1 of bf16 vectors in the
// words that held their inputs.
template <typename T, int VE>
__device__ __forceinline__ void put_pair(RawVec<T, VE>& a, RawVec<T, VE>& b, int k, float lo,
                                         float hi) {
    if constexpr (sizeof(T) == 4) {
        a.w[k] = __float_as_uint(lo);
        a.w[k + 1] = __float_as_uint(hi);
    } else {
        a.w[k / 2] = __float_as_uint(lo);
        b.w[k / 2] = __float_as_uint(hi);
    }
}
template <typename T, int VE>
__device__ __forceinline__ float kept_elem(const RawVec<T, VE>& a, const RawVec<T, VE>& b, int k) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(a.w[k]);
    else return __uint_as_float(k & 1 ? b.w[k / 2] : a.w[k / 2]);
}

// NIT: passes kept in registers, NL: passes after them kept in LDS (a thread's own words; no
// barrier), STREAM: there may be more, which are read twice.
template <typename T, bool FIRST, bool OUT_BLD, int SB, int THREADS, int NIT, int NL,
          bool STREAM, bool PAST>
__global__ __launch_bounds__(THREADS) void tile_norm_fwd_kernel(TileNormParams p) {
    using Sh = TileShape<T, SB, THREADS>;
    using Rows = RowLane<T, SB, THREADS>;
    constexpr int VE = Sh::VE, TT = Sh::TT, CPB = Sh::CPB;
    __shared__ float red[Sh::WAVES * TT], rstds[TT];
    __shared__ std::conditional_t<OUT_BLD, TurnTile<T, SB, THREADS>, NoTile> turn[2];
    using Vec = RawVec<T, VE>;
    constexpr int HELD = NIT + NL;
    __shared__ decltype(Vec::w) held[NL > 0 ? NL : 1][2][NL > 0 ? THREADS : 1];
    const int tid = threadIdx.x;
    const TileLane<T, SB, THREADS> me(p, tid);
    const int tile = tile_of_block();
    if (tile >= p.B * p.tiles) return;  // block-uniform
    const TilePlace<TT> at(p, tile);
    const int c0 = blockIdx.y * p.n;

    Vec x[NIT > 0 ? NIT : 1], z[NIT > 0 ? NIT : 1];
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
        x[i].w = 0;
        z[i].w = 0;
        if (i * CPB < p.n) {  // block-uniform, here and below
            x[i] = me.load(p, p.x, at, c0, i * CPB);
            z[i] = me.load(p, p.z, at, c0, i * CPB);
        }
    }
    float acc[1][VE] = {};
    const auto add = [&](Vec& ax, Vec& az) {  // gate first: v takes the place of x and z
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                v[e] = elem_of(ax, k + e);
                if constexpr (FIRST) v[e] *= silu_f(elem_of(az, k + e));
                acc[0][k + e] = fmaf(v[e], v[e], acc[0][k + e]);
            }
            if constexpr (FIRST) put_pair(ax, az, k, v[0], v[1]);
            one_at_a_time();
        }
    };
#pragma unroll
    for (int i = 0; i < NIT; ++i)
        if (i * CPB < p.n) add(x[i], z[i]);
    if constexpr (STREAM) {
        // gate last needs z for the output alone
        const auto want_z = [](int i) { return FIRST || i < HELD; };
        Vec sx = me.load(p, p.x, at, c0, NIT * CPB), sz;
        sz.w = 0;
        if (want_z(NIT)) sz = me.load(p, p.z, at, c0, NIT * CPB);
        for (int i = NIT; i * CPB < p.n; ++i) {  // one pass ahead
            Vec nx = me.load(p, p.x, at, c0, (i + 1) * CPB), nz;
            nz.w = 0;
            if (want_z(i + 1)) nz = me.load(p, p.z, at, c0, (i + 1) * CPB);
            add(sx, sz);
            if (NL > 0 && i < HELD) {
                held[i - NIT][0][tid] = sx.w;
                held[i - NIT][1][tid] = sz.w;
            }
            sx = nx;
            sz = nz;
        }
    }
    const float s = tile_sum<1, VE, Sh::VL, Sh::WAVES, TT>(acc, red, tid);
    if (tid < TT) rstds[tid] = rstd_of(s, 1.0f / static_cast<float>(p.n), p.eps);
    __syncthreads();
    float rstd[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) rstd[k] = rstds[me.vl * VE + k];

    // pass i; kept: x and z as add left them
    const auto emit = [&](auto kept, int i, const Vec& ax, const Vec& az) {
        const int c = i * CPB, ch = c + me.ch;
        const float w = ch < p.n && p.w != nullptr ? p.w[MSEL_IDX(c0 + ch, p.D)] : 1.0f;
        Vec o;
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                constexpr bool have = FIRST && kept.value;
                v[e] = have ? kept_elem(ax, az, k + e) : elem_of(ax, k + e);
                if constexpr (!have) v[e] *= silu_f(elem_of(az, k + e));
                v[e] *= rstd[k + e] * w;
            }
            set_pair(o, k, v[0], v[1]);
            one_at_a_time();
        }
        if constexpr (OUT_BLD) {
            turn[i & 1].put_tokens(me.vl, me.ch, o);
            // one barrier per pass: a buffer is written again two passes later, after the barrier
            // of the pass between, hence after every read of it
            __syncthreads();
            Rows::template store<PAST>(p, p.out, at, c0, c, tid, turn[i & 1].get_group(tid));
        } else {
            me.template store<PAST>(p, p.out, at, c0, c, o);
        }
    };
#pragma unroll
    for (int i = 0; i < NIT; ++i)
        if (i * CPB < p.n) emit(std::true_type{}, i, x[i], z[i]);
    if constexpr (NL > 0)
        for (int i = NIT; i < HELD && i * CPB < p.n; ++i) {
            Vec ax, az;
            ax.w = held[i - NIT][0][tid];
            az.w = held[i - NIT][1][tid];
            emit(std::true_type{}, i, ax, az);
        }
    if constexpr (STREAM) {
        Vec sx = me.load(p, p.x, at, c0, HELD * CPB), sz = me.load(p, p.z, at, c0, HELD * CPB);
        for (int i = HELD; i * CPB < p.n; ++i) {
            const Vec nx = me.load(p, p.x, at, c0, (i + 1) * CPB);
            const Vec nz = me.load(p, p.z, at, c0, (i + 1) * CPB);
            emit(std::false_type{}, i, sx, sz);
            sx = nx;
            sz = nz;
        }
    }
}

template <typename T, bool FIRST, bool OUT_BLD, int SB, int THREADS, int NIT, int NL,
          bool STREAM, bool PAST>
hipError_t tile_fwd_launch(TileNormParams p, hipStream_t stream) {
    using Sh = TileShape<T, SB, THREADS>;
    p.tiles = (p.L + Sh::TT - 1) / Sh::TT;
    hipLaunchKernelGGL(
        (tile_norm_fwd_kernel<T, FIRST, OUT_BLD, SB, THREADS, NIT, NL, STREAM, PAST>),
        tile_grid(static_cast<unsigned>(p.B) * static_cast<unsigned>(p.tiles),
                  static_cast<unsigned>(p.groups)),
        dim3(THREADS), 0, stream, p);
    return hipGetLastError();
}

template <typename T, bool FIRST, bool OUT_BLD, int SB, int THREADS, int NIT, int NL,
          bool STREAM>
hipError_t tile_fwd_go(const TileNormParams& p, hipStream_t stream) {
    // Past the caches where a wavefront stores whole lines (rows, or wide tiles) and a block has a
    // CU to itself: 5120 x 65536 bf16 515 us with it, 535 without; 8 x 640 x 16384 fp32, in smaller
    // blocks, 214 and 210.
    const int64_t bytes = static_cast<int64_t>(p.B) * p.D * p.L * static_cast<int64_t>(sizeof(T));
    if constexpr (THREADS == 1024 && (OUT_BLD || SB == 128))
        if (past_cache(bytes))
            return tile_fwd_launch<T, FIRST, OUT_BLD, SB, THREADS, NIT, NL, STREAM, true>(p, stream);
    return tile_fwd_launch<T, FIRST, OUT_BLD, SB, THREADS, NIT, NL, STREAM, false>(p, stream);
}

template <typename T, bool FIRST, bool OUT_BLD>
hipError_t tile_fwd_width(const TileNormParams& p, hipStream_t stream) {
    // Wide tiles where the group stays on the CU (n <= 1536 there) and enough of them fill the
    // chip: 8 x 1536 x 2048 bf16 33-36 us against 43 in tiles of 64 bytes.  Beyond that narrow
    // tiles hold twice the channels: 5120 x 65536 538 us against 597.  Narrow groups take smaller
    // blocks, several on a CU: 8 groups of 640 x 65536 399 us against 427; in narrow tiles 2000 x 64
    // x 17 10 us against 25, 600 x 512 x 17 fp32 13 against 22.
    constexpr int kBytes = static_cast<int>(sizeof(T));
    const bool wide = p.L >= 128 / kBytes && tile_blocks<T, 128>(p) >= kWideBlocks;
    if (wide && p.n <= 64) return tile_fwd_go<T, FIRST, OUT_BLD, 128, 128, 4, 0, false>(p, stream);
    if (wide && p.n <= 640) return tile_fwd_go<T, FIRST, OUT_BLD, 128, 512, 10, 0, false>(p, stream);
    if (wide && p.n <= 1536) return tile_fwd_go<T, FIRST, OUT_BLD, 128, 1024, 9, 3, true>(p, stream);
    if (narrow_bytes(p.B, p.groups, p.n, p.L, kBytes == 2) == 32)
        return tile_fwd_go<T, FIRST, OUT_BLD, 32, 1024, 9, 3, true>(p, stream);
    if (p.n <= 256) return tile_fwd_go<T, FIRST, OUT_BLD, 64, 256, 4, 0, false>(p, stream);
    if (p.n <= 512) return tile_fwd_go<T, FIRST, OUT_BLD, 64, 512, 4, 0, false>(p, stream);
    return tile_fwd_go<T, FIRST, OUT_BLD, 64, 1024, 9, 3, true>(p, stream);
}

template <typename T>
hipError_t tile_fwd(const TileNormParams& p, bool gate_first, hipStream_t stream) {
    if (gate_first)
        return p.out_bld ? tile_fwd_width<T, true, true>(p, stream)
                         : tile_fwd_width<T, true, false>(p, stream);
    return p.out_bld ? tile_fwd_width<T, false, true>(p, stream)
                     : tile_fwd_width<T, false, false>(p, stream);
}

}  // namespace

bool tile_is_short(int B, int groups, int L, bool bf16) {
    const int tt = 64 / (bf16 ? 2 : 4);
    return L < tt / 4 || static_cast<int64_t>(B) * groups * ((L + tt - 1) / tt) < kFewTiles;
}

int narrow_bytes(int B, int groups, int n, int L, bool bf16) {
    const int tt = 64 / (bf16 ? 2 : 4);
    const int64_t tiles = static_cast<int64_t>(B) * groups * ((L + tt - 1) / tt);
    return n > kHalfWidth && tiles < kHalfTiles ? 32 : 64;
}

hipError_t launch_tile_norm_fwd(const TileNormParams& p, bool gate_first, bool bf16,
                                hipStream_t stream) {
    if (tile_is_short(p.B, p.groups, p.L, bf16))
        return launch_tile_short(p, gate_first, bf16, false, stream);
    return bf16 ? tile_fwd<bf16_t>(p, gate_first, stream) : tile_fwd<float>(p, gate_first, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_tile_norm)

}  // namespace msel
