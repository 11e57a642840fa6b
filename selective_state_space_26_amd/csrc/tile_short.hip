// tile_short.hip -- the gated norm over the channels of [batch, dim, seqlen] for sequences of less
// than a 16-byte vector and for calls of a few tiles: forward and backward (the formulas stand in
// tile_norm.hip and tile_norm_bwd.hip).
//
// A block takes `tg` tokens of one batch row and group, 1 to 7, a thread one token and every C-th
// channel, C = kThreads / tg: neighbouring threads hold neighbouring tokens, so a step of the
// block reads C runs of tg elements.  A short sequence is read whole where there are blocks enough;
// otherwise tg is small, mostly 1: a thread reads single elements a row apart, and the blocks of
// neighbouring tokens read the same lines, which their XCD's cache holds (xcd_order).  Such calls
// are small: what counts is the number of blocks and of loads in flight (U per tensor and thread),
// not the width of a load.  Sums over channels: each thread over its steps, then a tree over the C
// threads of a token in LDS.  Rows in [batch, seqlen, dim] pass through LDS, U steps at a time.
// Measured: 3 x 6016 x 4 bf16 forward 10 us, backward 22; 1 x 8192 x 31 14 and 34, latency of a few
// blocks all of them.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

namespace {

constexpr int kThreads = 1024;
constexpr int U = 8;

// This thread's place.
struct ShortPlace {
    int C;           // channels per step
    int t, c;        // token within the block's, channel within a step
    int nt;          // tokens of the block
    bool on;
    int tile, b, t0, c0;  // of the launch; batch row, first token, first channel of the group
    int64_t at;      // element of channel c0 + c at token t0 + t

    __device__ __forceinline__ ShortPlace(const TileNormParams& p, int tg) {
        const int tid = threadIdx.x;
        C = kThreads / tg;
        t = tid % tg;
        c = tid / tg;
        tile = tile_of_block();
        b = tile / p.tiles;
        t0 = (tile - b * p.tiles) * tg;
        c0 = blockIdx.y * p.n;
        nt = min(tg, p.L - t0);
        on = c < C && t < nt;
        at = (static_cast<int64_t>(b) * p.D + c0 + c) * p.L + t0 + t;
    }
};

// Sums v over the threads of each token (c < C), in a tree whose shape C alone fixes; red:
// kThreads floats.  Returned in every thread.
__device__ __forceinline__ float token_sum(const ShortPlace& me, int tg, float v, float* red) {
    const int tid = threadIdx.x;
    red[tid] = me.on ? v : 0.0f;
    int half = 1;
    while (half < me.C) half *= 2;
    for (half /= 2; half > 0; half /= 2) {  // block-uniform
        __syncthreads();
        if (me.c < half && me.c + half < me.C) red[tid] += red[tid + half * tg];
    }
    __syncthreads();
    const float s = red[me.t];
    __syncthreads();
    return s;
}

template <typename T, bool FIRST, bool OUT_BLD>
__global__ __launch_bounds__(kThreads) void tile_short_fwd_kernel(TileNormParams p, int tg) {
    __shared__ float red[kThreads];
    __shared__ T turn[OUT_BLD ? kThreads * U : 1];
    const ShortPlace me(p, tg);
    if (me.tile >= p.B * p.tiles) return;  // block-uniform
    [[maybe_unused]] const int64_t elems = static_cast<int64_t>(p.B) * p.D * p.L;
    const T* x = static_cast<const T*>(p.x);
    const T* z = static_cast<const T*>(p.z);
    const int CU = me.C * U;
    float acc = 0.0f;
    for (int cb = 0; cb < p.n; cb += CU) {  // block-uniform, here and below
        float xv[U], zv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = cb + u * me.C;
            const bool in = me.on && c + me.c < p.n;
            const int64_t i = in ? MSEL_IDX(me.at + static_cast<int64_t>(c) * p.L, elems) : 0;
            xv[u] = in ? Elem<T>::load1(x + i) : 0.0f;
            zv[u] = in && FIRST ? Elem<T>::load1(z + i) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float v = FIRST ? xv[u] * silu_f(zv[u]) : xv[u];
            acc = fmaf(v, v, acc);
        }
    }
    const float rstd = rstd_of(token_sum(me, tg, acc, red), 1.0f / static_cast<float>(p.n), p.eps);
    T* out = static_cast<T*>(p.out);
    for (int cb = 0; cb < p.n; cb += CU) {
        float xv[U], zv[U], w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = cb + u * me.C;
            const bool in = me.on && c + me.c < p.n;
            const int64_t i = in ? MSEL_IDX(me.at + static_cast<int64_t>(c) * p.L, elems) : 0;
            xv[u] = in ? Elem<T>::load1(x + i) : 0.0f;
            zv[u] = in ? Elem<T>::load1(z + i) : 0.0f;
            w[u] = in && p.w != nullptr ? p.w[MSEL_IDX(me.c0 + c + me.c, p.D)] : 1.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = cb + u * me.C;
            const float o = xv[u] * silu_f(zv[u]) * (rstd * w[u]);
            if (OUT_BLD) {
                if (me.on)
                    Elem<T>::store1(turn + MSEL_IDX(me.t * CU + u * me.C + me.c, kThreads * U), o);
            } else if (me.on && c + me.c < p.n) {
                Elem<T>::store1(out + MSEL_IDX(me.at + static_cast<int64_t>(c) * p.L, elems), o);
            }
        }
        if constexpr (OUT_BLD) {
            __syncthreads();
            const int width = min(CU, p.n - cb);
            for (int t = threadIdx.x / 64; t < me.nt; t += kThreads / 64)
                for (int c = lane_id(); c < width; c += 64)
                    out[MSEL_IDX((static_cast<int64_t>(me.b) * p.L + me.t0 + t) * p.D + me.c0 + cb + c,
                                 elems)] = turn[t * CU + c];
            __syncthreads();
        }
    }
}

template <typename T, bool FIRST, bool DOUT_BLD>
__global__ __launch_bounds__(kThreads) void tile_short_bwd_kernel(TileNormParams p, int tg) {
    __shared__ float red[kThreads];
    __shared__ float dws[kThreads];
    __shared__ T turn[DOUT_BLD ? kThreads * U : 1];
    const ShortPlace me(p, tg);
    if (me.tile >= p.B * p.tiles) return;  // block-uniform
    [[maybe_unused]] const int64_t elems = static_cast<int64_t>(p.B) * p.D * p.L;
    const T* x = static_cast<const T*>(p.x);
    const T* z = static_cast<const T*>(p.z);
    const T* dout = static_cast<const T*>(p.dout);
    const int CU = me.C * U;
    float xv[U], zv[U], dy[U], w[U];
    const auto load = [&](int cb) {
        if constexpr (DOUT_BLD) {
            __syncthreads();  // turn is free
            const int width = min(CU, p.n - cb);
            for (int t = threadIdx.x / 64; t < me.nt; t += kThreads / 64)
                for (int c = lane_id(); c < width; c += 64)
                    turn[MSEL_IDX(t * CU + c, kThreads * U)] =
                        dout[MSEL_IDX((static_cast<int64_t>(me.b) * p.L + me.t0 + t) * p.D +
                                          me.c0 + cb + c,
                                      elems)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = cb + u * me.C;
            const bool in = me.on && c + me.c < p.n;
            const int64_t i = in ? MSEL_IDX(me.at + static_cast<int64_t>(c) * p.L, elems) : 0;
            xv[u] = in ? Elem<T>::load1(x + i) : 0.0f;
            zv[u] = in ? Elem<T>::load1(z + i) : 0.0f;
            if constexpr (!DOUT_BLD) dy[u] = in ? Elem<T>::load1(dout + i) : 0.0f;
            w[u] = in && p.w != nullptr ? p.w[MSEL_IDX(me.c0 + c + me.c, p.D)] : 1.0f;
        }
        if constexpr (DOUT_BLD) {
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = me.on && cb + u * me.C + me.c < p.n;
                dy[u] = in ? Elem<T>::load1(turn + MSEL_IDX(me.t * CU + u * me.C + me.c, kThreads * U))
                           : 0.0f;
            }
        }
    };
    float sv = 0.0f, sg = 0.0f;
    for (int cb = 0; cb < p.n; cb += CU) {  // block-uniform, here and below
        load(cb);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float xg = xv[u] * silu_f(zv[u]);
            const float v = FIRST ? xg : xv[u];
            sv = fmaf(v, v, sv);
            sg = fmaf(dy[u] * w[u], xg, sg);  // g v in either order
        }
    }
    const float inv_n = 1.0f / static_cast<float>(p.n);
    const float rstd = rstd_of(token_sum(me, tg, sv, red), inv_n, p.eps);
    const float cf = rstd * rstd * (token_sum(me, tg, sg, red) * inv_n);
    T* dx = static_cast<T*>(p.out);
    T* dz = static_cast<T*>(p.dz);
    for (int cb = 0; cb < p.n; cb += CU) {
        load(cb);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = cb + u * me.C;
            float gate, slope, gx, gz, dw;
            silu_grad_f(zv[u], gate, slope);
            if constexpr (FIRST) {
                const float v = xv[u] * gate;
                const float dv = rstd * fmaf(-v, cf, dy[u] * w[u]);
                gx = dv * gate;
                gz = dv * xv[u] * slope;
                dw = dy[u] * (v * rstd);
            } else {
                const float xh = xv[u] * rstd;
                gx = rstd * fmaf(-xv[u], cf, dy[u] * w[u] * gate);
                gz = dy[u] * w[u] * xh * slope;
                dw = dy[u] * gate * xh;
            }
            if (me.on && c + me.c < p.n) {
                const int64_t i = MSEL_IDX(me.at + static_cast<int64_t>(c) * p.L, elems);
                Elem<T>::store1(dx + i, gx);
                Elem<T>::store1(dz + i, gz);
            }
            if (p.dw_part != nullptr) {  // grid-uniform: a channel's tokens, added in token order
                __syncthreads();
                dws[threadIdx.x] = me.on ? dw : 0.0f;
                __syncthreads();
                if (me.t == 0 && me.on && c + me.c < p.n) {
                    float s = 0.0f;
                    for (int t = 0; t < me.nt; ++t) s += dws[threadIdx.x + t];
                    p.dw_part[static_cast<int64_t>(me.tile) * p.D +
                              MSEL_IDX(me.c0 + c + me.c, p.D)] = s;
                }
            }
        }
    }
}

// Tokens per block: all of a sequence below a vector (less than 8), fewer until the launch has 160
// blocks.  With fewer blocks CUs stand idle (bf16, forward and backward: 20 x 8192 x 7 47 and 87 us
// in 20 blocks of 7 tokens, 17 and 37 in 80 of 2, 12 and 28 in 140 of one; 64 x 2048 x 7 15 and 29
// in 64 blocks, 9 and 18 in 256); with more, too many blocks read each line (512 x 2048 x 7 26 and
// 68 us in 512 blocks of 7, 61 and 196 in 3584 of one).  Longer sequences come here in so few tiles
// that even blocks of one token are 160 at most (1 x 8192 x 31: 188 and 442 us in one block, 14 and
// 34 in 31).
constexpr int kShort = 8;
int short_tokens(int B, int groups, int L) {
    int tg = L < kShort ? L : 1;
    while (tg > 1 && static_cast<int64_t>(B) * groups * ((L + tg - 1) / tg) < 160) tg = (tg + 1) / 2;
    return tg;
}

template <typename T, bool FIRST, bool BLD>
hipError_t short_go(TileNormParams p, bool bwd, hipStream_t stream) {
    const int tg = short_tokens(p.B, p.groups, p.L);
    p.tiles = (p.L + tg - 1) / tg;
    const unsigned tiles = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.tiles);
    const dim3 grid = tile_grid(tiles, static_cast<unsigned>(p.groups));
    if (!bwd) {
        hipLaunchKernelGGL((tile_short_fwd_kernel<T, FIRST, BLD>), grid, dim3(kThreads), 0, stream,
                           p, tg);
        return hipGetLastError();
    }
    const bool one = tiles == 1 && p.dw_part != nullptr;
    if (one) p.dw_part = p.dw;  // one row of partial sums is the sum
    hipLaunchKernelGGL((tile_short_bwd_kernel<T, FIRST, BLD>), grid, dim3(kThreads), 0, stream, p,
                       tg);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.dw_part == nullptr || one) return e;
    return launch_column_sums(p.dw_part, tiles, p.D, p.dw, stream);
}

template <typename T>
hipError_t short_type(const TileNormParams& p, bool first, bool bwd, hipStream_t stream) {
    if (first)
        return p.out_bld ? short_go<T, true, true>(p, bwd, stream)
                         : short_go<T, true, false>(p, bwd, stream);
    return p.out_bld ? short_go<T, false, true>(p, bwd, stream)
                     : short_go<T, false, false>(p, bwd, stream);
}

}  // namespace

int64_t tile_short_partials(int B, int groups, int L) {
    const int tg = short_tokens(B, groups, L);
    return static_cast<int64_t>(B) * ((L + tg - 1) / tg);
}

hipError_t launch_tile_short(const TileNormParams& p, bool gate_first, bool bf16, bool bwd,
                             hipStream_t stream) {
    return bf16 ? short_type<bf16_t>(p, gate_first, bwd, stream)
                : short_type<float>(p, gate_first, bwd, stream);
}

MSEL_BOUNDS_TAKER(take_bounds_tile_short)

}  // namespace msel
