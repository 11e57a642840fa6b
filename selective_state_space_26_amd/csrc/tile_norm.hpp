// tile_norm.hpp -- what the forward and the backward of the gated norm over the channels of
// [batch, dim, seqlen] share (tile_norm.hip, tile_norm_bwd.hip).
//
// The normed axis is strided: token t of channel c lies seqlen elements from channel c + 1's.
// A block takes a tile of TT consecutive tokens of one batch row and one group of n channels.
// A lane loads one 16-byte vector, VE consecutive tokens of one channel; VL = TT / VE lanes
// side by side cover the tile's tokens, and a pass of the block CPB = THREADS / VL channels.
// Sums over channels: each lane over its passes, then over the lanes of a wavefront that hold
// the same tokens, then over the wavefronts through LDS, in a fixed order.
// Rows in [batch, seqlen, dim] are turned through LDS one pass of CPB channels at a time.
#pragma once

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

template <typename T, int TT, int THREADS>
struct TileShape {
    static constexpr int VE = 16 / static_cast<int>(sizeof(T));
    static constexpr int VL = TT / VE;
    static constexpr int CPB = THREADS / VL;
    static constexpr int WAVES = THREADS / 64;
    static constexpr int RV = CPB / VE;          // vectors of a turned row of one pass
    static constexpr int S = CPB + 16 / static_cast<int>(sizeof(T));  // its padded length
    static_assert(TT % VE == 0 && 64 % VL == 0 && TT * RV == THREADS, "one vector per thread");
};

// Consecutive tiles on one XCD: blocks go to the 8 XCDs in turn, and neighbouring tiles share
// cache lines wherever a tile's rows do not start and end on one.
__device__ __forceinline__ unsigned xcd_order(unsigned bid, unsigned n) {
    const unsigned x = bid & 7u, q = n >> 3, r = n & 7u;
    return x * q + (x < r ? x : r) + (bid >> 3);
}

// Sums acc over the lanes of the block that hold the same tokens; red: [WAVES][TT] floats.
// One barrier; the caller puts another between two calls on the same red.
template <int VE, int VL, int WAVES, int TT>
__device__ __forceinline__ void tile_sum(float (&acc)[VE], float* red, int lane, int wave) {
#pragma unroll
    for (int m = VL; m < 64; m *= 2)
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] += __shfl_xor(acc[k], m);
    if (lane < VL) {
#pragma unroll
        for (int k = 0; k < VE; ++k) red[wave * TT + lane * VE + k] = acc[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VE; ++k) acc[k] = 0.0f;
    const int vl = lane % VL;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
        for (int k = 0; k < VE; ++k) acc[k] += red[w * TT + vl * VE + k];
}

// A pass's turned tile in LDS: TT rows of CPB channels, padded to S.
template <typename T, int TT, int THREADS>
struct TurnTile {
    using Sh = TileShape<T, TT, THREADS>;
    T v[TT * Sh::S];

    // this thread's VE tokens of one channel
    __device__ __forceinline__ void put_tokens(int vl, int ch, const float (&o)[Sh::VE]) {
#pragma unroll
        for (int k = 0; k < Sh::VE; ++k)
            Elem<T>::store1(v + MSEL_IDX((vl * Sh::VE + k) * Sh::S + ch, TT * Sh::S), o[k]);
    }
    __device__ __forceinline__ void get_tokens(int vl, int ch, float (&o)[Sh::VE]) const {
#pragma unroll
        for (int k = 0; k < Sh::VE; ++k)
            o[k] = Elem<T>::load1(v + MSEL_IDX((vl * Sh::VE + k) * Sh::S + ch, TT * Sh::S));
    }
    // VE channels of one token (16-byte aligned)
    __device__ __forceinline__ void put_channels(int row, int cv, const RawVec<T, Sh::VE>& r) {
        *reinterpret_cast<decltype(r.w)*>(v + MSEL_SPAN(row * Sh::S + cv, Sh::VE, TT * Sh::S)) =
            r.w;
    }
    __device__ __forceinline__ RawVec<T, Sh::VE> get_channels(int row, int cv) const {
        RawVec<T, Sh::VE> r;
        r.w = *reinterpret_cast<const decltype(r.w)*>(
            v + MSEL_SPAN(row * Sh::S + cv, Sh::VE, TT * Sh::S));
        return r;
    }
};

}  // namespace msel
