// tile_norm.hpp -- what the forward and the backward of the gated norm over the channels of
// [batch, dim, seqlen] share (tile_norm.hip, tile_norm_bwd.hip).
//
// The normed axis is strided: token t of channel c lies seqlen elements from channel c + 1's.
// A block takes a tile of TT consecutive tokens of one batch row, SB bytes of the row of each of
// the n channels of a group: a lane loads one 16-byte vector, VE consecutive tokens of one
// channel; VL = TT / VE lanes side by side cover the tile's tokens and a pass of the block takes
// CPB channels.  Sums over channels: each lane over its passes, then over the lanes of a
// wavefront that hold the same tokens, then over the wavefronts through LDS, in a fixed order.
// Rows in [batch, seqlen, dim] are turned through LDS, a pass at a time.
//
// A tile's first passes stay in registers and LDS from the sums to the outputs; passes beyond
// them are read twice.  Reading is faster in wide tiles (two 671 MB tensors of 5120 rows in 221 us
// at SB = 256, 264 at 128, 306 at 64, 400 at 32), but a wide tile holds fewer channels, and two
// blocks on a CU, one loading while the other computes, are faster than one of twice the size.
// The launchers choose by n.
// Measured and not kept: blocks that walk tiles and load a pass of the next tile as they write
// one of the current (neighbouring tiles then run apart and no longer share cache lines: 790 us
// against 650 for the forward of 5120 x 65536 at SB = 32), and, for the forward, two kernels, sums
// and then outputs with all inputs read twice at SB = 256 (663 against 621 us there; 52 against 43
// for 8 x 1536 x 2048; with outputs through the caches).
//
// A last tile that is not full starts early, at seqlen - TT, and does the tokens it shares with
// the tile before it again (the same values in the same order, so the same bits; the backward
// leaves them out of dweight).  Within a tile, the last vectors of a sequence shorter than the
// tile start early in the same way.  Sequences shorter than a vector, and calls with few tiles, go
// to the kernels of tile_short.hip.
#pragma once

#include <algorithm>
#include <type_traits>

#include "lm_device.hpp"
#include "lm_kernels.hpp"

namespace msel {

template <typename T, int SB, int THREADS>
struct TileShape {
    static constexpr int VE = 16 / static_cast<int>(sizeof(T));
    static constexpr int TT = SB / static_cast<int>(sizeof(T));
    static constexpr int VL = SB / 16;
    static constexpr int CPB = THREADS / VL;        // channels per pass
    static constexpr int WAVES = THREADS / 64;
    static_assert(64 % VL == 0, "whole vectors of tokens");
};

// Blocks of a launch in tiles of SB bytes, and how many wide ones (SB = 128) make them worth it.
// us in wide tiles against the narrower ones, bf16 to and from rows:
//   128 blocks: 700 channels forward 14 and 11, backward 26 and 21; 5120 backward 185 and 167
//   192 blocks: 700 forward 16 and 17, backward 30 and 34; 5120 backward 229 and 250
//   256 blocks: 700 forward 17 and 19, backward 33 and 39; 5120 backward 265 and 291
//   800 blocks: 700 forward 58 and 62, backward 113 and 138; 5120 backward 889 and 860
// (with 256 channels and fewer the two differ by 10% at most at any of these).
template <typename T, int SB>
inline int64_t tile_blocks(const TileNormParams& p) {
    constexpr int TT = SB / static_cast<int>(sizeof(T));
    return static_cast<int64_t>(p.B) * p.groups * ((p.L + TT - 1) / TT);
}
constexpr int kWideBlocks = 224;
// Fewer tiles of 64 bytes than this go to tile_short.hip (1 x 8192 x 31 bf16, one tile, backward:
// 36 us there, 63 in tiles of 32; 1 x 5120 x 250, 8 tiles: 56 and 46).
constexpr int kFewTiles = 6;
// With fewer tiles of 64 bytes than this, wide groups go in tiles of 32: neighbouring tiles share
// lines, and run on one XCD (5120 x 4096 bf16, 128 tiles of 64: forward 63 us, 48 in tiles of 32,
// backward 119 and 89; 2560 x 6000, 188 tiles: 21 and 27, 50 and 64).
constexpr int kHalfTiles = 160;
constexpr int kHalfWidth = 512;

// Element k of a vector as loaded, and the other way round for two neighbours: unlike to_f32 and
// from_f32 these keep few fp32 values alive.
template <typename T, int VE>
__device__ __forceinline__ float elem_of(const RawVec<T, VE>& r, int k) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[k]);
    else return k & 1 ? bf16hi(r.w[k / 2]) : bf16lo(r.w[k / 2]);
}
template <typename T, int VE>
__device__ __forceinline__ void set_pair(RawVec<T, VE>& r, int k, float lo, float hi) {
    if constexpr (sizeof(T) == 4) {
        r.w[k] = __float_as_uint(lo);
        r.w[k + 1] = __float_as_uint(hi);
    } else {
        r.w[k / 2] = pack_bf16(lo, hi);
    }
}

// Keeps the scheduler from working on many elements at once, which costs registers that hold
// passes (the wavefronts hide the latencies).
__device__ __forceinline__ void one_at_a_time() { __builtin_amdgcn_sched_barrier(0); }

// One level of a sum over lanes: lanes l and l ^ M share their N values out, so that each is
// left with N / 2 sums (the upper half of the values where the lane's bit M is set); N = 1 adds.
template <int M, int N>
__device__ __forceinline__ void share_sums(float* v, int lane) {
    if constexpr (N > 1) {
        const bool up = (lane & M) != 0;
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const float give = up ? v[k] : v[k + N / 2];
            const float keep = up ? v[k + N / 2] : v[k];
            v[k] = keep + __shfl_xor(give, M);
        }
    } else {
        v[0] += __shfl_xor(v[0], M);
    }
}
template <int M, int N, int VL>
__device__ __forceinline__ void share_levels(float* v, int lane) {
    if constexpr (M >= VL) {
        share_sums<M, N>(v, lane);
        share_levels<M / 2, (N > 1 ? N / 2 : 1), VL>(v, lane);
    }
}

// Sums NS values per token (VE tokens per lane) over the lanes of the block that hold the same
// tokens; red: [NS][WAVES][TT] floats of LDS.  Returns sum tid / TT of token tid % TT in threads
// below NS * TT.  A wavefront's lanes share the values out between them, so a level moves half
// as many as the one before.  One barrier.
template <int NS, int VE, int VL, int WAVES, int TT>
__device__ __forceinline__ float tile_sum(float (&acc)[NS][VE], float* red, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
    constexpr int LEVELS = VL == 32 ? 1 : VL == 16 ? 2 : VL == 8 ? 3 : VL == 4 ? 4 : 5;  // log2(64 / VL)
    constexpr int BITS = VE == 8 ? 3 : 2;                                  // log2(VE)
    constexpr int SHARED = LEVELS < BITS ? LEVELS : BITS;  // levels that halve the values
    constexpr int LEFT = VE >> SHARED;
    static_assert(VL >= 2 && NS * TT <= WAVES * 64, "a thread per sum");
    // the lane's values start where its bits 5, 4, .. say; of the lanes that only added, the
    // first writes
    const int first = ((lane >> (6 - SHARED)) & ((1 << SHARED) - 1)) * LEFT;
    const int rest = lane & ((1 << (6 - SHARED)) - 1);  // lane within its values' holders
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        share_levels<32, VE, VL>(acc[s], lane);
        if (rest < VL) {
#pragma unroll
            for (int k = 0; k < LEFT; ++k)
                red[(s * WAVES + wave) * TT + (lane % VL) * VE + first + k] = acc[s][k];
        }
    }
    __syncthreads();
    float v = 0.0f;
    if (tid < NS * TT) {
        const int s = tid / TT, t = tid % TT;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += red[(s * WAVES + w) * TT + t];
    }
    return v;
}

// A tile's first token, and how many of its tokens the tile before has done (block-uniform).
template <int TT>
struct TilePlace {
    int b, t0, skip;

    __device__ __forceinline__ TilePlace(const TileNormParams& p, int tile) {
        b = tile / p.tiles;
        const int t = (tile - b * p.tiles) * TT;
        t0 = max(0, min(t, p.L - TT));
        skip = t - t0;
    }
};

// A thread's part of a tile.  Addresses are a block-uniform element plus the thread's offset.
template <typename T, int SB, int THREADS>
struct TileLane {
    using Sh = TileShape<T, SB, THREADS>;
    static constexpr int VE = Sh::VE;
    int vl, ch;   // vector of the tile's tokens, channel within a pass
    int early;    // tokens by which the vector starts early (they are the vector before's)
    int64_t off;  // ch * L + the vector's first token

    __device__ __forceinline__ TileLane(const TileNormParams& p, int tid) {
        vl = tid % Sh::VL;
        ch = tid / Sh::VL;
        early = max(0, (vl + 1) * VE - p.L);
        off = static_cast<int64_t>(ch) * p.L + vl * VE - early;
    }
    // element of this lane's tokens of channel c + ch of the group that starts at channel c0
    __device__ __forceinline__ int64_t at(const TileNormParams& p, const TilePlace<Sh::TT>& pl,
                                          int c0, int c) const {
        const int64_t first = (static_cast<int64_t>(pl.b) * p.D + c0 + c) * p.L + pl.t0;
        return MSEL_SPAN(first + off, VE, static_cast<int64_t>(p.B) * p.D * p.L);
    }
    __device__ __forceinline__ RawVec<T, VE> load(const TileNormParams& p, const void* q,
                                                  const TilePlace<Sh::TT>& pl, int c0,
                                                  int c) const {
        RawVec<T, VE> r;
        r.w = 0;
        if (c + ch < p.n) r = ld_raw<T, VE>(static_cast<const T*>(q) + at(p, pl, c0, c));
        return r;
    }
    template <bool PAST = false>
    __device__ __forceinline__ void store(const TileNormParams& p, void* q,
                                          const TilePlace<Sh::TT>& pl, int c0, int c,
                                          const RawVec<T, VE>& r) const {
        if (c + ch < p.n) st_raw<T, VE, PAST>(static_cast<T*>(q) + at(p, pl, c0, c), r);
    }
};

// A pass in LDS, TT rows of its CPB channels, between [batch, dim, seqlen] and
// [batch, seqlen, dim].  16-byte groups of a row are swapped by the row's vector of tokens, which
// spreads the accesses of a pass over the banks.
template <typename T, int SB, int THREADS>
struct TurnTile {
    using Sh = TileShape<T, SB, THREADS>;
    static constexpr int VE = Sh::VE, TT = Sh::TT, CH = Sh::CPB;
    static constexpr int G = CH / VE;  // groups per row: a group per thread
    static constexpr int kElems = TT * CH;
    static_assert(TT * G == THREADS && (G & (G - 1)) == 0, "a group per thread");
    T v[kElems] __attribute__((aligned(16)));

    __device__ __forceinline__ static int place(int row, int g) {
        return row * CH + (g ^ (row / VE & (G - 1))) * VE;
    }
    // VE tokens of channel c
    __device__ __forceinline__ void put_tokens(int vl, int c, const RawVec<T, VE>& o) {
        T* col = v + MSEL_SPAN(place(vl * VE, c / VE) + c % VE, (VE - 1) * CH + 1, kElems);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            T& to = col[k * CH];
            if constexpr (sizeof(T) == 4) to = __uint_as_float(o.w[k]);
            else to.bits = static_cast<uint16_t>(k & 1 ? o.w[k / 2] >> 16 : o.w[k / 2]);
        }
    }
    __device__ __forceinline__ RawVec<T, VE> get_tokens(int vl, int c) const {
        const T* col = v + MSEL_SPAN(place(vl * VE, c / VE) + c % VE, (VE - 1) * CH + 1, kElems);
        RawVec<T, VE> o;
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            const T& at = col[k * CH];
            if constexpr (sizeof(T) == 4) o.w[k] = __float_as_uint(at);
            else if (k & 1) o.w[k / 2] |= static_cast<uint32_t>(at.bits) << 16;
            else o.w[k / 2] = at.bits;
        }
        return o;
    }
    __device__ __forceinline__ void put_group(int tid, const RawVec<T, VE>& r) {
        *reinterpret_cast<decltype(RawVec<T, VE>::w)*>(
            v + MSEL_SPAN(place(tid / G, tid % G), VE, kElems)) = r.w;
    }
    __device__ __forceinline__ RawVec<T, VE> get_group(int tid) const {
        RawVec<T, VE> r;
        r.w = *reinterpret_cast<const decltype(r.w)*>(
            v + MSEL_SPAN(place(tid / G, tid % G), VE, kElems));
        return r;
    }
};
struct NoTile {};  // of a kernel that turns nothing

// The thread's group of a pass in [batch, L, D]: VE channels, from c on, of the group at c0.
template <typename T, int SB, int THREADS>
struct RowLane {
    using Sh = TileShape<T, SB, THREADS>;
    static constexpr int VE = Sh::VE, G = Sh::CPB / VE;

    __device__ __forceinline__ static int64_t at(const TileNormParams& p,
                                                 const TilePlace<Sh::TT>& pl, int c0, int c,
                                                 int tid) {
        const int row = tid / G, token = row - max(0, row / VE * VE + VE - p.L);
        const int64_t i =
            (static_cast<int64_t>(pl.b) * p.L + pl.t0 + token) * p.D + c0 + c + tid % G * VE;
        return MSEL_SPAN(i, min(p.n - c - tid % G * VE, VE), static_cast<int64_t>(p.B) * p.D * p.L);
    }
    __device__ __forceinline__ static RawVec<T, VE> load(const TileNormParams& p, const void* q,
                                                         const TilePlace<Sh::TT>& pl, int c0,
                                                         int c, int tid) {
        const int left = p.n - c - tid % G * VE;
        RawVec<T, VE> r;
        r.w = 0;
        if (left > 0)
            r = ld_part<T, VE>(static_cast<const T*>(q) + at(p, pl, c0, c, tid), left);
        return r;
    }
    template <bool PAST = false>
    __device__ __forceinline__ static void store(const TileNormParams& p, void* q,
                                                 const TilePlace<Sh::TT>& pl, int c0, int c,
                                                 int tid, const RawVec<T, VE>& r) {
        const int left = p.n - c - tid % G * VE;
        if (left > 0)
            st_part<T, VE, PAST>(static_cast<T*>(q) + at(p, pl, c0, c, tid), r, left);
    }
};

}  // namespace msel
